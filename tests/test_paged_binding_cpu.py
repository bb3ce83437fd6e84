"""The page pool's planes as the binding hands them to the library: a plane that
was replaced by another tensor is checked again before the next call."""
import pytest
import torch

from fp4_kv_cache_append_b200 import csa2 as C


@pytest.mark.parametrize("plane,other", [
    ("codes", lambda t: t[:3]), ("codes", lambda t: t[..., :32]), ("scales", lambda t: t.float()),
    ("refs", lambda t: t.long()), ("refs", lambda t: t[:2]), ("table", lambda t: t[:, :2]),
    ("table", lambda t: torch.zeros(3, 2, dtype=torch.int32).t()), ("n_entries", lambda t: t[:1])])
def test_replaced_planes_are_checked(plane, other):
    if torch.cuda.is_available():
        pytest.skip("host tensors are refused earlier where there is a GPU")
    p = C.PagePool(4, 16, 2, 3, 128, device="cpu")
    assert p.desc().n_pages == 4
    setattr(p, plane, getattr(p, plane).clone())
    assert p.desc().codes == p.codes.data_ptr() and p.desc().table == p.table.data_ptr()
    setattr(p, plane, other(getattr(p, plane)))
    with pytest.raises(ValueError):
        p.desc()
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        C.csa2_pages_fork(p, one, one, ws=torch.zeros(4096, dtype=torch.uint8))
