"""Host-side refusals of the paged cache and the dense attentions (no GPU
work): each bad argument is reported before anything is enqueued."""
import ctypes

import pytest
import torch

from fp4_kv_cache_append_b200 import csa2 as C

P = ctypes.c_void_p(16)
OUT = ctypes.c_void_p(1 << 40)      # behind any q at P
BIG = 1 << 40


def pool(**kw):
    d = dict(codes=16, scales=16, refs=16, table=16, n_entries=16, n_pages=8, page=16, n_seq=2, max_pages=4, D=512, m=1)
    d.update(kw)
    return ctypes.byref(C.PagePoolDesc(*d.values()))


def swa(**kw):
    d = dict(rows=16, scale=1.0, B=2, W_cap=256, D=512, window=128)
    d.update(kw)
    return ctypes.byref(C.SwaCacheDesc(*d.values()))


def main(**kw):
    d = dict(codes=32, scales=32, ik=32, ik_scale=32, n_entries=32, pk=32, pg=32, B=2, cap=128, D=512, d_I=64, m=1)
    d.update(kw)
    return ctypes.byref(C.MainCacheDesc(*d.values()))


@pytest.mark.parametrize("bad,status", [
    (dict(codes=None), 1), (dict(table=None), 1), (dict(refs=20), 1), (dict(n_pages=0), 1), (dict(max_pages=-1), 1),
    (dict(page=8), 2), (dict(page=24), 2), (dict(page=8192), 2), (dict(n_pages=1 << 28), 2), (dict(D=384), 2),
    (dict(m=3), 2), (dict(n_seq=0), 1)])
def test_pool_is_checked_by_every_entry(bad, status):
    L = C.lib()
    p = pool(**bad)
    assert L.csa2_pages_append(p, main(), None, P, None, P, BIG, None) == status
    assert L.csa2_pages_fork(p, P, P, 2, P, BIG, None) == status
    assert L.csa2_pages_compact(p, None, P, BIG, None) == status
    assert L.csa2_prefix_attn_decode(p, P, 0, None, P, P, 2, 1, 64, 1.0, P, P, BIG, None) == status
    assert C.lib().csa2_last_error().decode() != ""


def test_pages_refusals():
    L = C.lib()
    odd = ctypes.c_void_p(20)
    assert L.csa2_pages_append(None, main(), None, P, None, P, BIG, None) == 1
    assert L.csa2_pages_append(pool(), None, None, P, None, P, BIG, None) == 1
    assert L.csa2_pages_append(pool(), main(D=256), None, P, None, P, BIG, None) == 1
    assert L.csa2_pages_append(pool(), main(codes=16), None, P, None, P, BIG, None) == 1
    assert L.csa2_pages_append(pool(), main(), None, None, None, P, BIG, None) == 1
    assert L.csa2_pages_append(pool(), main(), odd, P, None, P, BIG, None) == 1
    assert L.csa2_pages_append(pool(), main(), None, P, odd, P, BIG, None) == 1
    assert L.csa2_pages_append(pool(), main(B=5000), None, P, None, P, BIG, None) == 2
    assert L.csa2_pages_append(pool(), main(), None, P, None, P, 8, None) == 5
    assert L.csa2_pages_append(pool(), main(), None, P, None, None, BIG, None) == 5
    assert L.csa2_pages_fork(pool(), None, P, 2, P, BIG, None) == 1
    assert L.csa2_pages_fork(pool(), P, P, 0, P, BIG, None) == 2
    assert L.csa2_pages_fork(pool(), P, P, 4097, P, BIG, None) == 2
    assert L.csa2_pages_fork(pool(), P, P, 2, P, 8, None) == 5
    assert L.csa2_pages_compact(pool(), odd, P, BIG, None) == 1
    assert L.csa2_pages_compact(pool(), None, P, 8, None) == 5
    assert L.csa2_pages_workspace_size(pool(), 0) == 0
    assert L.csa2_pages_workspace_size(pool(), 3) > 0


def test_attention_refusals():
    L = C.lib()
    odd = ctypes.c_void_p(18)

    def prefix(p=None, seq=P, n_shared=0, w=None, q=P, pos=P, B=2, T=1, H=64, out=OUT):
        return L.csa2_prefix_attn_decode(p or pool(), seq, n_shared, w, q, pos, B, T, H, 1.0, out, P, BIG, None)

    assert prefix(seq=None) == 1 and prefix(q=odd) == 1 and prefix(pos=None) == 1 and prefix(out=odd) == 1
    assert prefix(n_shared=-1) == 1 and prefix(n_shared=65) == 1
    assert prefix(B=0) == 1 and prefix(T=0) == 1 and prefix(B=300, T=300) == 1
    assert prefix(H=0) == 2 and prefix(H=65) == 2
    assert prefix(w=swa(B=3)) == 1 and prefix(w=swa(D=256)) == 1 and prefix(w=swa(window=2000, W_cap=4000)) == 1

    def window(w=None, k=None, q=P, T=1, H=64, out=OUT):
        return L.csa2_window_attn(w or swa(), k, q, P, T, H, 1.0, out, P, BIG, None)

    assert L.csa2_window_attn(None, None, P, P, 1, 64, 1.0, OUT, P, BIG, None) == 1
    assert window(w=swa(rows=None)) == 1 and window(w=swa(D=64)) == 2 and window(w=swa(scale=0.0)) == 1
    assert window(T=130) == 1                       # W_cap 256 holds chunks of up to 129 tokens
    assert window(k=swa(B=1)) == 1 and window(k=swa(rows=17)) == 1
    assert window(q=None) == 1 and window(out=odd) == 1 and window(H=70) == 2
    assert L.csa2_prefix_attn_workspace_size(2, 1, 64, 384) == 0
    assert L.csa2_window_attn_workspace_size(2, 1, 64, 512, 2000, 0) == 0


def test_the_binding_checks_shapes():
    if torch.cuda.is_available():
        pytest.skip("host tensors are refused earlier where there is a GPU")
    p = C.PagePool(4, 16, 2, 3, 128, device="cpu")
    with pytest.raises(ValueError):
        C.PagePool.of(p.codes, p.scales[:3], p.refs, p.table, p.n_entries)
    with pytest.raises(ValueError):
        C.PagePool.of(p.codes, p.scales, p.refs.long(), p.table, p.n_entries)
    with pytest.raises(ValueError):
        C.SwaCache.of(torch.zeros(2, 8, dtype=torch.uint8))
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        C.csa2_pages_fork(p, one, torch.zeros(2, dtype=torch.int32))
    q = torch.zeros(1, 1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        C.csa2_prefix_attn_decode(p, one, 0, None, q[..., :64], one.view(1, 1), 1.0, q)
    with pytest.raises(ValueError):
        C.csa2_prefix_attn_decode(p, one, 0, None, q, one.view(1, 1), 1.0, q[:, :, :4])


def test_attention_refuses_an_output_over_its_queries_and_a_short_ring():
    L, last = C.lib(), 16 + 2 * 64 * 512 * 2                # the queries end in front of it

    def prefix(out, w=None, T=1):
        return L.csa2_prefix_attn_decode(pool(), P, 0, w, P, P, 2, T, 64, 1.0, ctypes.c_void_p(out), P, BIG, None)

    for at in (16, 32, last - 16):
        assert prefix(at) == 1 and b"overlaps" in L.csa2_last_error()
        assert L.csa2_window_attn(swa(), None, P, P, 1, 64, 1.0, ctypes.c_void_p(at), P, BIG, None) == 1
        assert b"overlaps" in L.csa2_last_error()
    assert prefix(1 << 40, swa(W_cap=128), T=2) == 1 and b"W_cap" in L.csa2_last_error()
