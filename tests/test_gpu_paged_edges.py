"""Paged cache and dense attentions at the edges of what a call may hold: lists
with refused pairs, pools whose counts do not fit their tables, weights and
queries far below the largest, padded batches, and the paths on which a block
takes several units.  References and tolerances as in test_gpu_paged.py, from
which the helpers come; where a test needs another tolerance, it derives it."""
import math

import numpy as np
import pytest
import torch

from fp4_kv_cache_append_b200 import csa2 as C
from test_gpu_paged import (Model, _clean_status, attend64, check, e4m3_rows, gen, guarded, i32,  # noqa: F401
                            paged_batch, run_prefix, run_window, window_keys)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------- pages


@pytest.mark.parametrize("n,M", [(5, 3), (40, 3), (300, 3), (12, 5000)])
def test_fork_by_a_refused_parent_leaves_the_child_to_the_next_pair(n, M):
    """The first pair of a child names a parent out of range, a later one a good
    one, a third is the second good one: on either side of what one cluster takes."""
    rng = np.random.default_rng(n)
    S, pages = n + 3, 400
    pool = C.PagePool(pages, 16, S, M, 128)
    lens = rng.integers(0, min(M, 40) + 1, S)
    table = np.where(np.arange(M)[None] < lens[:, None], rng.integers(0, pages, (S, M)), -1).astype(np.int32)
    refs = np.zeros(pages, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    pool.table, pool.n_entries, pool.refs = i32(table), i32(16 * lens), i32(refs)
    ref = Model(pool)
    parent, child = rng.integers(-1, S, n), rng.permutation(S)[:n]
    parent[0], child[n // 2], parent[n // 2] = S, child[0], 1          # refused, then set
    child[n - 1], parent[n - 1] = child[0], 2                          # once only
    parent[1], child[n - 2] = -2, child[1]
    C.csa2_pages_fork(pool, i32(parent), i32(child))
    ref.fork(parent.tolist(), child.tolist())
    assert ref.n_entries[child[0]] == 16 * lens[1]
    ref.same(pool)
    assert C.csa2_device_status() == C.DEV_BAD_SEQUENCE


@pytest.mark.parametrize("n_pages,bad", [(20, [0]), (20, [1, 3, 5]), (6000, [7, 4000, 4500])])
def test_compact_moves_nothing_without_a_free_page(n_pages, bad):
    """Negative counts (a pool that was never well formed) leave fewer holes
    below the boundary than pages above it; what has no place stays."""
    pool = C.PagePool(n_pages, 16, 2, n_pages, 128)
    pool.codes.copy_((torch.arange(n_pages, device="cuda") % 251).view(-1, 1, 1).expand_as(pool.codes))
    refs = np.zeros(n_pages, np.int32)
    refs[[2, 4]], refs[n_pages // 2:], refs[bad] = 1, 1, -1
    live = np.flatnonzero(refs > 0)
    table = np.full((2, n_pages), -1, np.int32)
    table[0, : live.size] = live
    pool.refs, pool.table = i32(refs), i32(table)
    pool.n_entries = i32([16 * live.size, 0])
    L = live.size
    src, dst = live[live >= L], np.array([p for p in range(L) if refs[p] == 0])
    k = min(src.size, dst.size)
    assert dst.size < src.size
    to = np.arange(n_pages)
    to[src[:k]] = dst[:k]
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    C.csa2_pages_compact(pool, n_live)
    assert int(n_live) == L and C.csa2_device_status() == C.DEV_INDEX_RANGE
    assert np.array_equal(pool.table.cpu().numpy()[0, : live.size], to[live])
    want = refs.copy()
    want[dst[:k]], want[src[:k]] = refs[src[:k]], 0
    assert np.array_equal(pool.refs.cpu().numpy(), want)
    got = pool.codes[torch.as_tensor(to[live], device="cuda")][:, 0, 0].cpu().numpy()
    assert np.array_equal(got, live % 251)
