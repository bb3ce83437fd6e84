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
