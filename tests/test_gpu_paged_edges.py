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


# --------------------------------------------------------------------------- weights far below the largest


def attend64_tail(q, keys, scale):
    """attend64, but for weights that fp16 flushes.  The dense kernels hold the
    row's largest weight at 2^9 or above, so half of fp16's smallest step, 2^-25,
    is 2^-34 of it: n keys lose n 2^-34 max|v| / (sum of weights) at most."""
    out, _ = attend64(q, keys, scale)
    D, n = q.shape[1], keys.shape[0]
    x = q @ keys.T * scale
    w = torch.exp(x - x.amax(1, keepdim=True))
    tot = w.sum(1, keepdim=True)
    mag = (q.abs() @ keys.abs().T * abs(scale)).amax(1, keepdim=True)
    rel = 2.0 ** -11 + 2 * (D * 2.0 ** -23 * mag + 2.0 ** -20 * x.abs().amax(1, keepdim=True)) + n * 2.0 ** -23 \
        + 3 * 2.0 ** -20
    return out, 2.0 ** -8 * out.abs() + rel * (w @ keys.abs() / tot) + n * 2.0 ** -34 * keys.abs().amax() / tot


def levels(H, D):
    """Queries [H][D] whose product with sixteen ones in front is 10 to 31 bits."""
    q = torch.zeros(H, D, dtype=torch.float64, device="cuda")
    q[:, :16] = (torch.linspace(10, 31, H, dtype=torch.float64, device="cuda") * math.log(2) / 16).unsqueeze(1)
    return q.to(torch.bfloat16)


@pytest.mark.parametrize("D,B,n,shared", [(128, 300, 4096, True), (256, 300, 3000, True), (512, 150, 4096, True),
                                          (512, 160, 1500, False), (128, 300, 1500, False)])
def test_prefix_attention_keeps_the_tail_under_one_dominant_key(D, B, n, shared):
    """Entry 0 alone has the query's channels, the others alone the rest, where
    the output is their total weight.  As many row tiles as SMs: no cut in the keys."""
    H, page, g = 64, 64, gen(D + n)
    n_pages = -(-n // page)
    pool = C.PagePool(n_pages, page, 1, n_pages, D)
    codes = torch.randint(0x11, 0x78, (n_pages * page, D // 2), generator=g, device="cuda", dtype=torch.uint8) & 0x77
    codes[:, :8] = 0
    codes[0] = 0
    codes[0, :8] = 0x22                                  # sixteen ones
    scales = torch.full((n_pages * page, D // 16), 0x38, dtype=torch.uint8, device="cuda")
    pool.codes, pool.scales = codes.view(n_pages, page, -1), scales.view(n_pages, page, -1)
    pool.table, pool.refs, pool.n_entries = i32(range(n_pages)).view(1, -1), i32([1] * n_pages), i32([n])
    q = levels(H, D).expand(B, 1, H, D).contiguous()
    out = torch.empty_like(q)
    C.csa2_prefix_attn_decode(pool, i32([0] * B), n if shared else 0, None, q, i32([[n - 1]] * B), 1.0, out)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    keys = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()][:n]
    ref, tol = attend64_tail(q[0, 0].double(), keys, 1.0)
    for b in range(B):
        check(out[b, 0], ref, tol, f"b {b}")
    assert C.csa2_device_status() == 0


@pytest.mark.parametrize("D,W", [(128, 1024), (256, 700), (512, 1024), (512, 128)])
def test_window_attention_keeps_the_tail_under_one_dominant_key(D, W):
    H, g = 64, gen(D)
    rows = torch.rand(2, W, D, generator=g, device="cuda") + 0.5
    rows[:, :, :16] = 0
    rows[:, 0] = 0
    rows[:, 0, :16] = 1                                  # the window's first token
    rows = rows.to(torch.float8_e4m3fn)
    q = levels(H, D).expand(2, 1, H, D).contiguous()
    out = torch.empty_like(q)
    C.csa2_window_attn(C.SwaCache.of(rows.view(torch.uint8), scale=1.0, window=W), None, q, i32([[W - 1]] * 2), 1.0, out)
    for b in range(2):
        check(out[b, 0], *attend64_tail(q[b, 0].double(), rows[b].double(), 1.0), f"b {b}")
    assert C.csa2_device_status() == 0


# --------------------------------------------------------------------------- queries of any size
# Each row of q is multiplied by a power of two that keeps its largest element at
# 2^-2 or above, so rounding it to fp16 (2^-25 at most below the normal range; bf16
# is exact above) moves an element by 2^-23 of the largest: a logit by 2^-23
# max|q| sum|k| scale, a D-th or so of attend64's D 2^-23 sum|q k| scale.


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -100, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("D,H", [(128, 8), (256, 20), (512, 64)])
def test_queries_far_from_one(D, H, size):
    """The normalisation may be folded into the softmax scale, with either sign."""
    scale = 1.0 / math.sqrt(D) / size
    run_prefix(D, H, 2, 16, 70, [90, 200], 40, seed=4, scale=scale, spread=size)
    run_prefix(D, H, 1, 16, 70, [90, 200], 0, seed=5, scale=-scale, spread=size)
    run_window(1, 9, H, D, 400, 4, 300, seed=6, scale=-scale, spread=size)        # rows that do not fit a ring
    run_window(2, 70, H, D, 100, 4, 300, seed=7, scale=scale, spread=size)        # a resident ring


@pytest.mark.parametrize("D", [128, 256, 512])
def test_heads_of_very_different_sizes(D):
    H, B, n = 64, 3, 500
    pool, seq, values = paged_batch(D, D, 32, 400, [n, n - 50, 430])
    g = gen(D + 1)
    size = torch.exp2(torch.linspace(-60, -17, H, device="cuda")).view(1, 1, H, 1)
    q = (torch.randn(B, 1, H, D, generator=g, device="cuda") * size).to(torch.bfloat16)
    q[0, 0, 5], q[1, 0, 6] = 0, 0
    q[0, 0, 7, 1:] = 0
    rows = e4m3_rows(g, B, 1024, D)
    out, scale = torch.empty_like(q), 2.0 ** 20 / math.sqrt(D)
    C.csa2_prefix_attn_decode(pool, seq, 400, None, q, i32([[n]] * B), scale, out)
    for b in range(B):
        check(out[b, 0], *attend64(q[b, 0].double(), values[b], scale), f"prefix, b {b}")
    C.csa2_window_attn(C.SwaCache.of(rows, scale=0.5, window=700), None, q, i32([[2000]] * B), scale, out)
    for b in range(B):
        check(out[b, 0], *attend64(q[b, 0].double(), window_keys(rows[b], 0.5, 2000, 700), scale), f"window, b {b}")
    assert C.csa2_device_status() == 0


# --------------------------------------------------------------------------- every launch, bit by bit
# The stages that a block's two teams share are met in every order of arrival; a
# step that is read too early or too late is off by less than other tests allow.


def _launches(call, like, n=1000, at_once=50):
    first = torch.empty_like(like)
    call(first)
    outs = torch.empty(at_once, *like.shape, dtype=like.dtype, device="cuda")
    for _ in range(n // at_once):
        for o in outs:
            call(o)
        assert not bool((outs != first).any())
    assert C.csa2_device_status() == 0
    return first


@pytest.mark.parametrize("B,T,H,D,window,n_sink", [
    (2, 5, 64, 512, 1024, 64),        # many tiles of FP8 rows, both channel halves
    (16, 1, 64, 512, 128, 4),         # single tokens: no resident ring
    (3, 60, 64, 512, 300, 70),        # 180 units: a second one to some blocks
    (4, 60, 16, 256, 500, 0),
    (2, 200, 16, 128, 900, 9),
])
def test_windows_of_many_tiles_give_the_same_bits_in_every_launch(B, T, H, D, window, n_sink):
    g = gen(T + window)
    swa = C.SwaCache.of(e4m3_rows(g, B, window + T - 1 + 40, D), scale=0.75, window=window)
    sinks = C.SwaCache.of(e4m3_rows(g, B, n_sink, D), scale=1.25, window=n_sink) if n_sink else None
    q = torch.randn(B, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    pos = i32([[3000 + 13 * b + j for j in range(T)] for b in range(B)])
    scale = 1.0 / math.sqrt(D)
    out = _launches(lambda o: C.csa2_window_attn(swa, sinks, q, pos, scale, o), q)
    for b, j in ((0, 0), (B - 1, T - 1), (B // 2, T // 2)):
        t = int(pos[b, j])
        keys = [window_keys(swa.rows[b], 0.75, t, window)]
        if n_sink:
            keys.append(sinks.rows[b].view(torch.float8_e4m3fn).double() * 1.25)
        check(out[b, j], *attend64(q[b, j].double(), torch.cat(keys), scale), f"b {b} query {j}")


@pytest.mark.parametrize("D,window", [(512, 1000), (256, 600), (128, 1000)])
def test_entries_and_a_window_of_many_tiles_give_the_same_bits_in_every_launch(D, window):
    """FP4 steps, then FP8 steps of the same stages, over and over."""
    B, H, n_shared = 6, 48, 257
    pool, seq, values = paged_batch(D, D, 64, n_shared, [n_shared + 70 * b + 1 for b in range(B)])
    g = gen(D + window)
    swa = C.SwaCache.of(e4m3_rows(g, B, window + 9, D), scale=0.5, window=window)
    q = torch.randn(B, 2, H, D, generator=g, device="cuda").to(torch.bfloat16)
    pos = i32([[2000 + b, 2001 + b] for b in range(B)])
    ws = C.workspace(C.csa2_prefix_attn_workspace_size(B, 2, H, D))
    out = _launches(lambda o: C.csa2_prefix_attn_decode(pool, seq, n_shared, swa, q, pos, 0.05, o, ws=ws), q)
    for b in range(B):
        keys = torch.cat([values[b], window_keys(swa.rows[b], 0.5, 2001 + b, window)])
        check(out[b, 1], *attend64(q[b, 1].double(), keys, 0.05), f"b {b}")


# --------------------------------------------------------------------------- blocks with several units


@pytest.mark.parametrize("B,T,H,D,window,n_sink,start", [
    (3, 140, 64, 512, 200, 4, 90),        # no ring: 420 units of a channel half on the SMs
    (5, 90, 64, 256, 300, 20, 0),         # 225 units
    (7, 101, 40, 128, 512, 3, 400),       # 224 units, odd rows
    (40, 3, 64, 512, 1024, 5, 2000),      # 160 units, no sequence twice in a block
])
def test_windows_without_a_ring_over_several_units(B, T, H, D, window, n_sink, start):
    run_window(B, T, H, D, window, n_sink, start, seed=B, poison=True)


@pytest.mark.parametrize("B,T,H,D,window,n_sink,start", [
    (1, 500, 64, 512, 128, 4, 1000),      # 250 tiles: a block walks along a sequence
    (5, 130, 64, 512, 100, 4, 50),        # 325 tiles: blocks cross from one sequence to the next
    (60, 9, 64, 512, 128, 0, 700),        # 300 tiles of 60 sequences
    (11, 77, 20, 256, 128, 9, 0),         # tiles across queries, ragged ends
    (33, 40, 16, 128, 130, 4, 60),
    (9, 300, 8, 128, 60, 5, 5),
])
def test_resident_rings_over_several_units_and_sequences(B, T, H, D, window, n_sink, start):
    run_window(B, T, H, D, window, n_sink, start, seed=T, poison=True)


@pytest.mark.parametrize("B,H,D,window,n_sink", [(148, 64, 512, 128, 4), (75, 64, 512, 128, 4), (512, 64, 512, 128, 4),
                                                 (300, 17, 512, 50, 0), (700, 16, 256, 16, 4), (400, 64, 128, 30, 2)])
def test_single_tokens_of_many_sequences(B, H, D, window, n_sink):
    """Large decode batches of a window-only layer, each sequence at its own place, some padded."""
    rng = np.random.default_rng(B)
    pos = [[-1 if b % 17 == 5 else int(rng.integers(0, 3 * window if b % 2 else 100000))] for b in range(B)]
    run_window(B, 1, H, D, window, n_sink, 0, seed=B, q_pos=pos, poison=True)


# --------------------------------------------------------------------------- chunks over pages


@pytest.mark.parametrize("D,H,T,page,n_shared,lens,window,m", [
    (512, 64, 40, 64, 130, [400, 333], 128, 1),
    (512, 16, 70, 32, 0, [71, 300], 0, 2),
    (256, 20, 65, 48, 100, [300, 165, 129], 90, 1),
    (128, 8, 100, 16, 64, [700, 164], 128, 2),
    (128, 64, 33, 128, 0, [33, 34, 500], 0, 1),
])
def test_prefix_attention_of_prompt_chunks(D, H, T, page, n_shared, lens, window, m):
    """Many queries of a sequence at once, each seeing the entries up to its own."""
    run_prefix(D, H, T, page, n_shared, lens, window, m=m, seed=T, poison=True)


# --------------------------------------------------------------------------- padded batches


@pytest.mark.parametrize("D,H,T,n_shared,window,first", [(128, 8, 1, 300, 128, "none"), (512, 64, 1, 300, 0, "none"),
                                                         (256, 20, 3, 129, 40, "other"), (512, 16, 2, 64, 9, "short"),
                                                         (128, 64, 2, 65, 0, "empty")])
def test_prefix_is_read_whatever_the_first_row_is(D, H, T, n_shared, window, first):
    """A batch whose first slot is padded (no sequence, or some other one), empty,
    or shorter than the prefix."""
    lens = [n_shared + 50, n_shared + 1, n_shared - 20, n_shared + 130]
    pool, seq, values = paged_batch(D + T, D, 32, n_shared, lens)
    g = gen(D)
    spare = next(s for s in range(pool.n_seq) if s not in seq.tolist())
    if first == "other":                                      # as long, of other entries
        pool.table[spare, :] = torch.arange(pool.max_pages, device="cuda").flip(0) % pool.n_pages
        pool.n_entries[spare] = n_shared + 5
    order = [2, 0, 1, 3] if first == "short" else [0, 1, 2, 3]
    rows_seq = [int(seq[i]) for i in order]
    keys = [values[i] for i in order]
    n_of = [lens[i] for i in order]
    if first != "short":
        rows_seq = [{"none": -1, "other": spare, "empty": spare}[first]] + rows_seq
        keys, n_of = [keys[0][:0]] + keys, [0] + n_of
    B = len(rows_seq)
    pos = [[n - T + j for j in range(T)] for n in n_of]
    if first in ("none", "other"):
        pos[0] = [-1] * T
    q = torch.randn(B, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    rows = e4m3_rows(g, B, window + T + 2, D) if window else None
    swa = C.SwaCache.of(rows, scale=0.5, window=window) if window else None
    buf, out = guarded((B, T, H, D))
    C.csa2_prefix_attn_decode(pool, i32(rows_seq), n_shared, swa, q, i32(pos), 0.06, out)
    for b in range(B):
        for j in range(T):
            t = pos[b][j]
            k = [keys[b][: max(0, t + 1)]]
            if window and t >= 0:
                k.append(window_keys(rows[b], 0.5, t, window))
            check(out[b, j], *attend64(q[b, j].double(), torch.cat(k), 0.06), f"b {b} query {j}")
    assert bool((buf[:1024] == 7).all()) and bool((buf[-1024:] == 7).all())
    assert C.csa2_device_status() == 0


def test_prefix_longer_than_every_sequence():
    D, H = 256, 8
    pool, seq, values = paged_batch(3, D, 16, 100, [100, 40])
    q = torch.randn(2, 1, H, D, generator=gen(3), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    for order in ([0, 1], [1, 0]):
        C.csa2_prefix_attn_decode(pool, seq[order].contiguous(), 112, None, q, i32([[500], [500]]), 0.06, out)
        for b, i in enumerate(order):
            check(out[b, 0], *attend64(q[b, 0].double(), values[i], 0.06), f"b {b}")
    assert C.csa2_device_status() == 0


@pytest.mark.parametrize("D,H,B,window", [(128, 64, 150, 40), (256, 33, 90, 0), (512, 64, 80, 128)])
def test_powers_of_two_of_the_queries_change_no_bit(D, H, B, window):
    """q x 2^20 and q x 2^-30 are both brought to [2^14, 2^15), and the softmax
    scale takes the powers back exactly; units and segments by the hundred."""
    lens = [200 + 3 * i for i in range(20)]
    pool, seq, _ = paged_batch(D, D, 32, 150, lens)
    many = seq[torch.arange(B, device="cuda") % 20].contiguous()
    g = gen(H)
    q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
    swa = C.SwaCache.of(e4m3_rows(g, B, max(1, window), D), scale=0.5, window=window) if window else None
    wide = C.SwaCache.of(e4m3_rows(g, B, 520, D), scale=0.5, window=500)
    pos = i32([[lens[b % 20] + 9] for b in range(B)])
    outs = []
    for power in (20, -30, 20):
        x = (q.float() * 2.0 ** power).to(torch.bfloat16)
        for _ in range(3):
            a, b = torch.full_like(q, 7), torch.full_like(q, 7)
            C.csa2_prefix_attn_decode(pool, many, 150, swa, x, pos, 0.0625 * 2.0 ** -power, a)
            C.csa2_window_attn(wide, None, x, pos, 0.0625 * 2.0 ** -power, b)
            outs.append((a, b))
    assert all(torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1]) for a, b in outs)
    assert C.csa2_device_status() == 0


# --------------------------------------------------------------------------- planes of more than 4 GB


def test_pages_behind_four_gigabytes():
    """Append, attention, fork and compact where a page's bytes lie beyond 32 bits."""
    D, page, n_pages, n = 512, 128, 140_000, 300
    pool = C.PagePool(n_pages, page, 3, 4, D)
    assert pool.codes.numel() > 2 ** 32
    pool.refs[: n_pages - 8] = 1                          # only the last eight pages are free
    g = gen(9)
    src = C.MainCache(1, 384, D, 64, 1)
    src.codes.copy_(torch.randint(0, 256, src.codes.shape, generator=g, device="cuda", dtype=torch.uint8))
    src.scales.copy_(torch.randint(0x20, 0x38, src.scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    src.n_entries.copy_(i32([n]))
    C.csa2_pages_append(pool, src, i32([0]))
    C.csa2_pages_fork(pool, i32([0]), i32([1]))
    C.csa2_pages_append(pool, src, i32([1]), at=i32([200]), first=i32([250]))       # copies the second page's start
    assert pool.table[0, :3].tolist() == [n_pages - 8, n_pages - 7, n_pages - 6]
    assert pool.table[1, :2].tolist() == [n_pages - 8, n_pages - 5]
    from test_gpu_paged import fp4_values
    v0 = fp4_values(src.codes[0, :n], src.scales[0, :n])
    v1 = torch.cat([v0[:200], v0[250:300]])
    q = torch.randn(2, 1, 64, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)

    def attend(what):
        out.fill_(7)
        C.csa2_prefix_attn_decode(pool, i32([0, 1]), 200, None, q, i32([[n], [n]]), 0.044, out)
        for b, v in enumerate((v0, v1)):
            check(out[b, 0], *attend64(q[b, 0].double(), v, 0.044), f"{what}, b {b}")

    attend("far")
    pool.refs[: n_pages - 8] = 0
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    C.csa2_pages_compact(pool, live)
    assert int(live) == 4 and int(pool.table.max()) == 3
    attend("near")
    assert C.csa2_device_status() == 0


@pytest.mark.parametrize("window", [128, 600])
def test_window_rows_behind_four_gigabytes(window):
    B, W_cap, D, H = 4, 2_200_000, 512, 16
    rows = torch.zeros(B, W_cap, D, dtype=torch.uint8, device="cuda")
    assert rows.numel() > 2 ** 32
    g = gen(3)
    pos = [[1500], [W_cap - 1], [W_cap + 5], [2 * W_cap + 2_100_000]]
    for b in range(B):
        at = torch.arange(pos[b][0] - window + 1, pos[b][0] + 1, device="cuda") % W_cap
        rows[b, at] = e4m3_rows(g, window, D)
    q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    C.csa2_window_attn(C.SwaCache.of(rows, scale=0.5, window=window), None, q, i32(pos), 0.05, out)
    for b in range(B):
        check(out[b, 0], *attend64(q[b, 0].double(), window_keys(rows[b], 0.5, pos[b][0], window), 0.05), f"b {b}")
    assert C.csa2_device_status() == 0


# --------------------------------------------------------------------------- logits of millions


@pytest.mark.parametrize("D,H,size", [(128, 8, 2e5), (256, 20, 1e6), (512, 64, 4e5), (128, 64, 3e6)])
def test_logits_of_millions_stay_finite(D, H, size):
    """A step of fp32 is then larger than the headroom of the weights in fp16: no
    weight may leave fp16's range for it.  (One key takes all: attend64's tolerance
    is wide, but finite.)"""
    pool, seq, values = paged_batch(D + H, D, 16, 300, [700, 310, 433])
    g = gen(H)
    q = torch.randn(3, 4, H, D, generator=g, device="cuda").to(torch.bfloat16)
    rows = e4m3_rows(g, 3, 1100, D)
    pos = [[698 + j for j in range(4)], [305 + j for j in range(4)], [500 + j for j in range(4)]]
    for scale in (size, -size):
        for window, k in ((600, None), (100, None), (100, pool)):
            swa = C.SwaCache.of(rows, scale=0.5, window=window)
            out = torch.empty_like(q)
            if k is None:
                C.csa2_window_attn(swa, None, q, i32(pos), scale, out)
            else:
                C.csa2_prefix_attn_decode(k, seq, 300, swa, q, i32(pos), scale, out)
            assert bool(torch.isfinite(out).all()), (scale, window)
            for b in range(3):
                for j in range(4):
                    t = pos[b][j]
                    keys = [window_keys(rows[b], 0.5, t, window)] + ([] if k is None else [values[b][: t + 1]])
                    keys = torch.cat(keys)
                    ref, tol = attend64(q[b, j].double(), keys, scale)
                    check(out[b, j], ref, tol, f"scale {scale} window {window} b {b} query {j}")
    assert C.csa2_device_status() == 0


# --------------------------------------------------------------------------- the largest lists, batches and positions


def test_lists_of_the_largest_length():
    n, page, D = 4096, 16, 128
    g, rng = gen(4), np.random.default_rng(4)
    pool = C.PagePool(9000, page, n + 5, 3, D)
    ref = Model(pool)
    src = C.MainCache(n, 128, D, 64, 1)
    src.codes.copy_(torch.randint(0, 256, src.codes.shape, generator=g, device="cuda", dtype=torch.uint8))
    src.scales.copy_(torch.randint(0, 256, src.scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    src.n_entries.copy_(i32(rng.integers(0, 40, n)))
    host = (src.codes.cpu().numpy(), src.scales.cpu().numpy(), src.n_entries.cpu().numpy())
    ws = C.workspace(C.csa2_pages_workspace_size(pool, n))
    for _ in range(2):
        seq = rng.permutation(n + 5)[:n].astype(np.int32)
        seq[[5, 4000]], seq[77] = seq[9], -1
        C.csa2_pages_append(pool, src, i32(seq), ws=ws)
        ref.append(*host, seq)
        ref.same(pool, "append")
        parent, child = rng.integers(-1, n + 5, n), rng.permutation(n + 5)[:n]
        child[[100, 4095]] = child[3]
        C.csa2_pages_fork(pool, i32(parent), i32(child), ws=ws)
        ref.fork(parent.tolist(), child.tolist())
        ref.same(pool, "fork")
    C.csa2_pages_compact(pool, ws=ws)
    ref.compact()
    ref.same(pool, "compact")
    assert C.csa2_device_status() == (C.DEV_BAD_SEQUENCE | C.DEV_NO_PAGE if ref.no_page else C.DEV_BAD_SEQUENCE)


@pytest.mark.parametrize("B,T,n_shared,window", [(65535, 1, 0, 0), (65535, 1, 50, 3), (1, 65535, 100, 0), (255, 257, 70, 2)])
def test_prefix_attention_of_the_most_queries(B, T, n_shared, window):
    D, H = 128, 1
    lens = [n_shared + 5 + 7 * i for i in range(12)]
    pool, seq, values = paged_batch(B % 97, D, 16, n_shared, lens)
    pick = torch.arange(B, device="cuda") * 5 % 12
    g = gen(B)
    q = torch.randn(B, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    rows = e4m3_rows(g, B, window + T - 1, D) if window else None
    swa = C.SwaCache.of(rows, scale=0.5, window=window) if window else None
    pos = (torch.arange(B, device="cuda")[:, None] % 40 + torch.arange(T, device="cuda")[None]).to(torch.int32)
    buf, out = guarded((B, T, H, D))
    C.csa2_prefix_attn_decode(pool, seq[pick].contiguous(), n_shared, swa, q, pos, 0.09, out)
    assert bool((buf[:1024] == 7).all()) and bool((buf[-1024:] == 7).all())
    rng = np.random.default_rng(B)
    for b, j in [(0, 0), (B - 1, T - 1)] + [(int(rng.integers(B)), int(rng.integers(T))) for _ in range(60)]:
        t, i = int(pos[b, j]), int(pick[b])
        keys = [values[i][: min(lens[i], t + 1)]]
        if window:
            keys.append(window_keys(rows[b], 0.5, t, window))
        check(out[b, j], *attend64(q[b, j].double(), torch.cat(keys), 0.09), f"b {b} query {j}")
    assert C.csa2_device_status() == 0


@pytest.mark.parametrize("B,T,H", [(1, 1 << 22, 1), (1 << 22, 1, 1), (2048, 2048, 1)])
def test_window_attention_of_the_most_queries(B, T, H):
    D, W = 128, 3
    g = gen(T)
    rows = torch.randint(0x20, 0x48, (B, W + T - 1, D), generator=g, device="cuda", dtype=torch.uint8)
    q = torch.randn(B, T, H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    pos = (torch.arange(B, device="cuda")[:, None] % 50 + torch.arange(T, device="cuda")[None]).to(torch.int32)
    out = torch.empty_like(q)
    C.csa2_window_attn(C.SwaCache.of(rows, scale=0.5, window=W), None, q, pos, 0.09, out)
    rng = np.random.default_rng(T)
    for b, j in [(0, 0), (B - 1, T - 1)] + [(int(rng.integers(B)), int(rng.integers(T))) for _ in range(60)]:
        check(out[b, j], *attend64(q[b, j].double(), window_keys(rows[b], 0.5, int(pos[b, j]), W), 0.09), f"b {b} query {j}")
    assert C.csa2_device_status() == 0


@pytest.mark.parametrize("D,H,window,n_sink", [(128, 8, 100, 3), (512, 64, 100, 0), (256, 20, 700, 5), (512, 16, 1024, 2)])
def test_the_largest_positions(D, H, window, n_sink):
    """2^31 - 4,097 is the last position that is taken; those above count as padded queries."""
    last, T = 2 ** 31 - 4097, 3
    g = gen(D)
    rows = e4m3_rows(g, 2, window + 17, D)
    sink_rows = e4m3_rows(g, 2, max(1, n_sink), D)
    swa = C.SwaCache.of(rows, scale=0.5, window=window)
    sinks = C.SwaCache.of(sink_rows, scale=0.5, window=n_sink) if n_sink else None
    pool, seq, values = paged_batch(D, D, 16, 40, [50, 90])
    q = torch.randn(2, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    for pos, flags in (([[last - 2, last - 1, last], [last - 9, last, last - 5]], 0),
                       ([[last, last + 1, 2 ** 31 - 1], [last + 1, last - 1, last + 4096]], C.DEV_BAD_POSITION)):
        for paged in (False, True):
            out = torch.full_like(q, 7)
            if paged:
                C.csa2_prefix_attn_decode(pool, seq, 40, swa, q, i32(pos), 0.06, out)
            else:
                C.csa2_window_attn(swa, sinks, q, i32(pos), 0.06, out)
            for b in range(2):
                for j in range(T):
                    t = pos[b][j]
                    if t > last:
                        assert bool((out[b, j] == 0).all())
                        continue
                    keys = [window_keys(rows[b], 0.5, t, window)]
                    if paged:
                        keys.append(values[b])
                    elif n_sink:
                        keys.append(sink_rows[b, :n_sink].view(torch.float8_e4m3fn).double() * 0.5)
                    check(out[b, j], *attend64(q[b, j].double(), torch.cat(keys), 0.06), f"paged {paged} b {b} query {j}")
            assert C.csa2_device_status() == flags


@pytest.mark.parametrize("D,H,window", [(128, 8, 100), (512, 64, 100), (256, 20, 700), (512, 16, 1024)])
def test_padded_queries_may_hold_anything(D, H, window):
    """NaN and infinities in the q of padded queries reach neither their own
    outputs (zeros) nor a bit of the others'."""
    g = gen(D + window)
    B, T = 3, 4
    pool, seq, _ = paged_batch(D, D, 16, 40, [50, 90, 61])
    swa = C.SwaCache.of(e4m3_rows(g, B, window + T, D), scale=0.5, window=window)
    q = torch.randn(B, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    pos = i32([[70, -1, 71, 72], [-1, -1, -1, -1], [1500, 1501, -1, -1]])
    dirty = q.clone()
    dirty[pos < 0] = torch.tensor([math.nan, math.inf, -math.inf, 3e38], dtype=torch.bfloat16, device="cuda").repeat(D // 4)
    outs = []
    for x in (q, dirty):
        a, b = torch.full_like(q, 7), torch.full_like(q, 7)
        C.csa2_prefix_attn_decode(pool, seq, 40, swa, x, pos, 0.06, a)
        C.csa2_window_attn(swa, None, x, pos, 0.06, b)
        assert bool((a[pos < 0] == 0).all()) and bool((b[pos < 0] == 0).all())
        outs.append((a, b))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert C.csa2_device_status() == 0
