"""The paged FP4 cache (append, fork, compact) and the dense attentions that
read it or the window rows, each against a plain implementation: the pages
against a host model, exactly; the attentions against the definition in
binary64.

Tolerance of an attention output, per element, from the kernels' arithmetic
(keys and queries are exact in fp16, products exact in fp32):
  - the output's rounding to bf16: 2^-8 |out|;
  - each weight's rounding to fp16: 2^-11 of it, and 2^-25 for weights in
    fp16's subnormal range, in units of the row's largest weight (a reference
    maximum that lags the row's only makes the weights larger);
  - logits: fp32 accumulation of D products, at most D 2^-23 sum|q k| scale,
    and 2^-20 of |x| for the fold into base 2; weights move by twice that;
  - sums of n weights and products in fp32: n 2^-23 relative, 2^-20 for the
    exponential, the merge of partial results and the division.
Weight terms multiply sum p |v|, absolute ones n max|v| / sum of weights.
"""
import math

import numpy as np
import pytest
import torch

from fp4_kv_cache_append_b200 import csa2 as C

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    C.csa2_device_status(clear=True)
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def fp4_bytes(g, n, D):
    """Random codes, and scales between 2^-3 and 2^0 (bytes of E4M3)."""
    codes = torch.randint(0, 256, (n, D // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0x20, 0x38, (n, D // 16), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


def fp4_values(codes, scales):
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = grid[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    return v * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def e4m3_rows(g, *shape):
    return (torch.randn(*shape, generator=g, device="cuda")).to(torch.float8_e4m3fn).view(torch.uint8)


def attend64(q, keys, scale):
    """(out, tolerance) of rows q [H][D] over keys [n][D] in binary64."""
    H, D = q.shape
    if keys.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    x = q @ keys.T * scale
    w = torch.exp(x - x.amax(1, keepdim=True))
    tot = w.sum(1, keepdim=True)
    out = w @ keys / tot
    n = keys.shape[0]
    mag = (q.abs() @ keys.abs().T * abs(scale)).amax(1, keepdim=True)
    rel = 2.0 ** -11 + 2 * (D * 2.0 ** -23 * mag + 2.0 ** -20 * x.abs().amax(1, keepdim=True)) + n * 2.0 ** -23 \
        + 3 * 2.0 ** -20
    tol = 2.0 ** -8 * out.abs() + rel * (w @ keys.abs() / tot) + n * 2.0 ** -25 * keys.abs().amax() / tot
    return out, tol


def check(out, ref, tol, what=""):
    err = (out.double() - ref).abs()
    bad = ~(err <= tol + 1e-12)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / (tol + 1e-12)).max()):.2f}x"


# --------------------------------------------------------------------------- pages


class Model:
    """The pool on the host, entry bytes as lists."""

    def __init__(self, pool):
        for k in ("codes", "scales", "refs", "table", "n_entries"):
            setattr(self, k, getattr(pool, k).cpu().numpy().copy())
        self.page, self.M = pool.page, pool.max_pages
        self.no_page = self.bad = False

    def append(self, src_codes, src_scales, src_n, seq, at=None, first=None):
        refs0, nfree = self.refs.copy(), 0
        free = [p for p in range(len(refs0)) if refs0[p] == 0]
        seen = set()
        pages = lambda n: -(-n // self.page)  # noqa: E731
        for i, s in enumerate(seq):
            if s == -1:
                continue
            if not 0 <= s < len(self.n_entries) or s in seen:
                self.bad = True
                continue
            seen.add(s)
            old = int(self.n_entries[s])
            a = old if at is None else int(at[i])
            f = 0 if first is None else int(first[i])
            cnt = max(0, int(src_n[i]) - f)
            if f < 0 or a < 0 or a > old:
                self.bad = True
                continue
            if a + cnt > self.M * self.page:
                self.no_page = True
                continue
            row = self.table[s].copy()
            need = []
            for j in range(pages(a + cnt)):
                shared = j < pages(old) and refs0[row[j]] > 1
                if j >= pages(a):
                    if j >= pages(old) or shared:
                        need.append(j)
                elif j == pages(a) - 1 and a % self.page and cnt and shared:
                    need.append(j)
            if need and nfree + len(need) > len(free):
                self.no_page = True
                nfree += len(need)
                continue
            for j in need:
                p = free[nfree]
                nfree += 1
                if j < pages(old):
                    self.refs[row[j]] -= 1
                    if j < pages(a):
                        self.codes[p, : a % self.page] = self.codes[row[j], : a % self.page]
                        self.scales[p, : a % self.page] = self.scales[row[j], : a % self.page]
                row[j] = p
                self.refs[p] += 1
            for j in range(pages(a + cnt), pages(old)):
                self.refs[row[j]] -= 1
                row[j] = -1
            self.table[s] = row
            self.n_entries[s] = a + cnt
            for k in range(cnt):
                p, o = row[(a + k) // self.page], (a + k) % self.page
                self.codes[p, o], self.scales[p, o] = src_codes[i, f + k], src_scales[i, f + k]

    def fork(self, parent, child):
        t0, n0 = self.table.copy(), self.n_entries.copy()
        S, seen = len(n0), set()
        for p, c in zip(parent, child):
            if not -1 <= p < S or not 0 <= c < S or c in seen:
                self.bad = True
                continue
            seen.add(c)
            for x in t0[c]:
                if x >= 0:
                    self.refs[x] -= 1
            self.table[c] = t0[p] if p >= 0 else -1
            self.n_entries[c] = n0[p] if p >= 0 else 0
            for x in self.table[c]:
                if x >= 0:
                    self.refs[x] += 1

    def compact(self):
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        L = len(live)
        for f, t in zip([p for p in live if p >= L], [p for p in range(L) if self.refs[p] == 0]):
            self.codes[t], self.scales[t] = self.codes[f], self.scales[f]
            self.refs[t], self.refs[f] = self.refs[f], 0
            self.table[self.table == f] = t
        return L

    def same(self, pool, what=""):
        for k in ("table", "refs", "n_entries", "codes", "scales"):
            np.testing.assert_array_equal(getattr(pool, k).cpu().numpy(), getattr(self, k), err_msg=f"{what} {k}")


def staging(g, B, cap, D, n):
    src = C.MainCache(B, cap, D, 64, 1)
    c, s = fp4_bytes(g, B * cap, D)
    src.codes, src.scales = c.view(B, cap, -1), s.view(B, cap, -1)
    src.n_entries = i32(n)
    return src


def host(src):
    return src.codes.cpu().numpy(), src.scales.cpu().numpy(), src.n_entries.cpu().numpy()


@pytest.mark.parametrize("page,D,max_pages", [(16, 128, 70), (48, 256, 9), (128, 512, 5), (4096, 128, 1)])
def test_random_page_traffic_equals_the_host_model(page, D, max_pages):
    g, rng = gen(page + D), np.random.default_rng(page)
    S = 9
    pool = C.PagePool(max(12, 20 * max_pages // 5), page, S, max_pages, D)
    pool.codes.copy_(torch.randint(0, 256, pool.codes.shape, generator=g, device="cuda", dtype=torch.uint8))
    ref = Model(pool)
    ws = C.workspace(C.csa2_pages_workspace_size(pool, S))
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    room = page * max_pages
    for step in range(40):
        kind = rng.choice(["append", "append", "append", "fork", "compact"])
        if kind == "append":
            B = int(rng.integers(1, 7))
            cap = 128 * int(rng.integers(1, 1 + max(1, min(4, room // 128))))
            src = staging(g, B, cap, D, rng.integers(0, cap + 1, B).astype(np.int32))
            seq = rng.choice(S, B, replace=False).astype(np.int32)
            at = np.array([rng.integers(0, ref.n_entries[s] + 1) for s in seq], np.int32)
            if rng.random() < 0.3:
                at = None
            first = rng.integers(0, 60, B).astype(np.int32) if rng.random() < 0.5 else None
            C.csa2_pages_append(pool, src, i32(seq), at=None if at is None else i32(at),
                                first=None if first is None else i32(first), ws=ws)
            ref.append(*host(src), seq, at, first)
        elif kind == "fork":
            n = int(rng.integers(1, S + 1))
            child = rng.choice(S, n, replace=False).astype(np.int32)
            parent = rng.integers(-1, S, n).astype(np.int32)
            C.csa2_pages_fork(pool, i32(parent), i32(child), ws=ws)
            ref.fork(parent, child)
        else:
            C.csa2_pages_compact(pool, n_live, ws=ws)
            assert ref.compact() == int(n_live)
        ref.same(pool, f"step {step} {kind}")
    flags = C.csa2_device_status()
    assert bool(flags & C.DEV_NO_PAGE) == ref.no_page
    assert not flags & ~C.DEV_NO_PAGE


def test_append_writes_no_page_that_another_sequence_holds():
    g = gen(1)
    pool = C.PagePool(16, 16, 4, 4, 128)
    ref = Model(pool)
    src = staging(g, 1, 128, 128, [40])
    C.csa2_pages_append(pool, src, i32([0]))
    ref.append(*host(src), [0])
    C.csa2_pages_fork(pool, i32([0, 0]), i32([1, 2]))
    ref.fork([0, 0], [1, 2])
    # both children continue behind entry 37 of the shared third page, sequence 0 behind its end
    two = staging(g, 3, 128, 128, [3, 20, 1])
    C.csa2_pages_append(pool, two, i32([1, 2, 0]), at=i32([37, 37, 40]))
    ref.append(*host(two), [1, 2, 0], [37, 37, 40])
    ref.same(pool)
    # the same call again changes nothing but the pages that were shared
    C.csa2_pages_append(pool, two, i32([1, 2, 0]), at=i32([37, 37, 40]))
    ref.append(*host(two), [1, 2, 0], [37, 37, 40])
    ref.same(pool)
    assert C.csa2_device_status() == 0


def test_append_and_fork_skip_what_they_cannot_do_and_say_so():
    g = gen(2)
    pool = C.PagePool(6, 16, 4, 4, 128)
    ref = Model(pool)
    src = staging(g, 6, 128, 128, [30, 10, 10, 10, 70, 64])
    # a duplicate, an index out of range, none, table slots exceeded, then too few pages
    seq = [0, 0, 9, -1, 1, 2]
    C.csa2_pages_append(pool, src, i32(seq))
    ref.append(*host(src), seq)
    ref.same(pool)
    assert C.csa2_device_status() == C.DEV_NO_PAGE | C.DEV_BAD_SEQUENCE
    again = staging(g, 2, 128, 128, [50, 5])
    C.csa2_pages_append(pool, again, i32([3, 2]))       # takes the last four pages; none is left for the second
    ref.append(*host(again), [3, 2])
    ref.same(pool)
    assert C.csa2_device_status() == C.DEV_NO_PAGE
    C.csa2_pages_append(pool, again, i32([0, 2]), at=i32([31, -1]))   # behind the end; negative
    ref.append(*host(again), [0, 2], [31, -1])
    ref.same(pool)
    assert C.csa2_device_status() == C.DEV_BAD_SEQUENCE
    C.csa2_pages_fork(pool, i32([0, 3, 7, 0]), i32([1, 1, 2, -1]))
    ref.fork([0, 3, 7, 0], [1, 1, 2, -1])
    ref.same(pool)
    assert C.csa2_device_status() == C.DEV_BAD_SEQUENCE


def test_fork_takes_all_parents_as_they_stood():
    g = gen(3)
    pool = C.PagePool(32, 16, 5, 8, 256)
    ref = Model(pool)
    src = staging(g, 4, 128, 256, [16, 33, 100, 1])
    C.csa2_pages_append(pool, src, i32([0, 1, 2, 3]))
    ref.append(*host(src), [0, 1, 2, 3])
    for parent, child in (([1, 0], [0, 1]), ([1, 2, 3, 0], [0, 1, 2, 3]), ([2, 2, 2], [2, 0, 4]), ([-1, 0], [0, 3])):
        C.csa2_pages_fork(pool, i32(parent), i32(child))
        ref.fork(parent, child)
        ref.same(pool, f"{parent} -> {child}")


@pytest.mark.parametrize("n,S,M", [(1, 1, 1), (7, 9, 33), (255, 256, 3), (256, 300, 256), (257, 300, 5), (9, 12, 4096),
                                   (9, 12, 4097), (64, 80, 1025), (1000, 1100, 2)])
def test_fork_of_lists_of_any_length(n, S, M):
    """Either side of what one cluster takes: random tables, parents, children,
    a few of them out of range or listed twice."""
    rng = np.random.default_rng(n + M)
    pool = C.PagePool(500, 16, S, M, 128)
    lens = rng.integers(0, M + 1, S)
    table = np.where(np.arange(M)[None] < lens[:, None], rng.integers(0, 500, (S, M)), -1).astype(np.int32)
    pool.table, pool.n_entries = i32(table), i32(16 * lens)
    refs = np.zeros(500, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    pool.refs = i32(refs)
    ref = Model(pool)
    parent, child = rng.integers(-1, S, n), rng.permutation(S)[:n]
    if n > 5:
        child[n - 1], parent[2], child[4] = child[1], S, -1
    C.csa2_pages_fork(pool, i32(parent), i32(child))
    ref.fork(parent.tolist(), child.tolist())
    ref.same(pool)
    assert C.csa2_device_status() == (C.DEV_BAD_SEQUENCE if n > 5 else 0)


@pytest.mark.parametrize("n_pages,live", [(1, 0), (1, 1), (4, 4), (5, 2), (5000, 1700), (9001, 9000)])
def test_compact_closes_every_hole(n_pages, live):
    rng = np.random.default_rng(n_pages)
    pool = C.PagePool(n_pages, 16, 3, max(1, live), 128)
    at = rng.permutation(n_pages)[:live]
    table = np.full((3, max(1, live)), -1, np.int32)
    cut = live // 3
    table[0, :cut], table[1, : live - cut] = at[:cut], at[cut:]
    table[2, :cut] = at[:cut]
    refs = np.zeros(n_pages, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    pool.table.copy_(i32(table))
    pool.refs.copy_(i32(refs))
    pool.codes.copy_(torch.arange(n_pages, device="cuda").view(-1, 1, 1) % 251)
    ref = Model(pool)
    n_live = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    C.csa2_pages_compact(pool, n_live)
    assert ref.compact() == int(n_live) == live
    ref.same(pool)
    assert int((pool.refs[live:] != 0).sum()) == 0 and C.csa2_device_status() == 0


# --------------------------------------------------------------------------- prefix attention


def paged_batch(seed, D, page, n_shared, lens, n_seq_extra=1, m=1, poison=False):
    """A pool whose sequences agree on the first n_shared entries and own the
    rest, in shuffled pages; (pool, seq, entry values per batch row).  `poison`:
    every byte that no sequence's entry owns is 0xFF (a scale of NaN)."""
    g, rng = gen(seed), np.random.default_rng(seed)
    B, S = len(lens), len(lens) + n_seq_extra
    full = min(n_shared, min([max(n, 0) for n in lens if n >= n_shared] or [0])) // page
    M = max(1, max(-(-n // page) for n in lens), -(-n_shared // page)) + 1
    n_pages = full + B * M + 3
    order = rng.permutation(n_pages)
    pool = C.PagePool(n_pages, page, S, M, D, m=m)
    c, s = fp4_bytes(g, n_pages * page, D)
    pool.codes, pool.scales = c.view(n_pages, page, -1), s.view(n_pages, page, -1)
    seq = rng.permutation(S)[:B]
    table = np.full((S, M), -1, np.int32)
    values = []
    for b, n in enumerate(lens):
        need = -(-n // page)
        own = order[full + b * M: full + (b + 1) * M]
        row = np.concatenate([order[:full], own])[:need]
        table[seq[b], :need] = row
        if b and n > full * page and n_shared > full * page:      # the page the prefix ends in, copied
            k, e = table[seq[0], full], min(n, n_shared) - full * page
            if k >= 0 and e > 0 and full < need:
                for j in range(full, need):
                    hi = min(page, n_shared - j * page)
                    if hi > 0 and table[seq[0], j] >= 0:
                        pool.codes[int(row[j]), :hi] = pool.codes[int(table[seq[0], j]), :hi]
                        pool.scales[int(row[j]), :hi] = pool.scales[int(table[seq[0], j]), :hi]
    lens_t = np.zeros(S, np.int32)
    lens_t[seq] = lens
    pool.table, pool.n_entries = i32(table), i32(lens_t)
    refs = np.zeros(n_pages, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    pool.refs = i32(refs)
    for b, n in enumerate(lens):
        pg = torch.as_tensor(table[seq[b]][: -(-n // page)].astype(np.int64), device="cuda")
        values.append(fp4_values(pool.codes[pg].flatten(0, 1)[:n], pool.scales[pg].flatten(0, 1)[:n]) if n else
                      torch.zeros(0, D, dtype=torch.float64, device="cuda"))
    if poison:
        owned = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            for k in range(-(-n // page)):
                owned[int(table[seq[b], k]), : n - k * page] = True
        pool.codes[~owned] = 255
        pool.scales[~owned] = 255
    return pool, i32(seq), values


def window_keys(rows_b, scale, t, window):
    W_cap = rows_b.shape[0]
    tok = torch.arange(max(0, t - window + 1), t + 1, device="cuda")
    return rows_b.view(torch.float8_e4m3fn).double()[tok % W_cap] * scale


def poison_rows(rows, q_pos, window):
    """The ring's rows that no query sees: all NaN."""
    W_cap = rows.shape[1]
    for b, ts in enumerate(q_pos):
        seen = torch.zeros(W_cap, dtype=torch.bool, device="cuda")
        for t in ts:
            if t >= 0 and window:
                seen[torch.arange(max(0, t - window + 1), t + 1, device="cuda") % W_cap] = True
        rows[b, ~seen] = 255


def guarded(shape):
    """An output with marked rows before and behind it."""
    n = math.prod(shape)
    buf = torch.full((n + 2048,), 7.0, dtype=torch.bfloat16, device="cuda")
    return buf, buf[1024:1024 + n].view(shape)


def run_prefix(D, H, T, page, n_shared, lens, window, m=1, seed=0, s_swa=0.75, q_pos=None, scale=None, spread=1.0,
               poison=False):
    g = gen(seed + 77)
    pool, seq, values = paged_batch(seed, D, page, n_shared, lens, m=m, poison=poison)
    B = len(lens)
    q = (torch.randn(B, T, H, D, generator=g, device="cuda") * spread).to(torch.bfloat16)
    if q_pos is None:   # the last entry of a sequence was completed by its last query token
        q_pos = [[max(-1, m * n - T + j) for j in range(T)] for n in lens]
    W_cap = max(1, window + T + 3)
    rows = e4m3_rows(g, B, W_cap, D)
    if poison:
        poison_rows(rows, q_pos, window)
    swa = C.SwaCache.of(rows, scale=s_swa, window=window) if window else None
    buf, out = guarded((B, T, H, D))
    scale = scale or 1.0 / math.sqrt(D)
    C.csa2_prefix_attn_decode(pool, seq, n_shared, swa, q, i32(q_pos), scale, out)
    assert bool((buf[:1024] == 7).all()) and bool((buf[-1024:] == 7).all()), "wrote outside its output"
    for b in range(B):
        for j in range(T):
            t = q_pos[b][j]
            keys = [values[b][: max(0, min(lens[b], (t + 1) // m))]]
            if window and t >= 0:
                keys.append(window_keys(rows[b], s_swa, t, window))
            ref, tol = attend64(q[b, j].double(), torch.cat(keys), scale)
            check(out[b, j], ref, tol, f"b {b} query {j}")
    assert C.csa2_device_status() == 0
    return out


@pytest.mark.parametrize("D,H,T,page,n_shared,lens,window", [
    (128, 8, 1, 16, 300, [340, 301, 325], 128),
    (128, 1, 1, 16, 1, [1, 2], 0),
    (128, 64, 2, 32, 64, [64, 65, 128, 200], 100),
    (256, 20, 3, 48, 127, [130, 500, 127, 131, 222], 128),
    (256, 64, 1, 128, 0, [700, 1, 64, 63], 0),
    (256, 5, 1, 128, 257, [257], 1),
    (512, 64, 1, 128, 1000, [1100, 1001, 1000, 1128, 1400], 128),
    (512, 48, 2, 16, 65, [70, 66, 90], 200),
    (512, 3, 1, 4096, 4095, [4097, 4096], 0),
    (512, 64, 4, 64, 2048, [2052, 2100, 2048 + 513], 1024),
])
def test_prefix_attention(D, H, T, page, n_shared, lens, window):
    run_prefix(D, H, T, page, n_shared, lens, window, seed=D + H + page)


@pytest.mark.parametrize("B,H,D,n_shared,window", [(3000, 1, 128, 0, 0), (700, 2, 512, 40, 5), (513, 3, 256, 0, 33)])
def test_prefix_attention_of_many_short_sequences(B, H, D, n_shared, window):
    """More sequences than blocks many times over; lengths 0 to 90, sequences
    listed twice, workspace rows as few as a sequence has."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in (n_shared + rng.integers(0, 90, 40))]
    pool, seq, values = paged_batch(B, D, 16, n_shared, lens)
    pick = rng.integers(0, 40, B)
    pick[0] = 0
    many = seq[torch.as_tensor(pick, device="cuda")].contiguous()
    g = gen(B)
    q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
    rows = e4m3_rows(g, B, max(1, window), D)
    swa = C.SwaCache.of(rows, scale=0.5, window=window) if window else None
    pos = [[lens[p] + 7 if i % 11 else -1] for i, p in enumerate(pick)]
    buf, out = guarded((B, 1, H, D))
    nbytes = C.csa2_prefix_attn_workspace_size(B, 1, H, D)
    ws = torch.full((nbytes + 4096,), 77, dtype=torch.uint8, device="cuda")
    C.csa2_prefix_attn_decode(pool, many, n_shared, swa, q, i32(pos), 0.07, out, ws=ws[:nbytes])
    assert bool((ws[nbytes:] == 77).all()), "wrote behind its workspace"
    assert bool((buf[:1024] == 7).all()) and bool((buf[-1024:] == 7).all())
    for b in list(range(0, B, 37)) + [1, 2, B - 1]:
        t = pos[b][0]
        keys = [values[pick[b]][: max(0, min(lens[pick[b]], t + 1))]]
        if window and t >= 0:
            keys.append(window_keys(rows[b], 0.5, t, window))
        ref, tol = attend64(q[b, 0].double(), torch.cat(keys), 0.07)
        check(out[b, 0], ref, tol, f"b {b}")
    assert C.csa2_device_status() == 0


@pytest.mark.parametrize("D,H,T,page,n_shared,lens,window", [
    (128, 8, 1, 16, 300, [340, 301, 517], 128),
    (128, 3, 2, 48, 0, [1, 0, 49, 130], 0),
    (256, 20, 3, 32, 100, [101, 164, 333], 40),
    (256, 64, 1, 64, 130, [191, 200], 0),
    (512, 64, 1, 128, 129, [130, 700], 128),
    (512, 16, 2, 80, 77, [78, 240], 9),
])
def test_prefix_attention_among_bytes_of_nan(D, H, T, page, n_shared, lens, window):
    run_prefix(D, H, T, page, n_shared, lens, window, seed=D + H, poison=True)


def test_prefix_attention_gives_the_same_bits_in_every_launch():
    """Every one of a thousand launches is compared: a copy that overtakes the
    loads of the stage it overwrites shows in a few of a hundred (and by too
    little for the tolerances of the other tests)."""
    B, H, D, n_shared = 8, 64, 512, 4097
    g = gen(41)
    pool, seq, _ = paged_batch(5, D, 128, n_shared, [n_shared + 500 - 30 * b for b in range(B)])
    swa = C.SwaCache.of(e4m3_rows(g, B, 128, D), scale=1.0, window=128)
    q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
    pos = i32([[n_shared + 499 - 30 * b] for b in range(B)])
    ws = C.workspace(C.csa2_prefix_attn_workspace_size(B, 1, H, D))
    first = torch.empty_like(q)
    C.csa2_prefix_attn_decode(pool, seq, n_shared, swa, q, pos, 0.044, first, ws=ws)
    outs = torch.empty(50, *q.shape, dtype=q.dtype, device="cuda")
    for _ in range(20):
        for o in outs:
            C.csa2_prefix_attn_decode(pool, seq, n_shared, swa, q, pos, 0.044, o, ws=ws)
        assert not bool((outs != first).any())
    assert C.csa2_device_status() == 0


@pytest.mark.parametrize("form", ["prefix 512", "prefix 128", "window 256 of 333", "window 512 of 128"])
def test_attention_launched_back_to_back_gives_the_same_bits(form):
    """Thousands of launches that overlap at their ends: the stages that the
    teams of a block share are met in every order of arrival."""
    kind, D, *rest = form.split()
    D, B, H, g = int(D), 4, 16, gen(31)
    scale = 1.0 / math.sqrt(D)
    if kind == "prefix":
        pool, seq, _ = paged_batch(3, D, 64, 700, [1100, 900, 701, 1300])
        swa = C.SwaCache.of(e4m3_rows(g, B, 140, D), scale=1.0, window=128)
        q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
        pos, ws = i32([[2000]] * B), C.workspace(C.csa2_prefix_attn_workspace_size(B, 1, H, D))
        call = lambda out: C.csa2_prefix_attn_decode(pool, seq, 700, swa, q, pos, scale, out, ws=ws)   # noqa: E731
    else:
        T, W = 130, int(rest[1])
        swa = C.SwaCache.of(e4m3_rows(g, B, W + T + 30, D), scale=1.0, window=W)
        q = torch.randn(B, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
        pos = i32([[500 + j for j in range(T)]] * B)
        call = lambda out: C.csa2_window_attn(swa, None, q, pos, scale, out)   # noqa: E731
    first, again = torch.empty_like(q), torch.empty_like(q)
    call(first)
    for i in range(4000):
        call(again)
        if i % 500 == 499:
            assert torch.equal(first, again), i
    assert C.csa2_device_status() == 0


@pytest.mark.parametrize("scale", [-0.05, 1e-30])
def test_attention_by_a_negative_and_a_tiny_scale(scale):
    run_prefix(256, 20, 2, 32, 70, [90, 200], 40, seed=4, scale=scale)
    run_window(2, 5, 8, 512, 128, 4, 300, seed=5, scale=scale)
    run_window(1, 5, 8, 256, 400, 4, 300, seed=6, scale=scale)


def test_prefix_attention_long_and_many_rows():
    run_prefix(512, 64, 1, 128, 20000, [20000 + 7 * i for i in range(13)], 128, seed=5)
    run_prefix(128, 64, 1, 64, 5003, [5003 + i for i in range(40)], 32, seed=6)


def test_prefix_attention_of_two_token_entries():
    run_prefix(256, 16, 3, 32, 100, [140, 101, 133], 64, m=2, seed=9)


def test_prefix_attention_empty_sets_and_padded_queries():
    # no entries and no window, a padded query, a query before the prefix's end, a sequence shorter than the prefix
    run_prefix(128, 8, 1, 16, 0, [0, 5, 0], 0, seed=1, q_pos=[[0], [4], [-1]])
    run_prefix(256, 64, 2, 16, 200, [210, 50, 0, 205], 16, seed=2, q_pos=[[150, 209], [49, 300], [7, -1], [-1, -1]])


def test_prefix_attention_large_logits():
    # logits of several hundred: nearly one key a row, and reference maxima that move from tile to tile
    run_prefix(128, 16, 1, 16, 500, [600, 520], 64, seed=3, scale=0.5, spread=8.0)
    run_prefix(512, 64, 1, 128, 900, [1000, 920], 128, seed=4, scale=0.3, spread=4.0)


def test_prefix_attention_masks_bad_pages_and_sequences():
    D, H = 256, 8
    pool, seq, values = paged_batch(11, D, 16, 64, [100, 90])
    q = torch.randn(2, 1, H, D, generator=gen(3), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    s0, s1 = int(seq[0]), int(seq[1])
    pool.table[s1, 5] = pool.n_pages + 4    # entries 80 .. 89 of the second sequence
    C.csa2_prefix_attn_decode(pool, seq, 64, None, q, i32([[99], [89]]), 0.0625, out)
    for b, keys in enumerate((values[0], values[1][:80])):
        check(out[b, 0], *attend64(q[b, 0].double(), keys, 0.0625), f"b {b}")
    assert C.csa2_device_status() == C.DEV_INDEX_RANGE
    C.csa2_prefix_attn_decode(pool, i32([s0, 1000]), 64, None, q, i32([[99], [89]]), 0.0625, out)
    check(out[0, 0], *attend64(q[0, 0].double(), values[0], 0.0625))
    assert bool((out[1] == 0).all())
    assert C.csa2_device_status() & C.DEV_BAD_SEQUENCE


def test_prefix_attention_equals_the_sparse_attention_over_all_entries():
    """Both forms of the same set: entries 0 .. n-1 selected from a contiguous
    cache, and paged; each is within its own rounding of the other."""
    D, H, n, B, W = 512, 64, 512, 2, 128
    g = gen(8)
    main = staging(g, B, 512, D, [n, n])
    swa = C.SwaCache(B, W, D, window=W)
    swa.rows.copy_(e4m3_rows(g, B, W, D))
    q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
    pos = i32([[n - 1], [n - 1]])
    a, b = torch.empty_like(q), torch.empty_like(q)
    idx = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B, 1, 1)
    C.csa2_sparse_attn_decode(main, swa, q, pos, idx, 1 / math.sqrt(D), a)
    pool = C.PagePool(16, 64, B, 8, D)
    C.csa2_pages_append(pool, main, i32([1, 0]))
    C.csa2_prefix_attn_decode(pool, i32([1, 0]), 0, swa, q, pos, 1 / math.sqrt(D), b)
    err = (a.float() - b.float()).abs()
    assert float(err.max()) <= 2 ** -7 * float(a.float().abs().max()) + 1e-3
    assert float(err.sum() / a.float().abs().sum()) < 2e-3


# --------------------------------------------------------------------------- window attention


def run_window(B, T, H, D, window, n_sink, start, seed=0, s_swa=0.75, s_sink=1.5, q_pos=None, spread=1.0, scale=None,
               poison=False):
    g = gen(seed + 13)
    W_cap = max(1, window + T - 1 + seed % 5)
    rows = e4m3_rows(g, B, W_cap, D)
    sink_rows = e4m3_rows(g, B, max(1, n_sink) + seed % 3, D)
    swa = C.SwaCache.of(rows, scale=s_swa, window=window)
    sinks = C.SwaCache.of(sink_rows, scale=s_sink, window=n_sink) if n_sink else None
    q = (torch.randn(B, T, H, D, generator=g, device="cuda") * spread).to(torch.bfloat16)
    if q_pos is None:
        q_pos = [[start + 3 * b + j for j in range(T)] for b in range(B)]
    if poison:
        poison_rows(rows, q_pos, window)
        for b in range(B):
            first = max([max(0, t - window + 1) if window else t + 1 for t in q_pos[b] if t >= 0] or [0])
            sink_rows[b, min(n_sink, first):] = 255
    buf, out = guarded((B, T, H, D))
    scale = scale or 1.0 / math.sqrt(D)
    C.csa2_window_attn(swa, sinks, q, i32(q_pos), scale, out)
    assert bool((buf[:1024] == 7).all()) and bool((buf[-1024:] == 7).all()), "wrote outside its output"
    for b in range(B):
        for j in range(T):
            t = q_pos[b][j]
            lo = max(0, t - window + 1)
            keys = [window_keys(rows[b], s_swa, t, window)] if t >= 0 and window else []
            if n_sink and t >= 0:
                lo = lo if window else t + 1
                keys.append(sink_rows[b, : min(n_sink, lo)].view(torch.float8_e4m3fn).double() * s_sink)
            keys = torch.cat(keys) if keys else torch.zeros(0, D, dtype=torch.float64, device="cuda")
            ref, tol = attend64(q[b, j].double(), keys, scale)
            check(out[b, j], ref, tol, f"b {b} query {j}")
    assert C.csa2_device_status() == 0
    return out


@pytest.mark.parametrize("B,T,H,D,window,n_sink,start", [
    (2, 1, 8, 128, 128, 4, 1000),
    (1, 1, 1, 128, 1, 0, 0),
    (3, 5, 20, 256, 33, 7, 2),
    (2, 70, 64, 128, 128, 4, 0),
    (1, 131, 64, 512, 128, 4, 517),
    (2, 19, 48, 512, 128, 0, 0),
    (1, 40, 5, 256, 333, 16, 320),
    (2, 9, 64, 512, 1024, 64, 5000),
    (1, 200, 3, 512, 100, 1, 90),
    (4, 1, 64, 512, 128, 4, 5000),
    (1, 12, 64, 256, 7, 200, 150),
    (1, 3, 64, 512, 200, 0, 0),
])
def test_window_attention(B, T, H, D, window, n_sink, start):
    run_window(B, T, H, D, window, n_sink, start, seed=T + H)


@pytest.mark.parametrize("B,T,H,D,window,n_sink,start", [
    (2, 1, 8, 128, 128, 4, 1000),
    (2, 37, 64, 512, 128, 4, 0),
    (3, 5, 20, 256, 33, 7, 2),
    (1, 40, 5, 256, 333, 16, 320),
    (2, 9, 64, 512, 1024, 64, 5000),
    (2, 33, 4, 128, 700, 9, 650),
    (1, 3, 64, 512, 200, 0, 0),
])
def test_window_attention_among_rows_of_nan(B, T, H, D, window, n_sink, start):
    run_window(B, T, H, D, window, n_sink, start, seed=T + D, poison=True)


def test_window_attention_padded_and_unordered_queries():
    run_window(3, 4, 8, 128, 16, 3, 0, seed=1, q_pos=[[20, 21, -1, -1], [-1, -1, -1, -1], [40, 39, 38, 41]])
    run_window(1, 6, 64, 512, 128, 4, 0, seed=2, q_pos=[[300, -1, 299, 305, -1, 301]])


@pytest.mark.parametrize("H,D", [(64, 512), (8, 128), (20, 256)])
def test_window_attention_of_positions_far_apart(H, D):
    # tiles whose queries' windows lie far from one another, before one another, and in several sequences
    g = np.random.default_rng(H)
    T, W = 37, 100
    far = g.integers(0, 100000, T).tolist()
    near = (500 + g.permutation(T)).tolist()
    back = list(range(2000, 2000 - T, -1))
    mixed = [far[i] if i % 5 == 0 else (-1 if i % 7 == 0 else 300 + i) for i in range(T)]
    run_window(4, T, H, D, W, 4, 0, seed=3, q_pos=[far, near, back, mixed])


def test_window_attention_keeps_its_ring_over_a_long_chunk():
    # many more tokens than the ring of rows that a block keeps; unequal scales of sinks and window
    run_window(1, 700, 16, 128, 40, 5, 10, seed=6, s_swa=2.0 ** -9, s_sink=64.0)
    run_window(2, 300, 64, 256, 130, 12, 0, seed=7, s_swa=37.0, s_sink=0.01)


def test_window_attention_without_a_window_sees_its_sinks():
    run_window(2, 3, 8, 256, 0, 9, 4, seed=3)


def test_window_attention_of_more_queries_than_16_bits_count():
    # one visible key a query: the output is its row
    T, D = 70001, 128
    rows = e4m3_rows(gen(6), 1, T, D)
    q = torch.randn(1, T, 1, D, generator=gen(7), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    C.csa2_window_attn(C.SwaCache.of(rows, scale=0.5, window=1), None, q, i32(range(T)).view(1, T), 0.1, out)
    ref = (rows[0].view(torch.float8_e4m3fn).float() * 0.5).to(torch.bfloat16)
    assert torch.equal(out[0, :, 0], ref) and C.csa2_device_status() == 0


def test_window_attention_large_logits():
    run_window(1, 40, 64, 512, 128, 4, 400, seed=4, spread=6.0, scale=0.4)
    run_window(1, 40, 16, 128, 700, 4, 900, seed=5, spread=6.0, scale=0.7)


# --------------------------------------------------------------------------- together, streams, graphs


def test_prompt_forked_into_samples_that_decode():
    """A prompt is appended and quantised by csa2_append_quant, goes into
    pages, is forked into samples; every step appends an entry to each, and
    attends; one sample ends, the pool is compacted; outputs follow the
    definition all along, and compaction changes no bit."""
    D, H, n0, S = 512, 64, 300, 5
    g = gen(21)
    w_ik = (torch.randn(D, 64, generator=g, device="cuda") / math.sqrt(D)).to(torch.bfloat16)
    stage = C.MainCache(1, 384, D, 64, 1)
    kv = torch.randn(1, n0, D, generator=g, device="cuda").to(torch.bfloat16)
    C.csa2_append_quant(stage, kv, None, w_ik, None, None, i32([0]), n0)
    pool = C.PagePool(40, 64, S, 8, D)
    C.csa2_pages_append(pool, stage, i32([0]))
    C.csa2_pages_fork(pool, i32([0] * (S - 1)), i32(range(1, S)))
    tail = C.MainCache(S, 128, D, 64, 1)
    values = [[fp4_values(stage.codes[0, :n0], stage.scales[0, :n0])] for _ in range(S)]
    seq, scale = i32([3, 1, 0, 2, 4]), 1 / math.sqrt(D)
    for step in range(3):
        kv1 = torch.randn(S, 1, D, generator=g, device="cuda").to(torch.bfloat16)
        C.csa2_append_quant(tail, kv1, None, w_ik, None, None, i32([0] * S), 1)
        C.csa2_pages_append(pool, tail, seq)
        q = torch.randn(S, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
        out = torch.empty_like(q)
        pos = i32([[n0 + step]] * S)
        C.csa2_prefix_attn_decode(pool, seq, n0, None, q, pos, scale, out)
        for b in range(S):
            values[b].append(fp4_values(tail.codes[b, :1], tail.scales[b, :1]))
            check(out[b, 0], *attend64(q[b, 0].double(), torch.cat(values[b]), scale), f"step {step} b {b}")
    C.csa2_pages_fork(pool, i32([-1]), i32([1]))
    # (an ended sample has no keys, which moves the cuts of the work: the sums
    # of the others are joined in another order than before)
    C.csa2_prefix_attn_decode(pool, seq, n0, None, q, pos, scale, out)
    for b in range(S):
        if int(seq[b]) != 1:
            check(out[b, 0], *attend64(q[b, 0].double(), torch.cat(values[b]), scale), f"ended, b {b}")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    C.csa2_pages_compact(pool, live)
    assert int(live) == int((pool.refs > 0).sum())
    again = torch.empty_like(out)
    C.csa2_prefix_attn_decode(pool, seq, n0, None, q, pos, scale, again)
    keep = [b for b in range(S) if int(seq[b]) != 1]
    assert torch.equal(out[keep], again[keep])
    assert C.csa2_device_status() == 0


def test_calls_on_several_streams_at_once():
    """Persistent blocks of different launches, their tensor memory and shared
    memory side by side; each call with a workspace of its own."""
    g, D = gen(51), 256
    calls, outs = [], []
    for k, (n_shared, H) in enumerate(((900, 32), (0, 8))):
        pool, seq, _ = paged_batch(60 + k, D, 32, n_shared, [n_shared + 300, n_shared + 41, n_shared + 90])
        q = torch.randn(3, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
        pos, ws, out = i32([[2000]] * 3), C.workspace(C.csa2_prefix_attn_workspace_size(3, 1, H, D)), torch.empty_like(q)
        calls.append(lambda p=pool, s=seq, n=n_shared, q=q, t=pos, o=out, w=ws:
                     C.csa2_prefix_attn_decode(p, s, n, None, q, t, 0.06, o, ws=w))
        outs.append(out)
    for W, T in ((100, 40), (400, 40), (64, 1)):
        swa = C.SwaCache.of(e4m3_rows(g, 4, W + T, D), scale=0.5, window=W)
        q = torch.randn(4, T, 16, D, generator=g, device="cuda").to(torch.bfloat16)
        pos, out = i32([[700 + j for j in range(T)]] * 4), torch.empty_like(q)
        calls.append(lambda s=swa, q=q, t=pos, o=out: C.csa2_window_attn(s, None, q, t, 0.06, o))
        outs.append(out)
    for call in calls:
        call()
    ref = [o.clone() for o in outs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for o in outs:
            o.fill_(7)
        torch.cuda.synchronize()
        for _ in range(30):
            for stream, call in zip(streams, calls):
                with torch.cuda.stream(stream):
                    call()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, ref))
    assert C.csa2_device_status() == 0


def test_on_a_side_stream_and_in_a_replayed_graph():
    D, H, B = 256, 16, 3
    pool, seq, values = paged_batch(31, D, 32, 200, [230, 201, 260])
    g = gen(5)
    q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
    pos = i32([[229], [200], [259]])
    rows = e4m3_rows(g, B, 64, D)
    swa = C.SwaCache.of(rows, scale=1.0, window=64)
    outs = [torch.empty_like(q) for _ in range(2)]
    src = staging(g, B, 128, D, [2, 3, 1])
    at = i32([230, 201, 260])

    def step():
        C.csa2_pages_append(pool, src, seq, at=at, ws=ws_p)
        C.csa2_prefix_attn_decode(pool, seq, 200, swa, q, pos, 0.0625, outs[0], ws=ws_a)
        C.csa2_window_attn(swa, None, q, pos, 0.0625, outs[1], ws=ws_w)

    ws_p = C.workspace(C.csa2_pages_workspace_size(pool, B))
    ws_a = C.workspace(C.csa2_prefix_attn_workspace_size(B, 1, H, D))
    ws_w = C.workspace(C.csa2_window_attn_workspace_size(B, 1, H, D, 64, 0))
    step()
    first = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], first[0]) and torch.equal(outs[1], first[1])
    q.neg_()                       # the graph reads its inputs anew
    graph.replay()
    torch.cuda.synchronize()
    check(outs[0][0, 0], *attend64(q[0, 0].double(), torch.cat([values[0], window_keys(rows[0], 1.0, 229, 64)]), 0.0625))
    # a stream given by the caller, without a workspace
    C.csa2_prefix_attn_decode(pool, seq, 200, swa, q, pos, 0.0625, outs[1], stream=side)
    side.synchronize()
    assert torch.equal(outs[0], outs[1])
