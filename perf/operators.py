"""Timed cases of the paged FP4 cache and of the dense attentions beside the sparse one.

Five operators: `prefix` is the decode attention of a batch over a paged FP4
cache whose sequences share a long prefix; `window` is the sliding-window
attention over FP8 rows with a few first tokens that stay visible; `append`,
`fork` and `compact` move a paged cache's pages.  Each has a plain form here
(elementary torch operations in 32 bits), the framework's call, and for the
attentions the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # two short chats of the tiny configuration (8 heads, D 128), pages of 16: latency of one small call
        dict(name="prefix_tiny", op="prefix", B=2, T=1, H=8, D=128, shared=300, own=40, page=16, window=128),
        # eight samples of one 4,097-token prompt at the decode configuration's widths
        dict(name="prefix_chat", op="prefix", B=8, T=1, H=64, D=512, shared=4097, own=500, page=128, window=128),
        # thirty-two samples of one 65,536-entry document: the decode configuration's context
        dict(name="prefix_long", op="prefix", B=32, T=1, H=64, D=512, shared=65536, own=1024, page=128, window=128),
        # single tokens of a decode batch in a window-only layer
        dict(name="window_decode", op="window", B=16, T=1, H=64, D=512, window=128, sinks=4, start=5000),
        # a ragged chunk: 20 heads, D 256, an odd window that spans several key tiles, three sequences
        dict(name="window_odd", op="window", B=3, T=517, H=20, D=256, window=333, sinks=7, start=100),
        # the prefill configuration's chunk of 8,192 tokens in a window-only layer
        dict(name="window_prefill", op="window", B=1, T=8192, H=64, D=512, window=128, sinks=4, start=131072),
        # one decode step's entry of each of 32 sequences goes into its page; some pages are still shared
        dict(name="append_step", op="append", B=32, D=512, page=128, at=1000, most=1, cap=128),
        # eight prompts of up to 8,192 entries go from the staging cache into pages
        dict(name="append_prompt", op="append", B=8, D=512, page=128, at=0, most=8192, cap=8192),
        # a beam step: 8 sequences continue two others
        dict(name="fork_beam", op="fork", n=8, parents=2, pages=40, page=16),
        # 64 samples start from four documents of 512 pages
        dict(name="fork_samples", op="fork", n=64, parents=4, pages=512, page=128),
        # a small pool closes its holes
        dict(name="compact_small", op="compact", n_pages=128, page=16, D=128, seqs=8),
        # a pool of 8,192 pages of 128 entries, half of them free
        dict(name="compact_large", op="compact", n_pages=8192, page=128, D=512, seqs=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "window", "window", "append", "fork", "compact"])
    D = rng.choice([128, 256, 512])
    page = 16 * _log(rng, 1, 16)
    if op == "prefix":
        B, H, T = _log(rng, 1, 32), _log(rng, 1, 64), rng.choice([1, 1, 2, 3])
        shared = _log(rng, 16, min(65536, 2.4e11 / (B * H * T * 4 * D)))
        return dict(op=op, B=B, T=T, H=H, D=D, shared=shared, own=rng.randint(T, 1024), page=page,
                    window=rng.choice([0, 1, 128, rng.randint(1, 256)]))
    if op == "window":
        window, sinks, H = _log(rng, 1, 1024), rng.randint(0, 16), _log(rng, 1, 64)
        keys = window + sinks
        most = min(8192 * 132 * 512 / (keys * D), 8192 * 64 * 132 * 512 / (H * keys * D))
        rows = _log(rng, 1, most)
        B = min(rows, _log(rng, 1, 32))
        return dict(op=op, B=B, T=max(1, rows // B), H=H, D=D, window=window, sinks=sinks,
                    start=rng.choice([0, rng.randint(0, 2000), rng.randint(0, 200000)]))
    if op == "append":
        B, most = _log(rng, 1, 64), _log(rng, 1, 8192)
        most = max(1, min(most, 65536 // B))
        return dict(op=op, B=B, D=D, page=page, at=rng.choice([0, rng.randint(1, 2000)]), most=most,
                    cap=(most + 127) // 128 * 128)
    if op == "fork":
        n = _log(rng, 1, 64)
        return dict(op=op, n=n, parents=rng.randint(1, max(1, n // 2)), pages=_log(rng, 1, 512), page=page)
    return dict(op=op, n_pages=min(_log(rng, 64, 8192), 8192 * 128 * 512 // (page * D)), page=page, D=D,
                seqs=_log(rng, 1, 64))


def work(case):
    c = case
    if c["op"] == "prefix":
        rows, entry = c["B"] * c["T"] * c["H"], c["D"] // 2 + c["D"] // 16
        own_n = c["B"] * c["own"] * 3 // 4       # own lengths are between a half and the whole
        keys = rows * (c["shared"] + c["own"] * 3 // 4 + c["window"])
        win = c["B"] * (c["window"] + c["T"] - 1) * c["D"] if c["window"] else 0
        return dict(bytes=(c["shared"] + own_n) * entry + win + rows * c["D"] * 4, flops=keys * c["D"] * 4)
    if c["op"] == "window":
        rows = c["B"] * c["T"] * c["H"]
        first, last = c["start"], c["start"] + c["T"] - 1
        sums = sum(min(t + 1, c["window"]) + min(c["sinks"], max(0, t + 1 - c["window"])) for t in range(first, last + 1))
        kept = min(last + 1, c["window"] + c["T"] - 1) + min(c["sinks"], last + 1)
        return dict(bytes=c["B"] * kept * c["D"] + rows * c["D"] * 4, flops=c["B"] * c["H"] * sums * c["D"] * 4)
    if c["op"] == "append":
        n = c["B"] if c["most"] == 1 else c["B"] * c["most"] * 3 // 4
        return dict(bytes=2 * n * (c["D"] // 2 + c["D"] // 16) + 16 * c["B"], flops=0)
    if c["op"] == "fork":
        return dict(bytes=c["n"] * c["pages"] * 4 * 4 + c["n"] * 16, flops=0)
    # a quarter of the pages moves; the reference counts are read, the tables read and written
    moved = c["n_pages"] // 4
    return dict(bytes=2 * moved * c["page"] * (c["D"] // 2 + c["D"] // 16) + c["n_pages"] * 4, flops=0)


# --------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _ri(g, lo, hi, shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV)


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _fp4(x):
    """E2M1 codes (two to a byte) and one E4M3 scale per 16 channels of x [n][D]."""
    n, D = x.shape
    s = _e4m3(x.view(n, D // 16, 16).abs().amax(-1) / 6)
    y = (x.view(n, D // 16, 16) / s.float().clamp(min=2.0 ** -9).unsqueeze(-1)).view(n, D)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(y.abs(), edges).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.view(torch.uint8)


def _fp4_random(g, n, D):
    """As _fp4 of normal rows, made in pieces."""
    codes = torch.empty(n, D // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(n, D // 16, dtype=torch.uint8, device=DEV)
    for i in range(0, n, 1 << 16):
        m = min(n, i + (1 << 16)) - i
        codes[i:i + m], scales[i:i + m] = _fp4(torch.randn(m, D, generator=g, device=DEV))
    return codes, scales


def _i32(x):
    return x.to(torch.int32).contiguous()


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "prefix":
        B, T, H, D, page, shared = (c[k] for k in ("B", "T", "H", "D", "page", "shared"))
        n_b = shared + _ri(g, max(T, c["own"] // 2), c["own"], (B,))
        full = shared // page                         # pages that the sequences really share
        M = (shared + c["own"] + page - 1) // page
        n_pages = full + B * (M - full) + 8
        order = torch.randperm(n_pages, generator=g, device=DEV)
        table = torch.full((B, M), -1, dtype=torch.int64, device=DEV)
        table[:, :full] = order[:full]
        table[:, full:] = order[full:full + B * (M - full)].view(B, M - full)
        codes, scales = _fp4_random(g, n_pages * page, D)
        codes, scales = codes.view(n_pages, page, -1), scales.view(n_pages, page, -1)
        if shared % page:                             # the page the prefix ends in was copied by each sequence
            codes[table[1:, full], : shared % page] = codes[table[0, full], : shared % page]
            scales[table[1:, full], : shared % page] = scales[table[0, full], : shared % page]
        used = torch.arange(M, device=DEV)[None] < ((n_b + page - 1) // page)[:, None]
        table = torch.where(used, table, torch.full_like(table, -1))
        refs = torch.zeros(n_pages, dtype=torch.int64, device=DEV)
        refs.scatter_add_(0, table[used], torch.ones_like(table[used]))
        s.update(codes=codes, scales=scales, refs=_i32(refs), table=_i32(table), n_entries=_i32(n_b), m=1)
        s["seq"] = _i32(torch.randperm(B, generator=g, device=DEV))
        # the last T entries are the tokens of this step
        s["q_pos"] = _i32(n_b[s["seq"].long()][:, None] - T + torch.arange(T, device=DEV)[None])
        W = c["window"]
        s["w_cap"] = max(1, W + T - 1)
        s["rows"] = _e4m3(torch.randn(B, s["w_cap"], D, generator=g, device=DEV)).view(torch.uint8) if W else None
        s["w_scale"] = 1.0
        s["q"] = torch.randn(B, T, H, D, generator=g, device=DEV).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty_like(s["q"])
    elif c["op"] == "window":
        B, T, H, D, W, n = (c[k] for k in ("B", "T", "H", "D", "window", "sinks"))
        s["w_cap"] = W + T - 1
        s["rows"] = _e4m3(torch.randn(B, s["w_cap"], D, generator=g, device=DEV) / 0.75).view(torch.uint8)
        s["sink_rows"] = _e4m3(torch.randn(B, n, D, generator=g, device=DEV) / 0.5).view(torch.uint8) if n else None
        s["w_scale"], s["s_scale"] = 0.75, 0.5
        s["q_pos"] = _i32((c["start"] + torch.arange(T, device=DEV))[None].repeat(B, 1))
        s["q"] = torch.randn(B, T, H, D, generator=g, device=DEV).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty_like(s["q"])
    elif c["op"] == "append":
        B, D, page, at, most = (c[k] for k in ("B", "D", "page", "at", "most"))
        s["src_codes"], s["src_scales"] = _fp4_random(g, B * c["cap"], D)
        s["src_codes"] = s["src_codes"].view(B, c["cap"], -1)
        s["src_scales"] = s["src_scales"].view(B, c["cap"], -1)
        s["src_n"] = _i32(_ri(g, (most + 1) // 2, most, (B,)))
        M = (at + most + page - 1) // page + 1
        full = (at + page - 1) // page                # pages that hold the entries so far
        n_pages = B * M + full + 16
        order = torch.randperm(n_pages, generator=g, device=DEV)
        table = torch.full((B + 1, M), -1, dtype=torch.int64, device=DEV)
        part = 1 if at % page else 0
        table[:, :full - part] = order[:full - part]  # every sequence was forked from the last one
        if part:                                      # half of the sequences have their own last page already
            table[:, full - 1] = order[full - 1]
            table[:B // 2, full - 1] = order[full:full + B // 2]
        refs = torch.zeros(n_pages, dtype=torch.int64, device=DEV)
        refs.scatter_add_(0, table[table >= 0], torch.ones_like(table[table >= 0]))
        s["codes"], s["scales"] = _fp4_random(g, n_pages * page, D)
        s["codes"], s["scales"] = s["codes"].view(n_pages, page, -1), s["scales"].view(n_pages, page, -1)
        s["refs"], s["table"], s["m"] = _i32(refs), _i32(table), 1
        s["n_entries"] = torch.full((B + 1,), at, dtype=torch.int32, device=DEV)
        s["seq"] = _i32(torch.randperm(B, generator=g, device=DEV))
        s["at"] = torch.full((B,), at, dtype=torch.int32, device=DEV)
    elif c["op"] == "fork":
        n, p, M = c["n"], c["parents"], c["pages"] + 1
        total = p * c["pages"] + 64
        order = torch.randperm(total, generator=g, device=DEV)
        table = torch.full((p + n, M), -1, dtype=torch.int64, device=DEV)
        table[:p, : c["pages"]] = order[: p * c["pages"]].view(p, -1)
        refs = torch.zeros(total, dtype=torch.int64, device=DEV)
        refs[table[:p, : c["pages"]]] = 1
        s["refs"], s["table"] = _i32(refs), _i32(table)
        lens = torch.zeros(p + n, dtype=torch.int64, device=DEV)
        lens[:p] = (c["pages"] - 1) * c["page"] + _ri(g, 1, c["page"], (p,))
        s["n_entries"], s["m"] = _i32(lens), 1
        s["codes"] = torch.zeros(total, c["page"], 64, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(total, c["page"], 8, dtype=torch.uint8, device=DEV)
        s["parent"] = _i32(_ri(g, 0, p - 1, (n,)))
        s["child"] = _i32(p + torch.randperm(n, generator=g, device=DEV))
    else:
        N, page, S = c["n_pages"], c["page"], c["seqs"]
        live = torch.randperm(N, generator=g, device=DEV)[: N // 2]
        M = (N // 2 + S - 1) // S
        table = torch.full((S * M,), -1, dtype=torch.int64, device=DEV)
        table[: N // 2] = live
        refs = torch.zeros(N, dtype=torch.int64, device=DEV)
        refs[live] = 1
        s["codes"], s["scales"] = _fp4_random(g, N * page, c["D"])
        s["codes"], s["scales"] = s["codes"].view(N, page, -1), s["scales"].view(N, page, -1)
        s["refs"], s["table"], s["m"] = _i32(refs), _i32(table.view(S, M)), 1
        s["n_entries"] = _i32((table.view(S, M) >= 0).sum(1) * page)
        s["refs0"], s["table0"] = s["refs"].clone(), s["table"].clone()
        s["n_live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# --------------------------------------------------------------------------- the framework's calls


def _handle(s):
    """The cache objects and workspaces that a serving program keeps."""
    h = s.get("handle")
    if h is None:
        from fp4_kv_cache_append_b200 import csa2 as C
        c = s["case"]
        h = s["handle"] = {"C": C}
        if "table" in s:
            h["pool"] = C.PagePool.of(s["codes"], s["scales"], s["refs"], s["table"], s["n_entries"], m=s["m"])
            h["ws"] = C.workspace(C.csa2_pages_workspace_size(h["pool"], c.get("B", c.get("n", 1))))
        if c["op"] == "prefix":
            B, T, H, D = s["q"].shape
            h["swa"] = C.SwaCache.of(s["rows"], scale=s["w_scale"], window=c["window"]) if c["window"] else None
            h["ws"] = C.workspace(C.csa2_prefix_attn_workspace_size(B, T, H, D))
        elif c["op"] == "window":
            B, T, H, D = s["q"].shape
            h["swa"] = C.SwaCache.of(s["rows"], scale=s["w_scale"], window=c["window"])
            h["sinks"] = C.SwaCache.of(s["sink_rows"], scale=s["s_scale"], window=c["sinks"]) if c["sinks"] else None
            h["ws"] = C.workspace(C.csa2_window_attn_workspace_size(B, T, H, D, c["window"], c["sinks"]))
        elif c["op"] == "append":
            B, cap, half = s["src_codes"].shape
            h["src"] = C.MainCache(B, cap, 2 * half, 64, 1)
            h["src"].codes, h["src"].scales, h["src"].n_entries = s["src_codes"], s["src_scales"], s["src_n"]
    return h


def _own(s):
    h, op = _handle(s), s["case"]["op"]
    C = h["C"]
    if op == "prefix":
        C.csa2_prefix_attn_decode(h["pool"], s["seq"], s["case"]["shared"], h["swa"], s["q"], s["q_pos"], s["scale"],
                                  s["out"], ws=h["ws"])
        return s["out"]
    if op == "window":
        C.csa2_window_attn(h["swa"], h["sinks"], s["q"], s["q_pos"], s["scale"], s["out"], ws=h["ws"])
        return s["out"]
    if op == "append":
        C.csa2_pages_append(h["pool"], h["src"], s["seq"], at=s["at"], ws=h["ws"])
        return [s["codes"], s["scales"], s["refs"], s["table"], s["n_entries"]]
    if op == "fork":
        C.csa2_pages_fork(h["pool"], s["parent"], s["child"], ws=h["ws"])
        return [s["refs"], s["table"], s["n_entries"]]
    s["refs"].copy_(s["refs0"])      # the holes are there again
    s["table"].copy_(s["table0"])
    C.csa2_pages_compact(h["pool"], s["n_live"], ws=h["ws"])
    return [s["codes"], s["scales"], s["refs"], s["table"], s["n_live"]]


# --------------------------------------------------------------------------- the plain forms


def _values(codes, scales):
    """FP4 entries [..][D/2], [..][D/16] as float32 [..][D]."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = lut[torch.stack([codes & 15, codes >> 4], -1).long()]
    v = v.view(*codes.shape[:-1], -1, 16) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return v.flatten(-2)


def _softmax(x):
    """Over the last dimension; rows with nothing visible are zeros."""
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def _plain_prefix(s):
    c = s["case"]
    B, T, H, D = s["q"].shape
    page, n_sh = c["page"], c["shared"]
    q = s["q"].float() * s["scale"]
    seq, t = s["seq"].long(), s["q_pos"].long()
    n_vis = torch.minimum(s["n_entries"].long()[seq][:, None], (t + 1) // s["m"])        # [B][T]
    flat_c, flat_s = s["codes"].flatten(0, 1), s["scales"].flatten(0, 1)
    table = s["table"].long()
    e = torch.arange(n_sh, device=q.device)
    at = table[seq[0], e // page] * page + e % page
    k_sh = _values(flat_c[at], flat_s[at])                                               # [shared][D]
    inf = torch.full((), -math.inf, device=q.device)
    hide = e[None, None, None] >= n_vis[:, :, None, None]
    x = [torch.where(hide, inf, (q.view(-1, D) @ k_sh.t()).view(B, T, H, -1))]
    e = torch.arange(n_sh, table.shape[1] * page, device=q.device)
    at = table[seq][:, e // page] * page + e % page                                      # [B][own]
    seen = at >= 0
    at = at.clamp(min=0)
    k_own = _values(flat_c[at], flat_s[at])                                              # [B][own][D]
    hide = (e[None, None] >= n_vis[:, :, None]) | ~seen[:, None]
    x.append(torch.where(hide[:, :, None], inf, torch.einsum("bthd,bkd->bthk", q, k_own)))
    if c["window"]:
        tok = t[:, :, None] - c["window"] + 1 + torch.arange(c["window"], device=q.device)
        k_w = s["rows"].view(torch.float8_e4m3fn).float() * s["w_scale"]
        k_w = k_w[torch.arange(B, device=q.device)[:, None, None], tok % s["w_cap"]]     # [B][T][W][D]
        x.append(torch.where((tok < 0)[:, :, None], inf, torch.einsum("bthd,btkd->bthk", q, k_w)))
    p = _softmax(torch.cat(x, -1))
    n1 = n_sh + k_own.shape[1]
    out = (p[..., :n_sh].reshape(-1, n_sh) @ k_sh).view(B, T, H, D)
    out = out + torch.einsum("bthk,bkd->bthd", p[..., n_sh:n1], k_own)
    if c["window"]:
        out = out + torch.einsum("bthk,btkd->bthd", p[..., n1:], k_w)
    return out.to(torch.bfloat16)


def _plain_window(s):
    c = s["case"]
    B, T, H, D = s["q"].shape
    W, n = c["window"], c["sinks"]
    q, t = s["q"].float() * s["scale"], s["q_pos"].long()
    b = torch.arange(B, device=q.device)[:, None, None]
    tok = t[:, :, None] - W + 1 + torch.arange(W, device=q.device)
    k = (s["rows"].view(torch.float8_e4m3fn).float() * s["w_scale"])[b, tok % s["w_cap"]]
    hide = tok < 0
    if n:
        first = torch.arange(n, device=q.device).expand(B, T, n)
        sink = s["sink_rows"].view(torch.float8_e4m3fn).float() * s["s_scale"]
        k = torch.cat([sink[:, None].expand(B, T, n, D), k], 2)
        hide = torch.cat([first >= (t[:, :, None] - W + 1).clamp(min=0), hide], 2)
    x = torch.einsum("bthd,btkd->bthk", q, k)
    p = _softmax(torch.where(hide[:, :, None], torch.full((), -math.inf, device=q.device), x))
    return torch.einsum("bthk,btkd->bthd", p, k).to(torch.bfloat16)


def _plain_append(s):
    page = s["case"]["page"]
    refs, M = s["refs"].long(), s["table"].shape[1]
    seq, at = s["seq"].long(), s["at"].long()
    cnt = s["src_n"].long()
    row, old = s["table"].long()[seq], s["n_entries"].long()[seq]
    pages = lambda x: (x + page - 1) // page  # noqa: E731
    keep, held, want = pages(at)[:, None], pages(old)[:, None], pages(at + cnt)[:, None]
    j = torch.arange(M, device=refs.device)[None]
    many = refs[row.clamp(min=0)] > 1
    copied = ((at % page != 0) & (cnt > 0))[:, None] & (j == keep - 1) & many
    fresh = copied | ((j >= keep) & (j < want) & ((j >= held) | many))
    need = fresh.sum(1)
    before = need.cumsum(0) - need
    free = torch.argsort((refs > 0).int(), stable=True)
    done = (before + need <= (refs == 0).sum())[:, None]
    fresh, copied = fresh & done, copied & done
    rank = (before[:, None] + fresh.cumsum(1) - 1).clamp(0, free.shape[0] - 1)
    new = torch.where(fresh, free[rank], row)
    new = torch.where(done & (j >= want), torch.full_like(new, -1), new)
    left = done & (row >= 0) & (j < held) & (fresh | (j >= want))
    refs.scatter_add_(0, row[left], -torch.ones_like(row[left]))
    refs.scatter_add_(0, new[fresh], torch.ones_like(new[fresh]))
    flat_c, flat_s = s["codes"].view(-1, s["codes"].shape[-1]), s["scales"].view(-1, s["scales"].shape[-1])
    # the entries before `at` of a page that was shared
    i = torch.arange(page, device=refs.device)
    some = copied[:, :, None] & (i < (at % page)[:, None, None])
    src, dst = (row[:, :, None] * page + i)[some], (new[:, :, None] * page + i)[some]
    flat_c[dst], flat_s[dst] = flat_c[src], flat_s[src]
    k = torch.arange(s["src_codes"].shape[1], device=refs.device)[None]
    put = (k < cnt[:, None]) & done
    e = (at[:, None] + k)
    dst = (torch.gather(new, 1, (e // page).clamp(max=M - 1)) * page + e % page)[put]
    flat_c[dst], flat_s[dst] = s["src_codes"][put], s["src_scales"][put]
    s["table"][seq] = new.int()
    s["refs"].copy_(refs)
    s["n_entries"][seq] = torch.where(done[:, 0], at + cnt, old).int()
    return [s["codes"], s["scales"], s["refs"], s["table"], s["n_entries"]]


def _plain_fork(s):
    parent, child = s["parent"].long(), s["child"].long()
    rows, lens, gone = s["table"][parent], s["n_entries"][parent], s["table"][child]
    for x, one in ((rows, 1), (gone, -1)):
        held = x[x >= 0].long()
        s["refs"].scatter_add_(0, held, torch.full_like(held, one, dtype=torch.int32))
    s["table"][child] = rows
    s["n_entries"][child] = lens
    return [s["refs"], s["table"], s["n_entries"]]


def _plain_compact(s):
    s["refs"].copy_(s["refs0"])
    s["table"].copy_(s["table0"])
    live = s["refs"] > 0
    n = live.sum()
    i = torch.arange(live.shape[0], device=live.device)
    src, dst = i[live & (i >= n)], i[~live & (i < n)]
    s["codes"][dst], s["scales"][dst] = s["codes"][src], s["scales"][src]
    to = i.clone()
    to[src] = dst
    s["refs"][dst] = s["refs"][src]
    s["refs"][src] = 0
    t = s["table"].long()
    s["table"].copy_(torch.where(t >= 0, to[t.clamp(min=0)], t))
    s["n_live"].copy_(n)
    return [s["codes"], s["scales"], s["refs"], s["table"], s["n_live"]]


def run(state):
    if own:
        return _own(state)
    return {"prefix": _plain_prefix, "window": _plain_window, "append": _plain_append, "fork": _plain_fork,
            "compact": _plain_compact}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- the definition in 64 bits


def _attend64(q, keys):
    """Rows q [n][D] over keys [k][D], all visible."""
    if keys.shape[0] == 0:
        return torch.zeros_like(q)
    x = q @ keys.T
    p = torch.exp(x - x.max(1, keepdim=True).values)
    return (p @ keys) / p.sum(1, keepdim=True)


def _decode64(codes, scales):
    low, high = (codes % 16).double(), torch.div(codes, 16, rounding_mode="floor").double()
    c = torch.stack([low, high], -1).flatten(-2)
    sign, c = torch.where(c >= 8, -1.0, 1.0), c % 8
    exp, man = torch.div(c, 2, rounding_mode="floor"), c % 2
    mag = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * 2.0 ** (exp - 1))
    return sign * mag * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def exact(case, seed):
    if case["op"] not in ("prefix", "window"):
        return None     # whole numbers only
    s = prepare(case, seed)
    c = case
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    B, T = s["q"].shape[:2]
    if c["op"] == "prefix":
        codes, scales = s["codes"], s["scales"]
        for b in range(B):
            i = int(s["seq"][b])
            n = int(s["n_entries"][i])
            pages = s["table"][i, : (n + c["page"] - 1) // c["page"]].long()
            keys = _decode64(codes[pages].flatten(0, 1)[:n], scales[pages].flatten(0, 1)[:n])
            for j in range(T):
                t = int(s["q_pos"][b, j])
                mine = [keys[: min(n, (t + 1) // s["m"])]]
                if c["window"]:
                    tok = torch.arange(max(0, t - c["window"] + 1), t + 1, device=DEV)
                    mine.append(s["rows"][b].view(torch.float8_e4m3fn).double()[tok % s["w_cap"]] * s["w_scale"])
                out[b, j] = _attend64(s["q"][b, j].double() * s["scale"], torch.cat(mine))
        return out
    # blocks of queries against all rows that any of them sees
    W, n = c["window"], c["sinks"]
    for b in range(B):
        ring = s["rows"][b].view(torch.float8_e4m3fn).double() * s["w_scale"]
        sink = s["sink_rows"][b].view(torch.float8_e4m3fn).double() * s["s_scale"] if n else ring[:0]
        for j in range(0, T, 512):
            t = torch.arange(c["start"] + j, c["start"] + min(T, j + 512), device=DEV)
            tok = torch.arange(max(0, int(t[0]) - W + 1), int(t[-1]) + 1, device=DEV)
            keys = torch.cat([sink, ring[tok % s["w_cap"]]])
            first = torch.arange(n, device=DEV)
            sees = torch.cat([first[None] <= t[:, None] - W, (tok[None] <= t[:, None]) & (tok[None] > t[:, None] - W)], 1)
            x = (s["q"][b, j:j + 512].double() * s["scale"]) @ keys.T          # [queries][H][keys]
            x = torch.where(sees[:, None], x, -math.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            out[b, j:j + 512] = (x @ keys) / x.sum(-1, keepdim=True)
    return out
