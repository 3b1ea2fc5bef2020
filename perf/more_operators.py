"""Serving attention over a cache held in 4 bits, and attention of many new tokens at once, with a
sliding window and a few first tokens that stay visible.

Every case is a pass through one operator on inputs of its own.  With ``own`` false the
operators are computed by elementary torch operations in 32 bits (64 for the angles of far
positions); with ``own`` true by the package's kernels.

Kinds of cases:
  append   new tokens' queries and keys normed per head and rotated, keys and values quantised
           into the paged cache on the way (MXFP4: E2M1 codes with a power of two for each 32
           of a row); what the cache then holds for them is read back
  decode   one new query token per sequence over its cached tokens
  prefill  several new query tokens per sequence, each over the cached tokens up to its own
           (a prompt, a chunk behind a context, a few drafted tokens to be checked)

With a window W and S sinks a query at position p sees the tokens t <= p with t > p - W or t < S.
"""
import math

import torch

own = False

DEV = "cuda"
FP8_MAX = 448.0  # the largest E4M3 value
MIN_SCALE = 2.0 ** -100  # the smallest scale (rows of zeros and next to it)
EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # the decode step of a small batch: latency
        dict(name="append_step", kind="append", T=24, Hq=64, Hkv=8, D=128, R=128, inter=False, page=16, far=32768),
        # a prefill chunk, half of the dims rotated, interleaved pairs
        dict(name="append_chunk", kind="append", T=8192, Hq=64, Hkv=8, D=128, R=64, inter=True, page=64, far=131072),
        # one sequence with a short prompt behind it: launch and memory latency
        dict(name="decode_short", kind="decode", fmt="mxfp4", B=1, L=347, Hq=32, Hkv=8, D=128, page=16, window=0,
             sinks=0),
        # a serving batch, ragged lengths up to 8192
        dict(name="decode_batch", kind="decode", fmt="mxfp4", B=64, L=8192, Hq=64, Hkv=8, D=128, page=64, window=0,
             sinks=0),
        # two long documents: few rows, the work split over the length
        dict(name="decode_long", kind="decode", fmt="mxfp4", B=2, L=262143, Hq=64, Hkv=8, D=128, page=32, window=0,
             sinks=0),
        # many chats on a sliding-window layer with sinks, empty places of the batch among them,
        # twelve query heads on each key head, an odd page size
        dict(name="decode_window_odd", kind="decode", fmt="mxfp4", B=201, L=2900, Hq=36, Hkv=3, D=192, page=24,
             window=1000, sinks=4),
        # long chats on a windowed layer with sinks, 16-bit cache
        dict(name="decode_sinks_bf16", kind="decode", fmt="bf16", B=48, L=30000, Hq=64, Hkv=8, D=64, page=64,
             window=4096, sinks=16),
        # one prompt, causal, 16-bit cache
        dict(name="prefill_prompt", kind="prefill", fmt="bf16", B=1, n=8192, ctx=0, Hq=64, Hkv=8, D=128, page=64,
             window=0, sinks=0),
        # a ragged batch of prompts on a windowed layer with sinks, 8-bit cache
        dict(name="prefill_window", kind="prefill", fmt="e4m3", B=6, n=3000, ctx=1500, Hq=48, Hkv=8, D=128, page=32,
             window=1000, sinks=4),
        # a chunk of a long document behind what is cached of it, 4-bit cache
        dict(name="prefill_chunk", kind="prefill", fmt="mxfp4", B=1, n=1500, ctx=30001, Hq=64, Hkv=8, D=128, page=64,
             window=0, sinks=0),
        # a few drafted tokens of each sequence of a batch, checked in one pass; 8-bit cache
        dict(name="prefill_drafts", kind="prefill", fmt="e4m3", B=32, n=4, ctx=8000, Hq=64, Hkv=8, D=128, page=64,
             window=0, sinks=0),
        # a few short prompts of a small model: latency, odd sizes
        dict(name="prefill_short_odd", kind="prefill", fmt="mxfp4", B=3, n=37, ctx=90, Hq=15, Hkv=3, D=96, page=7,
             window=50, sinks=2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "append", "prefill", "prefill", "prefill"])
    page = rng.choice([7, 16, 16, 24, 32, 64, 64, 100, 128])
    if kind == "append":
        D = rng.choice([64, 96, 128, 128, 192, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        T = _log_int(rng, 1, int(8.3e6 / (Hkv * D)))
        return dict(kind=kind, T=T, Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2, 32]),
                    inter=rng.random() < 0.4, page=page, far=rng.choice([4096, 131072, 1 << 20]))
    fmt = rng.choice(["mxfp4", "mxfp4", "e4m3", "bf16"] if kind == "prefill" else ["mxfp4", "mxfp4", "mxfp4", "bf16", "e4m3"])
    D = rng.choice([64, 96, 128, 128, 128, 192, 256] if fmt == "mxfp4" else [64, 80, 128, 128, 128, 192, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16])
    window = rng.choice([0, 0, 0, 128, 1000, 4096])
    sinks = rng.choice([0, 1, 4, 16, 130]) if window else 0
    if kind == "decode":
        if fmt != "mxfp4" and not window:  # (the other formats' full attention is measured elsewhere)
            window, sinks = rng.choice([128, 1000, 4096]), rng.choice([1, 4, 16, 130])
        B = _log_int(rng, 1, 256)
        # at most as many cached values and products as the largest listed case has
        most = min(5e8 / (Hkv * D), 1.6e10 / (4 * Hkv * G * D))
        L = _log_int(rng, 1, max(2, min(262143, int(most / B))))
        return dict(kind=kind, fmt=fmt, B=B, L=L, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, window=window, sinks=sinks)
    B = _log_int(rng, 1, 64)
    n = _log_int(rng, 1, 8192)
    while B * Hkv * G * n * n > 2e9:  # at most half of the pairs of the largest listed case
        B, n = max(1, B // 2), max(1, int(n / 1.3))
    ctx = rng.choice([0, _log_int(rng, 1, max(2, int(min(1e5, 2e9 / (B * Hkv * G * n), 2e8 / (B * Hkv * D)))))])
    return dict(kind=kind, fmt=fmt, B=B, n=n, ctx=ctx, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, window=window, sinks=sinks)


def _spread(B, most, step):
    """B numbers spread evenly over 1..most in a scattered order, the largest first."""
    return [max(1, min(most, math.ceil(most * (1.0 - math.fmod(b * step, 1.0))))) for b in range(B)]


def _sizes(case):
    """The sequences' (new tokens, cached tokens with the new ones).  In a batch of 8 and more every
    16th place is empty."""
    B = case["B"]
    empty = [B >= 8 and b % 16 == 7 for b in range(B)]
    if case["kind"] == "decode":
        return [(1, 0 if e else n) for e, n in zip(empty, _spread(B, case["L"], 0.6180339887498949))]
    new = _spread(B, case["n"], 0.6180339887498949)
    old = _spread(B, case["ctx"], 0.7548776662466927) if case["ctx"] else [0] * B
    return [(0, 0) if e else (n, n + c) for e, n, c in zip(empty, new, old)]


def _pairs(case):
    """(Pairs of query and visible key, keys that any query sees), of all sequences, for one head."""
    W, S = case["window"], case["sinks"]
    pairs = keys = 0
    for new, length in _sizes(case):
        if not new or not length:
            continue
        first = length - new  # position of the first new token
        if not W:
            pairs += new * (first + length + 1) // 2
            keys += length
            continue
        start = max(0, first - W + 1)
        keys += length - start + min(S, start)
        for p in range(first, length):
            f = max(0, p - W + 1)
            pairs += p + 1 - f + min(S, f)
    return pairs, keys


def _row(fmt, D):
    """Bytes of one head's cached key or value."""
    return {"bf16": 2 * D, "e4m3": D + 4, "mxfp4": D // 2 + D // 32}[fmt]


def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["kind"] == "append":
        T, row = case["T"], _row("mxfp4", D)
        # in: q, k, v, positions, slots; out: q and the cache's rows, which are read again for the
        # values that come back
        moved = T * (Hq * 4 * D + Hkv * (2 * 2 * D + 4 * row + 2 * 2 * D) + 12)
        return {"bytes": moved + 8 * D + 4 * case["R"], "flops": 10 * T * (Hq + Hkv) * D}
    pairs, keys = _pairs(case)
    T = sum(n for n, _ in _sizes(case))
    moved = 2 * keys * Hkv * _row(case["fmt"], D) + T * Hq * (4 * D + 4) + 8 * case["B"] + 4 * (keys // case["page"])
    return {"bytes": moved, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------ the 4-bit rows
def _power(e):
    """2^e in f32, for whole e in -126..127."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _mxfp4(rows):
    """f32 rows [..., D] -> (codes [..., D / 2] uint8, two to a byte, the even element low; scales
    [..., D / 32] uint8, E8M0).  A scale is the smallest power of two (at least 2^-100) of which
    the group's largest is at most 7 times (what is above 6 becomes 6: no further off than the
    steps below are); codes are rounded to the nearest, ties to the even code."""
    groups = rows.unflatten(-1, (-1, 32))
    amax = groups.abs().amax(-1)
    mantissa, exponent = torch.frexp(amax)  # amax = mantissa 2^exponent, mantissa in [1/2, 1)
    e = (exponent - 3 + (mantissa > 0.875)).clamp_min(-100).masked_fill(amax == 0, -100)
    z = groups * _power(-e.unsqueeze(-1))
    a = z.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * (z < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _from_mxfp4(codes, scales):
    """The f32 values of rows: codes [..., D / 2], scales [..., D / 32]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    m = (c & 7).float()
    value = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))
    value = torch.where(c >= 8, -value, value)
    return value * _power(scales.to(torch.int32) - 127).repeat_interleave(32, -1)


def _scale_width(D):
    """Bytes of a row's scales in the cache: whole words of four."""
    return 4 * -(-D // 128)


# ------------------------------------------------------------------------------ the inputs
def _fill_cache(g, pages, Hkv, page, D, fmt, spread):
    """Random pool of one of K, V: rows ~N(0, 1) times a size of their own."""
    rows = torch.randn(pages, Hkv, page, D, generator=g, device=DEV, dtype=torch.float32)
    if spread:
        rows *= torch.exp(spread * torch.randn(pages, Hkv, page, 1, generator=g, device=DEV))
    if fmt == "bf16":
        return rows.to(torch.bfloat16), None
    if fmt == "mxfp4":
        codes, scales = _mxfp4(rows)
        return codes, torch.nn.functional.pad(scales, (0, _scale_width(D) - scales.shape[-1]))
    scale = (rows.abs().amax(-1) / FP8_MAX).clamp_min(MIN_SCALE)
    rows = (rows * (1.0 / scale).unsqueeze(-1)).clamp_(-FP8_MAX, FP8_MAX)
    return rows.to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    kind, D, Hq, Hkv, page = case["kind"], case["D"], case["Hq"], case["Hkv"], case["page"]
    s = dict(case)
    s.setdefault("fmt", "mxfp4")
    randn = lambda *shape: torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)  # noqa: E731
    if kind == "append":
        T = case["T"]
        pages = -(-T // page) + 3
    else:
        sizes = _sizes(case)
        T, used = sum(n for n, _ in sizes), [-(-n // page) for _, n in sizes]
        pages = sum(used) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s["k"], s["k_scale"] = _fill_cache(g, pages, Hkv, page, D, s["fmt"], 0.0)
    s["v"], s["v_scale"] = _fill_cache(g, pages, Hkv, page, D, s["fmt"], 0.5)
    if kind == "append":
        # q, k and v are slices of one projection's output
        qkv = (randn(T, Hq + 2 * Hkv, D) * torch.exp(0.5 * randn(T, 1, 1))).to(torch.bfloat16)
        s["q"], s["kin"], s["vin"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        # consecutive tokens of scattered pages
        t = torch.arange(T, device=DEV)
        s["slots"] = ids[t // page] * page + (t % page).to(torch.int32)
        s["pos"] = torch.randint(0, case["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
        s["inv_freq"] = THETA ** (-torch.arange(0, case["R"], 2, device=DEV, dtype=torch.float64) / case["R"])
        s["qw"], s["kw"] = 1.0 + 0.1 * randn(D), 1.0 + 0.1 * randn(D)
        s["q_out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
        s["k_out"], s["v_out"] = (torch.empty(T, Hkv, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        return s
    # sequence b's pages are scattered over the pool; entries past its last page are unused
    wide = max(1, max(used))
    n = torch.tensor(used, device=DEV)
    at = (n.cumsum(0) - n).unsqueeze(1) + torch.arange(wide, device=DEV)
    unused = torch.arange(wide, device=DEV) >= n.unsqueeze(1)
    s["table"] = ids[at.clamp_max(pages - 1)].masked_fill(unused, 0).contiguous()
    s["lens"] = torch.tensor([n for _, n in sizes], device=DEV, dtype=torch.int32)
    if kind == "prefill":
        new = torch.tensor([n for n, _ in sizes], device=DEV)
        s["starts"] = torch.cat((new.new_zeros(1), new.cumsum(0))).to(torch.int32)
        s["most"], s["longest"] = max(n for n, _ in sizes), max(n for _, n in sizes)
    else:
        s["longest"] = max(n for _, n in sizes)
    # queries come out of a fused projection, beside the keys and values
    qkv = (2.0 * randn(T, Hq + 2 * Hkv, D)).to(torch.bfloat16)
    s["q"] = qkv[:, :Hq]
    s["out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
    s["lse"] = torch.empty(T, Hq, device=DEV, dtype=torch.float32)
    return s


# ------------------------------------------------------------------------------ plain forms
def _norm_rope(x, w, pos, inv_freq, inter):
    """x [T, H, D] bf16 -> f32: the norm over D, then the rotation of the first R dims."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    half = inv_freq.numel()
    angle = pos.double().unsqueeze(-1) * inv_freq
    c, si = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * c - b * si, b * c + a * si), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat((a * c - b * si, b * c + a * si), -1)
    return torch.cat((r, rest), -1)


def _append(s):
    s["q_out"].copy_(_norm_rope(s["q"], s["qw"], s["pos"], s["inv_freq"], s["inter"]))
    slots = s["slots"].long()
    page, off, groups = slots // s["page"], slots % s["page"], s["D"] // 32
    k = _norm_rope(s["kin"], s["kw"], s["pos"], s["inv_freq"], s["inter"])
    for rows, pool, scales in ((k, s["k"], s["k_scale"]), (s["vin"].float(), s["v"], s["v_scale"])):
        codes, exps = _mxfp4(rows)
        pool[page, :, off] = codes
        scales[page, :, off, :groups] = exps
    for x in ("k", "v"):
        s[x + "_out"].copy_(_from_mxfp4(s[x][page, :, off], s[x + "_scale"][page, :, off, :groups]))


def _get(s, x, page, off):
    """The rows of pool x at (page, off) [..., H, D] in f32."""
    pool, scales = s[x], s[x + "_scale"]
    if s["fmt"] == "bf16":
        return pool[page, :, off].float()
    if s["fmt"] == "mxfp4":
        return _from_mxfp4(pool[page, :, off], scales[page, :, off, :s["D"] // 32])
    codes = pool.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn)
    return codes.float() * scales[page, :, off].unsqueeze(-1)


def _attend(s, q, pos):
    """q [B, n, Hq, D] f32 at positions pos [B, n] (-1: nothing to attend to) -> (out, lse)."""
    B, n, Hq, D = q.shape
    Hkv, page = s["Hkv"], s["page"]
    t = torch.arange(max(1, s["longest"]), device=DEV)
    seen = t <= pos.unsqueeze(-1)  # [B, n, L]
    if s["window"]:
        seen &= (t > pos.unsqueeze(-1) - s["window"]) | (t < s["sinks"])
    at = s["table"].long()[:, t // page]
    off = (t % page).expand_as(at)
    q = q.view(B, n, Hkv, Hq // Hkv, D) / math.sqrt(D)
    logits = torch.einsum("bnhgd,blhd->bhgnl", q, _get(s, "k", at, off))
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logits.sub_(top))
    del logits
    total = p.sum(-1, keepdim=True)
    v = _get(s, "v", at, off).masked_fill_(~seen.any(1)[:, :, None, None], 0.0)
    out = torch.einsum("bhgnl,blhd->bhgnd", p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top).squeeze(-1)
    return out.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D), lse.permute(0, 3, 1, 2).reshape(B, n, Hq)


def _prefill(s):
    starts = s["starts"].long()
    new = starts.diff()
    i = torch.arange(max(1, s["most"]), device=DEV)
    there = i < new.unsqueeze(1)  # [B, n]
    row = (starts[:-1].unsqueeze(1) + i).clamp_max(s["q"].shape[0] - 1)
    pos = torch.where(there, (s["lens"].long() - new).unsqueeze(1) + i, torch.full_like(row, -1))
    out, lse = _attend(s, s["q"].float()[row], pos)
    s["out"].copy_(out[there])
    s["lse"].copy_(lse[there])


_workspaces = {}


def _handles(attn, s):
    """What a program keeps for its calls: the head shapes, the cache's description and one
    workspace for each head shape."""
    Hq, Hkv, D, many = s["Hq"], s["Hkv"], s["D"], s["kind"] == "prefill"
    s["dims"] = attn.dims(Hq, Hkv, D, rot_dim=s.get("R", 0), rot_interleaved=s.get("inter", False), rms_eps=EPS,
                          window=s.get("window", 0))
    if (Hq, Hkv, D, many) not in _workspaces:
        _workspaces[Hq, Hkv, D, many] = attn.workspace(s["dims"], DEV, prefill=many)
    s["ws"] = _workspaces[Hq, Hkv, D, many]
    s["cache"] = attn.KVCache(s["dims"], s["k"], s["v"], s["k_scale"], s["v_scale"])


def run(s):
    kind = s["kind"]
    if own:
        from mxfp4_routed_expert_latentmoe_gb300 import attn
        if "ws" not in s:
            _handles(attn, s)
        if kind == "append":
            attn.kv_append(s["dims"], s["q"], s["kin"], s["vin"], s["pos"], s["slots"], s["inv_freq"], s["qw"],
                           s["kw"], s["cache"], s["q_out"], s["ws"])
            attn.kv_read(s["dims"], s["slots"], s["cache"], s["k_out"], s["v_out"], s["ws"])
        elif kind == "decode":
            attn.decode(s["dims"], s["q"], s["cache"], s["table"], s["lens"], s["out"], s["ws"], lse=s["lse"],
                        sinks=s["sinks"])
        else:
            attn.prefill(s["dims"], s["q"], s["starts"], s["cache"], s["table"], s["lens"], s["out"], s["ws"],
                         lse=s["lse"], sinks=s["sinks"])
    elif kind == "append":
        _append(s)
    elif kind == "decode":
        out, lse = _attend(s, s["q"].float().unsqueeze(1), s["lens"].long().unsqueeze(1) - 1)
        s["out"].copy_(out.squeeze(1))
        s["lse"].copy_(lse.squeeze(1))
    else:
        _prefill(s)
    if kind == "append":
        # the 4-bit rows' values, in an 8-bit type that holds them exactly
        return {"q": s["q_out"], "k": s["k_out"].to(torch.float8_e4m3fn), "v": s["v_out"].to(torch.float8_e4m3fn)}
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------ from the definition, in 64 bits
def _turned(x, w, pos, inv_freq, inter):
    """The norm and the rotation as complex products."""
    x = x.double()
    x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    half = inv_freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV).expand(pos.numel(), half),
                       torch.outer(pos.double(), inv_freq)).unsqueeze(1)
    y = x.clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else (slice(0, half), slice(half, 2 * half))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _power64(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest(rows):
    """The MXFP4 values of f64 rows: the nearest of the format's values, by distance."""
    x = rows.reshape(*rows.shape[:-1], -1, 32)
    largest = x.abs().max(-1, keepdim=True).values.clamp_min(7 * MIN_SCALE)
    size = _power64(torch.round(torch.log2(largest / 7)))  # (or a step off)
    size = torch.where(largest <= 3.5 * size, size / 2, torch.where(largest > 7 * size, 2 * size, size))
    y = (x / size).abs()
    best, off = torch.zeros_like(y), y.clone()
    # ties go to the even code: 0, 1, 2, 4 (reached from below as well as from above)
    for value, even in ((0.5, False), (1.0, True), (1.5, False), (2.0, True), (3.0, False), (4.0, True), (6.0, False)):
        d = (y - value).abs()
        nearer = (d <= off) if even else (d < off)
        best, off = torch.where(nearer, torch.full_like(y, value), best), torch.where(nearer, d, off)
    return (best * size * x.sign()).reshape(rows.shape)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _rows64(s, x, page, off):
    """[n, Hkv, D] f64 of pool x at (page, off)."""
    raw = s[x].view(torch.uint8)[page, :, off]
    if s["fmt"] == "bf16":
        return raw.view(torch.bfloat16).double()
    if s["fmt"] == "e4m3":
        return raw.view(torch.float8_e4m3fn).double() * s[x + "_scale"][page, :, off].double()[..., None]
    pairs = torch.tensor([[_E2M1[b & 15], _E2M1[b >> 4]] for b in range(256)], dtype=torch.float64, device=DEV)
    values = pairs[raw.long()].reshape(*raw.shape[:2], s["D"] // 32, 32)
    size = _power64(s[x + "_scale"][page, :, off, :s["D"] // 32].double() - 127)
    return (values * size[..., None]).reshape(*raw.shape[:2], s["D"])


def exact(case, seed):
    s = prepare(case, seed)
    D, Hq, Hkv, page = case["D"], case["Hq"], case["Hkv"], case["page"]
    if case["kind"] == "append":
        q = _turned(s["q"], s["qw"], s["pos"], s["inv_freq"], case["inter"])
        k = _turned(s["kin"], s["kw"], s["pos"], s["inv_freq"], case["inter"])
        return {"q": q, "k": _nearest(k), "v": _nearest(s["vin"].double())}
    T = s["q"].shape[0]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    W, row = case["window"], 0
    for b, (new, length) in enumerate(_sizes(case)):
        r, row = slice(row, row + new), row + new
        if not new or not length:
            continue
        t = torch.arange(length, device=DEV)
        p = torch.arange(length - new, length, device=DEV)[:, None]
        hidden = t > p
        if W:
            hidden |= (t <= p - W) & (t >= case["sinks"])
        some = ~hidden.all(0)  # tokens that no query sees are left out
        t, hidden = t[some], hidden[:, some]
        where = s["table"][b].long()[t.div(page, rounding_mode="floor")]
        k, v = (_rows64(s, x, where, t % page) for x in ("k", "v"))
        for h in range(Hq):
            j = h // (Hq // Hkv)
            logits = (s["q"][r, h].double() @ k[:, j].t()) * D ** -0.5
            logits = torch.where(hidden, -math.inf, logits)
            lse[r, h] = torch.logsumexp(logits, -1)
            out[r, h] = torch.softmax(logits, -1) @ v[:, j]
    return {"out": out, "lse": lse}
