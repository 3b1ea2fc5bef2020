"""The attention half of a decoder layer, as a serving step runs it before the routed-expert
block: per-head norms with the position rotation, the paged key-value cache (written in 16
bits or quantised to 8, and read back), and the attention of one new token over its pages.

Every case is one call of one operator on inputs of its own.  With ``own`` false the
operators are computed by elementary torch operations in 32 bits (64 for the angles of far
positions); with ``own`` true by the package's kernels.

Kinds of cases:
  norm_rope  queries and keys of T tokens, normed per head and rotated (dense bf16 results)
  append     the same, with the keys and values going into the paged cache in the same call
  write      keys and values of T tokens written into the cache as they are
  read       the rows of T cached tokens back as dense bf16
  decode     one new query token per sequence over its cached tokens
"""
import math

import torch

own = False

DEV = "cuda"
FP8_MAX = 448.0  # the largest E4M3 value
MIN_SCALE = 2.0 ** -100  # the smallest row scale (rows of zeros and next to it)
EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one sequence with a short prompt behind it: launch and memory latency
        dict(name="decode_one_short", kind="decode", B=1, L=347, Hq=32, Hkv=8, D=128, fmt="e4m3", page=16, window=0),
        # a serving batch, ragged lengths up to 8192, 16-bit cache
        dict(name="decode_batch_bf16", kind="decode", B=64, L=8192, Hq=64, Hkv=8, D=128, fmt="bf16", page=64,
             window=0),
        # two long documents: few rows, the work split over the length; 8-bit cache
        dict(name="decode_long_e4m3", kind="decode", B=2, L=262143, Hq=64, Hkv=8, D=128, fmt="e4m3", page=32,
             window=0),
        # many chats on a sliding-window layer, empty places of the batch among them, twelve
        # query heads on each key head, an odd page size
        dict(name="decode_window_odd", kind="decode", B=201, L=2900, Hq=36, Hkv=3, D=192, fmt="e4m3", page=24,
             window=1000),
        # the decode step of a small batch
        dict(name="append_step", kind="append", T=24, Hq=64, Hkv=8, D=128, R=128, inter=False, fmt="e4m3", page=16,
             far=32768),
        # a prefill chunk, half of the dims rotated, interleaved pairs
        dict(name="append_prefill", kind="append", T=8192, Hq=64, Hkv=8, D=128, R=64, inter=True, fmt="e4m3", page=64,
             far=131072),
        # one token of a small model
        dict(name="norm_rope_token", kind="norm_rope", T=1, Hq=16, Hkv=2, D=64, R=64, inter=False, far=4096),
        # a long prefill at far positions
        dict(name="norm_rope_prefill", kind="norm_rope", T=16381, Hq=64, Hkv=8, D=128, R=128, inter=False,
             far=1 << 20),
        # a prefix computed elsewhere enters the cache, 16 bits
        dict(name="write_prefix_bf16", kind="write", T=1000, Hkv=4, D=192, fmt="bf16", page=16),
        # a large import, quantised
        dict(name="write_import_e4m3", kind="write", T=65536, Hkv=8, D=128, fmt="e4m3", page=64),
        # a short prefix read back, rows of a width that is no power of two
        dict(name="read_short_bf16", kind="read", T=257, Hkv=2, D=96, fmt="bf16", page=24),
        # a long shared prefix read back for a prefill's attention
        dict(name="read_prefix_e4m3", kind="read", T=100003, Hkv=8, D=128, fmt="e4m3", page=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "decode", "append", "norm_rope", "write", "read"])
    D = rng.choice([64, 64, 96, 128, 128, 192, 256])
    fmt = rng.choice(["e4m3", "bf16"])
    page = rng.choice([7, 16, 16, 24, 32, 64, 64, 100, 128])
    if kind == "decode":
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16])
        B = _log_int(rng, 1, 256)
        # at most as many cached bytes and products as the largest listed cases have
        row = 2 * Hkv * D * (1 if fmt == "e4m3" else 2)
        most = min(5e8 / row, 1.6e10 / (4 * Hkv * G * D), 2.5e8 / (Hkv * D))
        L = _log_int(rng, 1, max(2, min(262143, int(most / B))))
        window = rng.choice([0, 0, 0, 128, 1000, 4096])
        return dict(kind=kind, B=B, L=L, Hq=Hkv * G, Hkv=Hkv, D=D, fmt=fmt, page=page, window=window)
    Hkv = rng.choice([1, 2, 4, 8])
    T = _log_int(rng, 1, max(2, int((6.5e7 if kind in ("write", "read") else 1e7) / (Hkv * D))))
    if kind in ("write", "read"):
        return dict(kind=kind, T=T, Hkv=Hkv, D=D, fmt=fmt, page=page)
    G = rng.choice([1, 2, 4, 5, 8])
    R = rng.choice([D, D, D // 2, 32])
    inter = rng.random() < 0.4
    far = rng.choice([4096, 131072, 1 << 20])
    case = dict(kind=kind, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, R=R, inter=inter, far=far)
    if kind == "append":
        case.update(fmt=fmt, page=page)
    return case


def _lengths(case):
    """The sequences' lengths: spread evenly over 1..L in a scattered order, the longest
    first; in a batch of 8 and more every 16th place is empty."""
    B, L = case["B"], case["L"]
    lens = [max(1, min(L, math.ceil(L * (1.0 - math.fmod(b * 0.6180339887498949, 1.0))))) for b in range(B)]
    return [0 if B >= 8 and b % 16 == 7 else n for b, n in enumerate(lens)]


def _attended(case):
    return [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    e4m3 = case.get("fmt") == "e4m3"
    row = D * (1 if e4m3 else 2) + (4 if e4m3 else 0)  # one head's cached key or value
    if case["kind"] == "decode":
        n = sum(_attended(case))
        pages = sum(-(-k // case["page"]) for k in _attended(case))
        return {"bytes": 2 * n * Hkv * row + case["B"] * (case["Hq"] * (4 * D + 4) + 4) + 4 * pages,
                "flops": 4 * n * case["Hq"] * D}
    T = case["T"]
    if case["kind"] in ("write", "read"):
        return {"bytes": T * (2 * Hkv * (row + 2 * D) + 4), "flops": 2 * T * Hkv * D}
    Hq = case["Hq"]
    if case["kind"] == "append":
        moved = T * (Hq * 4 * D + 2 * Hkv * (2 * D + row) + 8)
        return {"bytes": moved + 8 * D + 4 * case["R"], "flops": 10 * T * (Hq + Hkv) * D}
    return {"bytes": T * ((Hq + Hkv) * 4 * D + 4) + 8 * D + 4 * case["R"], "flops": 10 * T * (Hq + Hkv) * D}


# ------------------------------------------------------------------------------ the inputs
def _fill_cache(g, pages, Hkv, page, D, fmt, spread):
    """Random pool of one of K, V: rows ~N(0, 1) times a size of their own."""
    rows = torch.randn(pages, Hkv, page, D, generator=g, device=DEV, dtype=torch.float32)
    if spread:
        rows *= torch.exp(spread * torch.randn(pages, Hkv, page, 1, generator=g, device=DEV))
    if fmt == "bf16":
        return rows.to(torch.bfloat16), None
    scale = (rows.abs().amax(-1) / FP8_MAX).clamp_min(MIN_SCALE)
    rows = (rows * (1.0 / scale).unsqueeze(-1)).clamp_(-FP8_MAX, FP8_MAX)
    return rows.to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    kind, D, Hkv = case["kind"], case["D"], case["Hkv"]
    s = dict(case)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)  # noqa: E731
    if kind != "norm_rope":
        page = case["page"]
        if kind == "decode":
            lens = _lengths(case)
            wide = -(-max(lens) // page)
            used = [-(-n // page) for n in lens]
            pages = sum(used) + 3
        else:
            pages = -(-case["T"] // page) + 3
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["k"], s["k_scale"] = _fill_cache(g, pages, Hkv, page, D, case["fmt"], 0.0)
        s["v"], s["v_scale"] = _fill_cache(g, pages, Hkv, page, D, case["fmt"], 0.5)
    if kind == "decode":
        # sequence b's pages are scattered over the pool; entries past its last page are unused
        n = torch.tensor(used, device=DEV)
        at = (n.cumsum(0) - n).unsqueeze(1) + torch.arange(wide, device=DEV)
        unused = torch.arange(wide, device=DEV) >= n.unsqueeze(1)
        s["table"] = ids[at.clamp_max(pages - 1)].masked_fill(unused, 0).contiguous()
        s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
        # queries come out of a fused projection, beside the keys and values
        qkv = (2.0 * randn(case["B"], case["Hq"] + 2 * Hkv, D)).to(torch.bfloat16)
        s["q"] = qkv[:, :case["Hq"]]
        s["out"] = torch.empty(case["B"], case["Hq"], D, device=DEV, dtype=torch.bfloat16)
        s["lse"] = torch.empty(case["B"], case["Hq"], device=DEV, dtype=torch.float32)
    else:
        T, Hq = case["T"], case.get("Hq", 0)
        qkv = (randn(T, Hq + 2 * Hkv, D) * torch.exp(0.5 * randn(T, 1, 1))).to(torch.bfloat16)
        s["q"], s["kin"], s["vin"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if kind != "norm_rope":
            # consecutive tokens of scattered pages
            t = torch.arange(T, device=DEV)
            s["slots"] = ids[t // page] * page + (t % page).to(torch.int32)
        if kind in ("norm_rope", "append"):
            s["pos"] = torch.randint(0, case["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
            s["inv_freq"] = THETA ** (-torch.arange(0, case["R"], 2, device=DEV, dtype=torch.float64) / case["R"])
            s["qw"], s["kw"] = 1.0 + 0.1 * randn(D), 1.0 + 0.1 * randn(D)
            s["q_out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
        if kind in ("norm_rope", "read"):
            s["k_out"] = torch.empty(T, Hkv, D, device=DEV, dtype=torch.bfloat16)
        if kind == "read":
            s["v_out"] = torch.empty(T, Hkv, D, device=DEV, dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------------------------ plain forms
def _norm_rope(x, w, pos, inv_freq, inter):
    """x [T, H, D] bf16 -> f32: the norm over D, then the rotation of the first R dims."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    half = inv_freq.numel()
    if half == 0:
        return x
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


def _put(pool, scales, rows, page, off):
    """Rows [T, H, D] f32 into the pool's places (page, off) of every head, quantised if it
    has scales."""
    if scales is None:
        pool[page, :, off] = rows.to(torch.bfloat16)
        return
    scale = (rows.abs().amax(-1) / FP8_MAX).clamp_min(MIN_SCALE)
    codes = (rows * (1.0 / scale).unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    pool.view(torch.uint8)[page, :, off] = codes.view(torch.uint8)
    scales[page, :, off] = scale


def _get(pool, scales, page, off):
    """The pool's rows at (page, off) [..., H, D] in f32."""
    if scales is None:
        return pool[page, :, off].float()
    codes = pool.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn)
    return codes.float() * scales[page, :, off].unsqueeze(-1)


def _decode(s):
    B, Hq, D = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]
    t = torch.arange(s["table"].shape[1] * page, device=DEV)[:s["L"]]
    n = s["lens"].unsqueeze(1)
    first = (n - s["window"]).clamp_min(0) if s["window"] else torch.zeros_like(n)
    seen = (t >= first) & (t < n)  # [B, L]
    at = s["table"].long()[:, t // page]
    off = (t % page).expand_as(at)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D) / math.sqrt(D)
    k = _get(s["k"], s["k_scale"], at, off)  # [B, L, Hkv, D]
    logits = torch.einsum("bhgd,blhd->bhgl", q, k)
    del k
    logits = logits.masked_fill(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    v = _get(s["v"], s["v_scale"], at, off).masked_fill_(~seen[:, :, None, None], 0.0)
    out = torch.einsum("bhgl,blhd->bhgd", p, v) / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(out.reshape(B, Hq, D))
    s["lse"].copy_((torch.log(total) + top).reshape(B, Hq))
    return {"out": s["out"], "lse": s["lse"]}


def _pool(s):
    got = {"k": s["k"], "v": s["v"]}
    if s["k_scale"] is not None:
        got.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return got


_workspaces = {}


def _handles(attn, s):
    """What a program keeps for its calls: the head shapes, the cache's description and one
    workspace for each head shape."""
    Hq, Hkv, D = s.get("Hq", s["Hkv"]), s["Hkv"], s["D"]
    s["dims"] = attn.dims(Hq, Hkv, D, rot_dim=s.get("R", 0), rot_interleaved=s.get("inter", False), rms_eps=EPS,
                          window=s.get("window", 0))
    if (Hq, Hkv, D) not in _workspaces:
        _workspaces[Hq, Hkv, D] = attn.workspace(s["dims"], DEV)
    s["ws"] = _workspaces[Hq, Hkv, D]
    if "k_scale" in s:
        s["cache"] = attn.KVCache(s["dims"], s["k"], s["v"], s["k_scale"], s["v_scale"])


def run(s):
    kind = s["kind"]
    if own:
        from mxfp4_routed_expert_latentmoe_gb300 import attn
        if "ws" not in s:
            _handles(attn, s)
        if kind == "decode":
            attn.decode(s["dims"], s["q"], s["cache"], s["table"], s["lens"], s["out"], s["ws"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if kind == "norm_rope":
            attn.qk_norm_rope(s["dims"], s["q"], s["kin"], s["pos"], s["inv_freq"], s["qw"], s["kw"], s["q_out"],
                              s["k_out"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if kind == "append":
            attn.kv_append(s["dims"], s["q"], s["kin"], s["vin"], s["pos"], s["slots"], s["inv_freq"], s["qw"],
                           s["kw"], s["cache"], s["q_out"], s["ws"])
            return {"q": s["q_out"], **_pool(s)}
        if kind == "write":
            attn.kv_write(s["dims"], s["kin"], s["vin"], s["slots"], s["cache"], s["ws"])
            return _pool(s)
        attn.kv_read(s["dims"], s["slots"], s["cache"], s["k_out"], s["v_out"], s["ws"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if kind == "decode":
        return _decode(s)
    if kind in ("norm_rope", "append"):
        s["q_out"].copy_(_norm_rope(s["q"], s["qw"], s["pos"], s["inv_freq"], s["inter"]))
        k = _norm_rope(s["kin"], s["kw"], s["pos"], s["inv_freq"], s["inter"])
        if kind == "norm_rope":
            s["k_out"].copy_(k)
            return {"q": s["q_out"], "k": s["k_out"]}
    slots = s["slots"].long()
    page, off = slots // s["page"], slots % s["page"]
    if kind == "read":
        s["k_out"].copy_(_get(s["k"], s["k_scale"], page, off))
        s["v_out"].copy_(_get(s["v"], s["v_scale"], page, off))
        return {"k": s["k_out"], "v": s["v_out"]}
    _put(s["k"], s["k_scale"], k if kind == "append" else s["kin"].float(), page, off)
    _put(s["v"], s["v_scale"], s["vin"].float(), page, off)
    return {"q": s["q_out"], **_pool(s)} if kind == "append" else _pool(s)


# ------------------------------------------------------------------------------ from the definition, in 64 bits
def _turned(x, w, pos, inv_freq, inter):
    """The norm and the rotation as complex products."""
    x = x.double()
    x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    half = inv_freq.numel()
    if not half:
        return x
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV).expand(pos.numel(), half),
                       torch.outer(pos.double(), inv_freq)).unsqueeze(1)
    y = x.clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else (slice(0, half), slice(half, 2 * half))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _pool_after(pool, scales, rows, slots, page):
    """The pool after the write, with the values before their rounding (in units of the row's
    scale where there is one), and the scales."""
    P, H, S, D = pool.shape
    after = pool.to(torch.float64).transpose(1, 2).reshape(P * S, H, D)
    if scales is None:
        after[slots] = rows
        return after.view(P, S, H, D).transpose(1, 2), None
    after_scales = scales.double().transpose(1, 2).reshape(P * S, H)
    scale = torch.maximum(rows.abs().max(-1).values / FP8_MAX, torch.full((), MIN_SCALE, dtype=torch.float64,
                                                                          device=DEV))
    after[slots], after_scales[slots] = rows / scale[..., None], scale
    return after.view(P, S, H, D).transpose(1, 2), after_scales.view(P, S, H).transpose(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    kind, D, Hkv = case["kind"], case["D"], case["Hkv"]
    if kind == "decode":
        B, Hq, page = case["B"], case["Hq"], case["page"]
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(_lengths(case)):
            f = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            t = torch.arange(f, n, device=DEV)
            where = s["table"][b].long()[t.div(page, rounding_mode="floor")]
            kv = []
            for x in ("k", "v"):
                rows = s[x].view(torch.uint8)[where, :, t % page].view(s[x].dtype).double()
                if s[x + "_scale"] is not None:
                    rows *= s[x + "_scale"][where, :, t % page].double()[..., None]
                kv.append(rows.transpose(0, 1))  # [Hkv, n, D]
            q = s["q"][b].double().reshape(Hkv, Hq // Hkv, D)
            logits = torch.bmm(q, kv[0].transpose(1, 2)) * D ** -0.5
            lse[b] = torch.logsumexp(logits, -1).reshape(Hq)
            out[b] = torch.bmm(torch.softmax(logits, -1), kv[1]).reshape(Hq, D)
        return {"out": out, "lse": lse}
    if kind in ("norm_rope", "append"):
        q = _turned(s["q"], s["qw"], s["pos"], s["inv_freq"], case["inter"])
        k = _turned(s["kin"], s["kw"], s["pos"], s["inv_freq"], case["inter"])
        if kind == "norm_rope":
            return {"q": q, "k": k}
    slots = s["slots"].long()
    if kind == "read":
        got = {}
        for x in ("k", "v"):
            rows = s[x].to(torch.float64)
            if s[x + "_scale"] is not None:
                rows = rows * s[x + "_scale"].double()[..., None]
            got[x] = rows.transpose(1, 2).reshape(-1, Hkv, D)[slots]
        return got
    got = {"q": q} if kind == "append" else {}
    for x, rows in (("k", k if kind == "append" else s["kin"].double()), ("v", s["vin"].double())):
        got[x], scales = _pool_after(s[x], s[x + "_scale"], rows, slots, case["page"])
        if scales is not None:
            got[x + "_scale"] = scales
    return got
