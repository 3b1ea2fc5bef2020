"""The attention operators on the GPU against plain 64-bit forms: norms with the rotation, the
paged cache written and read, and the decode attention over it.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of E4M3 2^-4 (2^-10 of
the row's scale below its normal range), of fp16 2^-11, of fp32 2^-24."""
import pytest

from tests import _attn_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16_HALF, E4M3_HALF = 2.0 ** -8, 2.0 ** -4
# fp32 roundings of a normed and rotated element, relative to the magnitudes it combines: the
# sum of squares takes at most 8 + 5 of them (13 halved by the root), the root, quotient and
# two products 5, the turn's fraction and its sine or cosine 8, the rotation 3: under 32
F32_ROWS = 32 * 2.0 ** -24


@pytest.fixture(scope="module")
def attn():
    import __graft_entry__ as g
    g.build()
    from mxfp4_routed_expert_latentmoe_gb300 import attn as mod
    torch.cuda.set_device(0)
    return mod


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _qkv(T, Hq, Hkv, D, seed):
    """q, k, v as slices of one projection's output (token strides of (Hq + 2 Hkv) D)."""
    x = (2.0 * torch.randn(T, Hq + 2 * Hkv, D, generator=_gen(seed), device="cuda")).to(torch.bfloat16)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _weights(D, seed):
    g = _gen(seed + 1000)
    return [1.0 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]


def _close(got, want, tol, what=""):
    off = (got.double().cpu() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off - tol).max()):.3e} over"


NORM_CASES = [  # T, Hq, Hkv, D, R, interleaved
    (1, 1, 1, 16, 0, False), (1, 1, 1, 16, 16, True), (1, 16, 2, 64, 64, False), (5, 6, 3, 96, 32, True),
    (3, 8, 8, 128, 64, False), (67, 5, 1, 256, 256, True), (2, 3, 1, 192, 96, False), (7, 2, 2, 48, 48, False),
    (130, 12, 2, 80, 16, False), (33, 64, 8, 128, 128, False), (600, 4, 1, 240, 240, False), (301, 9, 3, 112, 0, True)]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,inter", NORM_CASES)
def test_norm_rope(attn, T, Hq, Hkv, D, R, inter):
    d = attn.dims(Hq, Hkv, D, rot_dim=R, rot_interleaved=inter, rms_eps=1e-5)
    q, k, _ = _qkv(T, Hq, Hkv, D, 1)
    qw, kw = _weights(D, 1)
    pos = torch.randint(0, 5000, (T,), generator=_gen(2), device="cuda", dtype=torch.int32)
    pos[0] = 0
    freq = attn.rope_frequencies(R, 1e4) if R else None
    qo, ko = torch.empty(T, Hq, D, device="cuda", dtype=torch.bfloat16), torch.empty(T, Hkv, D, device="cuda",
                                                                                      dtype=torch.bfloat16)
    attn.qk_norm_rope(d, q, k, pos, freq, qw, kw, qo, ko)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        y, size = ref.norm_rope(x, w, pos, freq, 1e-5, inter)
        _close(got, y, BF16_HALF * y.abs() + 2 * F32_ROWS * size)


def test_norm_rope_at_far_and_negative_positions(attn):
    """Angles whose whole turns fp32 could not hold: the product in fp64 leaves pos * f * 2^-52
    radians, 2^-21 at 2^31."""
    T, D = 6, 128
    d = attn.dims(2, 1, D)
    q, k, _ = _qkv(T, 2, 1, D, 3)
    qw, kw = _weights(D, 3)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 1 << 20, -1, 123456789, 16777217], device="cuda", dtype=torch.int32)
    freq = attn.rope_frequencies(D, 1e6)
    qo, ko = (torch.empty(T, h, D, device="cuda", dtype=torch.bfloat16) for h in (2, 1))
    attn.qk_norm_rope(d, q, k, pos, freq, qw, kw, qo, ko)
    y, size = ref.norm_rope(q, qw, pos, freq, 1e-6, False)
    _close(qo, y, BF16_HALF * y.abs() + (2 * F32_ROWS + 2 * 2.0 ** -21) * size)


def test_norm_rope_in_place_rows_of_zeros_and_non_finite_rows(attn):
    T, D = 4, 64
    d = attn.dims(2, 2, D, rms_eps=1e-6)
    x = torch.randn(T, 4, D, generator=_gen(4), device="cuda").to(torch.bfloat16)
    x[1, 0] = 0.0
    x[2, 1, 3] = float("nan")
    q, k = x[:, :2].contiguous(), x[:, 2:].contiguous()
    qw, kw = _weights(D, 4)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    freq = attn.rope_frequencies(D)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    attn.qk_norm_rope(d, q, k, pos, freq, qw, kw, qo, ko)
    assert (qo[1, 0] == 0).all() and torch.isnan(qo[2, 1]).all() and torch.isfinite(qo[2, 0]).all()
    attn.qk_norm_rope(d, q, k, pos, freq, qw, kw, q, k)
    assert torch.equal(q.view(torch.int16), qo.view(torch.int16)) and torch.equal(k, ko)


# ------------------------------------------------------------------------------ the cache
def _pools(attn, d, n_pages, page, fmt, seed, order="phtd"):
    """A cache of random contents over tensors in the given memory order of pages, heads, tokens
    and the row's values."""
    g = _gen(seed)
    H, D = d.n_kv_heads, d.head_dim
    sizes = dict(p=n_pages, h=H, t=page, d=D)

    def tensor(dtype, o):
        raw = torch.randint(0, 256, [sizes[c] for c in o], generator=g, device="cuda", dtype=torch.uint8)
        raw = (raw & 0x77) if dtype == torch.float8_e4m3fn else raw
        t = raw.view(dtype) if dtype == torch.float8_e4m3fn else (raw.float() / 64 - 2).to(dtype)
        return t.permute([o.index(c) for c in "phtd" if c in o])

    if fmt == "bf16":
        return attn.KVCache(d, tensor(torch.bfloat16, order), tensor(torch.bfloat16, order))
    so = order.replace("d", "")
    return attn.KVCache(d, tensor(torch.float8_e4m3fn, order), tensor(torch.float8_e4m3fn, order),
                        tensor(torch.float32, so), tensor(torch.float32, so))


def _slots(T, n_pages, page, seed):
    return torch.randperm(n_pages * page, generator=_gen(seed), device="cuda")[:T].to(torch.int32)


def _bytes(t):
    return t.contiguous().view(torch.uint8 if t.dtype == torch.float8_e4m3fn else
                               (torch.int16 if t.dtype == torch.bfloat16 else torch.int32)).cpu()


CACHE_CASES = [  # T, Hkv, D, page, order
    (1, 1, 16, 1, "phtd"), (5, 2, 64, 7, "phtd"), (40, 3, 96, 16, "pthd"), (129, 8, 128, 64, "hptd"),
    (300, 1, 256, 24, "tphd"), (33, 5, 80, 3, "phtd")]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,Hkv,D,page,order", CACHE_CASES)
def test_write_and_read_are_exact(attn, T, Hkv, D, page, order, fmt):
    """Written rows equal the definition's bit for bit, all others stay; reading gives code *
    scale rounded to bf16.  Rows of zeros, tiny, huge and non-finite ones among them."""
    d = attn.dims(Hkv, Hkv, D, rot_dim=0)
    n_pages = -(-T // page) + 2
    cache = _pools(attn, d, n_pages, page, fmt, 5, order)
    ws = attn.workspace(d)
    _, k, v = _qkv(T, 1, Hkv, D, 6)
    k[0, 0] = 0.0
    v[T // 2, Hkv - 1] *= 1e-38
    v[T - 1, 0] *= 1e37
    if T > 4:
        k[2, 0, 5] = float("inf")
        v[3, 0, 0] = float("nan")
    slots = _slots(T, n_pages, page, 7)
    if T > 1:
        slots[1] = -1
    before = {n: _bytes(getattr(cache, n)).clone() for n in ("k", "v")}
    attn.kv_write(d, k, v, slots, cache, ws)
    written = slots >= 0
    pg, at = (slots[written] // page).long().cpu(), (slots[written] % page).long().cpu()
    for name, x in (("k", k), ("v", v)):
        want = before[name].clone()
        if fmt == "bf16":
            want[pg, :, at] = x[written].contiguous().view(torch.int16).cpu()
            assert torch.equal(_bytes(getattr(cache, name)), want)
            continue
        codes, scale = ref.quantise_f32(x[written])
        want[pg, :, at] = codes
        got = _bytes(getattr(cache, name))
        nan = torch.isnan(scale)
        assert torch.equal(got[pg, :, at][~nan], codes[~nan])
        assert ((got[pg, :, at][nan] & 0x7F) == 0x7F).all()
        got[pg, :, at] = want[pg, :, at]
        assert torch.equal(got, want)  # the other rows
        gs = getattr(cache, name + "_scale").cpu()[pg, :, at]
        assert torch.equal(gs[~nan], scale[~nan]) and torch.isnan(gs[nan]).all()
    ko, vo = (torch.full((T, Hkv, D), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    attn.kv_read(d, slots, cache, ko, vo, ws)
    for got, pool, scales in ((ko, cache.k, cache.k_scale), (vo, cache.v, cache.v_scale)):
        want = ref.gather(pool, scales, pg, at).float().to(torch.bfloat16)
        g = got[written].cpu()
        same = (g.view(torch.int16) == want.view(torch.int16)) | (torch.isnan(g) & torch.isnan(want))
        assert same.all()
        assert (got[~written] == 0).all()
    assert attn.device_status(ws) == 0


def test_slots_outside_the_cache_are_skipped_and_reported(attn):
    d = attn.dims(2, 2, 64, rot_dim=0)
    cache = _pools(attn, d, 3, 16, "e4m3", 8)
    ws = attn.workspace(d)
    _, k, v = _qkv(4, 1, 2, 64, 9)
    before = [_bytes(t).clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    bad = torch.tensor([48, -2, 2 ** 31 - 1, -1], device="cuda", dtype=torch.int32)
    attn.kv_write(d, k, v, torch.full_like(bad, -1), cache, ws)
    assert attn.device_status(ws) == 0
    attn.kv_write(d, k, v, bad, cache, ws)
    assert attn.device_status(ws) == attn.DEV_BAD_SLOT
    assert all(torch.equal(_bytes(t), b) for t, b in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before))
    attn.workspace_init(ws)
    assert attn.device_status(ws) == 0
    ko, vo = torch.ones(4, 2, 64, device="cuda", dtype=torch.bfloat16), torch.ones(4, 2, 64, device="cuda",
                                                                                     dtype=torch.bfloat16)
    attn.kv_read(d, bad, cache, ko, vo, ws)
    assert (ko == 0).all() and (vo == 0).all() and attn.device_status(ws) == attn.DEV_BAD_SLOT


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,inter,page", [
    (1, 8, 2, 64, 64, False, 16), (37, 6, 3, 96, 48, True, 5), (260, 16, 2, 256, 128, False, 64),
    (64, 12, 4, 128, 128, True, 16), (5, 7, 7, 176, 0, False, 7)])
def test_append(attn, T, Hq, Hkv, D, R, inter, page, fmt):
    """The fused pass: queries as qk_norm_rope gives them, values as kv_write does (bit for bit),
    keys quantised from their fp32 values."""
    d = attn.dims(Hq, Hkv, D, rot_dim=R, rot_interleaved=inter)
    n_pages = -(-T // page) + 1
    cache, plain = (_pools(attn, d, n_pages, page, fmt, 10) for _ in range(2))
    ws = attn.workspace(d)
    q, k, v = _qkv(T, Hq, Hkv, D, 11)
    qw, kw = _weights(D, 11)
    pos = torch.randint(0, 100000, (T,), generator=_gen(12), device="cuda", dtype=torch.int32)
    freq = attn.rope_frequencies(R) if R else None
    slots = _slots(T, n_pages, page, 13)
    if T > 2:
        slots[2] = -1
    qo, ko, q1, k1 = (torch.empty(T, h, D, device="cuda", dtype=torch.bfloat16) for h in (Hq, Hkv, Hq, Hkv))
    attn.kv_append(d, q, k, v, pos, slots, freq, qw, kw, cache, qo, ws, k_out=ko)
    attn.qk_norm_rope(d, q, k, pos, freq, qw, kw, q1, k1)
    attn.kv_write(d, k, v, slots, plain, ws)
    assert torch.equal(qo, q1) and torch.equal(ko, k1)
    assert torch.equal(_bytes(cache.v), _bytes(plain.v))
    written = slots >= 0
    pg, at = (slots[written] // page).long(), (slots[written] % page).long()
    y, size = ref.norm_rope(k[written], kw, pos[written], freq, 1e-6, inter)
    got = ref.gather(cache.k, cache.k_scale, pg, at)
    if fmt == "bf16":
        _close(got, y, BF16_HALF * y.abs() + 2 * F32_ROWS * size)
    else:
        scale = y.abs().amax(-1, keepdim=True) / 448.0
        _close(got, y, torch.maximum(E4M3_HALF * y.abs(), 2.0 ** -10 * scale) + 4 * F32_ROWS * (size + 448 * scale))
        assert torch.equal(_bytes(cache.v_scale), _bytes(plain.v_scale))
    qo2 = torch.empty_like(qo)
    attn.kv_append(d, q, k, v, pos, slots, freq, qw, kw, plain, qo2, ws)  # without k_out
    assert torch.equal(qo, qo2) and torch.equal(_bytes(plain.k), _bytes(cache.k))
    assert attn.device_status(ws) == 0


# ------------------------------------------------------------------------------ decode
def _sequences(attn, d, lens, page, fmt, seed, spread=0.5, order="phtd", q_size=2.0):
    """Queries and a cache that holds the sequences on scattered pages, with NaN (bf16) or NaN
    scales in every row that no sequence has; table entries past a sequence's end point
    nowhere."""
    g = _gen(seed)
    B, H, D = len(lens), d.n_kv_heads, d.head_dim
    wide = max(1, max(-(-n // page) for n in lens))
    used = sum(-(-n // page) for n in lens)
    n_pages = used + 2
    cache = _pools(attn, d, n_pages, page, fmt, seed, order)
    stale = cache.k if fmt == "bf16" else cache.k_scale
    stale.fill_(float("nan"))
    (cache.v if fmt == "bf16" else cache.v_scale).fill_(float("nan"))
    ids = torch.randperm(n_pages, generator=g, device="cuda")[:used].to(torch.int32)
    table = torch.full((B, wide), -7, device="cuda", dtype=torch.int32)
    table[:, wide // 2:] = 2 ** 31 - 1
    slots, at = [], 0
    for b, n in enumerate(lens):
        np_ = -(-n // page)
        table[b, :np_] = ids[at:at + np_]
        t = torch.arange(n, device="cuda", dtype=torch.int32)
        slots.append(ids[at:at + np_][(t // page).long()] * page + t % page)
        at += np_
    slots = torch.cat(slots).to(torch.int32)
    T = slots.numel()
    k = torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    v = (torch.randn(T, H, D, generator=g, device="cuda") *
         torch.exp(spread * torch.randn(T, H, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    ws = attn.workspace(d)
    if T:
        attn.kv_write(d, k, v, slots, cache, ws)
    q, _, _ = _qkv(B, d.n_heads, H, D, seed + 1)
    q = (q.float() * (q_size / 2)).to(torch.bfloat16) if q_size != 2.0 else q
    return q, cache, table, torch.tensor(lens, device="cuda", dtype=torch.int32), slots, ws


def _check_decode(attn, d, q, cache, slots, lens, out, lse, page):
    at = 0
    for b, n in enumerate(lens):
        f = max(0, n - d.window) if d.window else 0
        s = slots[at + f:at + n].long()
        at += n
        k = ref.gather(cache.k, cache.k_scale, s // page, s % page)
        v = ref.gather(cache.v, cache.v_scale, s // page, s % page)
        o, z, mean_abs, slack = ref.decode(q[b].double().cpu(), k, v, d.softmax_scale)
        # the weights enter the second product rounded to bf16 at most, with the logits' fp32
        # error in their exponent (twice: above and below); the output is rounded to bf16
        tol = BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + (64 + n / 8) * 2.0 ** -24)
        _close(out[b], o, tol, f"sequence {b} of {n}")
        if n - f == 0:
            assert (lse[b] == -torch.inf).all()
        else:
            _close(lse[b], z, slack + (64 + n / 8) * 2.0 ** -24 + 2.0 ** -22 * z.abs(), f"lse {b}")


def _run_decode(attn, d, q, cache, table, lens_t, ws):
    B = q.shape[0]
    out = torch.full((B, d.n_heads, d.head_dim), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((B, d.n_heads), 7.0, device="cuda")
    attn.decode(d, q, cache, table, lens_t, out, ws, lse=lse)
    return out, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 0, 127, 129, 300, 1000]
DECODE_CASES = [  # Hq, Hkv, D, page, window, order, lens
    (1, 1, 16, 1, 0, "phtd", [1]), (8, 8, 64, 16, 0, "phtd", LENS), (8, 1, 128, 16, 0, "phtd", LENS),
    (64, 8, 128, 64, 0, "phtd", [1, 700, 0, 5000]), (6, 2, 96, 7, 0, "pthd", LENS),
    (24, 2, 256, 24, 0, "phtd", LENS), (36, 3, 192, 24, 100, "hptd", LENS), (5, 1, 80, 3, 17, "tphd", LENS),
    (16, 1, 64, 128, 0, "phtd", [4097]), (34, 2, 128, 16, 0, "phtd", LENS), (40, 1, 256, 32, 0, "phtd", [77, 513]),
    (7, 7, 48, 16, 1, "phtd", LENS), (2, 1, 128, 32, 0, "phtd", [70001]), (9, 3, 240, 5, 64, "phtd", LENS),
    (8, 2, 128, 64, 0, "phtd", [0, 0, 0]), (16, 8, 64, 16, 0, "phtd", [3 * i % 97 for i in range(400)]),
    (100, 1, 64, 16, 0, "phtd", [200, 0, 1])]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,window,order,lens", DECODE_CASES,
                         ids=[f"{c[0]}x{c[1]}x{c[2]}-p{c[3]}-w{c[4]}-{c[5]}-{len(c[6])}of{max(c[6])}"
                              for c in DECODE_CASES])
def test_decode(attn, Hq, Hkv, D, page, window, order, lens, fmt):
    d = attn.dims(Hq, Hkv, D, window=window)
    q, cache, table, lens_t, slots, ws = _sequences(attn, d, lens, page, fmt, 20, order=order)
    out, lse = _run_decode(attn, d, q, cache, table, lens_t, ws)
    _check_decode(attn, d, q, cache, slots, lens, out, lse, page)
    # the same call again (the workspace is left ready), without lse: the same bits
    out2 = torch.empty_like(out)
    attn.decode(d, q, cache, table, lens_t, out2, ws)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    assert attn.device_status(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 1, 64), (24, 2, 96), (32, 2, 128), (60, 3, 128), (36, 3, 192), (24, 2, 256),
                                      (17, 1, 256)])
def test_decode_of_many_query_heads_with_room_in_the_page_table(attn, Hq, Hkv, D, fmt):
    """Calls are shaped by the lengths that the table allows: the same ones with a table of just
    the pages that the sequences have and with one for 2^20 tokens (its rest is never read)."""
    d = attn.dims(Hq, Hkv, D)
    for lens in (LENS, [0, 500, 2300]):
        q, cache, table, lens_t, slots, ws = _sequences(attn, d, lens, 16, fmt, 28)
        wide = torch.full((len(lens), 2 ** 16), -1, device="cuda", dtype=torch.int32)
        wide[:, :table.shape[1]] = table
        for t in (table, wide, table):
            out, lse = _run_decode(attn, d, q, cache, t, lens_t, ws)
            _check_decode(attn, d, q, cache, slots, lens, out, lse, 16)
            out2, lse2 = _run_decode(attn, d, q, cache, t, lens_t, ws)
            assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)
        assert attn.device_status(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_decode_sharp_logits_and_values_of_many_sizes(attn, fmt):
    """Logits of hundreds (one token takes all) and values whose rows differ by up to e^(4 * 4)
    in size."""
    d = attn.dims(16, 2, 128)
    lens = [3, 70, 900]
    for q_size, spread in ((60.0, 0.5), (2.0, 4.0), (20.0, 4.0)):
        q, cache, table, lens_t, slots, ws = _sequences(attn, d, lens, 16, fmt, 21, spread=spread, q_size=q_size)
        out, lse = _run_decode(attn, d, q, cache, table, lens_t, ws)
        _check_decode(attn, d, q, cache, slots, lens, out, lse, 16)


def test_decode_rows_without_weight_and_non_finite_tokens(attn):
    d = attn.dims(4, 2, 64)
    q, cache, table, lens_t, slots, ws = _sequences(attn, d, [40, 40, 40], 16, "bf16", 22)
    q[0] = q[0].abs() + 0.1
    pg, at = (slots // 16).long(), (slots % 16).long()
    cache.k[pg[:40], :, at[:40]] = float("-inf")  # sequence 0: every logit is -infinity
    cache.k[pg[45], 0, at[45], 0] = float("nan")  # sequence 1: a NaN in one key of key head 0
    out, lse = _run_decode(attn, d, q, cache, table, lens_t, ws)
    assert (out[0] == 0).all() and (lse[0] == -torch.inf).all()
    assert torch.isnan(out[1, :2]).all() and torch.isnan(lse[1, :2]).all()
    assert torch.isfinite(out[1, 2:]).all() and torch.isfinite(out[2]).all()
    # E4M3: rows of zero scale, a NaN scale
    q, cache, table, lens_t, slots, ws = _sequences(attn, d, [40, 40], 16, "e4m3", 23)
    pg, at = (slots // 16).long(), (slots % 16).long()
    cache.v_scale[pg[:20], :, at[:20]] = 0.0
    cache.k_scale[pg[5:10], :, at[5:10]] = 0.0
    cache.v_scale[pg[60], 1, at[60]] = float("nan")
    out, lse = _run_decode(attn, d, q, cache, table, lens_t, ws)
    _check_decode(attn, d, q[:1], cache, slots, [40], out, lse, 16)
    assert torch.isnan(out[1, 2:]).all() and torch.isfinite(out[1, :2]).all() and torch.isfinite(lse).all()


def test_decode_bad_pages_and_lengths_are_left_out_and_reported(attn):
    d = attn.dims(8, 2, 128)
    lens = [100, 64, 50]
    q, cache, table, lens_t, slots, ws = _sequences(attn, d, lens, 16, "e4m3", 24)
    table[0, 2] = -3
    table[0, 4] = cache.n_pages
    out, lse = _run_decode(attn, d, q, cache, table, lens_t, ws)
    assert attn.device_status(ws) == attn.DEV_BAD_PAGE
    keep = torch.cat([slots[:32], slots[48:64], slots[80:]])
    _check_decode(attn, d, q, cache, keep, [68, 64, 50], out, lse, 16)
    attn.workspace_init(ws)
    table[0, 2] = table[0, 4] = table[0, 0]
    bad = torch.tensor([0, -5, 2 ** 31 - 1], device="cuda", dtype=torch.int32)
    table[2] = table[1, 0]
    out, lse = _run_decode(attn, d, q, cache, table, bad, ws)
    assert attn.device_status(ws) == attn.DEV_BAD_LENGTH
    assert (out[:2] == 0).all() and (lse[:2] == -torch.inf).all() and torch.isfinite(out[2]).all()


def test_decode_of_a_cache_past_32_bits(attn):
    """Pages whose bytes and elements lie past 2^32 (only the used ones are filled)."""
    d = attn.dims(8, 4, 128)
    page, n_pages = 256, 36000  # 4.7e9 codes
    k, v = (torch.empty(n_pages, 4, page, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            for _ in range(2))
    ks, vs = (torch.empty(n_pages, 4, page, device="cuda") for _ in range(2))
    cache = attn.KVCache(d, k, v, ks, vs)
    ws = attn.workspace(d)
    n = 600
    table = torch.tensor([[n_pages - 1, 5, n_pages - 2]], device="cuda", dtype=torch.int32)
    t = torch.arange(n, device="cuda")
    slots = (table[0].long()[t // page] * page + t % page).to(torch.int32)
    q, kk, vv = _qkv(n, 8, 4, 128, 25)
    attn.kv_write(d, kk, vv, slots, cache, ws)
    out, lse = _run_decode(attn, d, q[:1], cache, table, torch.tensor([n], device="cuda", dtype=torch.int32), ws)
    kr, vr = (torch.empty(n, 4, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    attn.kv_read(d, slots, cache, kr, vr, ws)
    codes, scale = ref.quantise_f32(kk)
    back = (codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]).float().to(torch.bfloat16)
    assert torch.equal(kr.cpu(), back)
    rows = [(c.view(torch.float8_e4m3fn).double() * s.double()[..., None]) for c, s in
            (ref.quantise_f32(kk), ref.quantise_f32(vv))]
    o, z, mean_abs, slack = ref.decode(q[0].double().cpu(), *rows, d.softmax_scale)
    _close(out[0], o, BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + 139 * 2.0 ** -24))
    assert attn.device_status(ws) == 0


def test_streams_and_a_captured_step_that_replays_with_new_lengths(attn):
    d = attn.dims(16, 4, 128)
    lens = [130, 1, 77]
    q, cache, table, lens_t, slots, ws = _sequences(attn, d, lens, 16, "e4m3", 26)
    out, lse = _run_decode(attn, d, q, cache, table, lens_t, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    attn.decode(d, q, cache, table, lens_t, out2, ws, lse=lse2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    # a step (append, then decode) as a graph: replayed with other inputs in the same buffers
    x, k, v = _qkv(3, 16, 4, 128, 27)
    qw, kw = _weights(128, 27)
    freq = attn.rope_frequencies(128)
    pos, new = torch.tensor(lens, device="cuda", dtype=torch.int32), lens_t + 1
    ends = torch.tensor(lens).cumsum(0) - 1
    at = torch.tensor([130 % 16, 1, 77 % 16], device="cuda", dtype=torch.int32)
    step_slots = table[torch.arange(3, device="cuda"), (pos // 16).long()] * 16 + at
    assert ends[-1] + 1 == slots.numel()
    q_out = torch.empty(3, 16, 128, device="cuda", dtype=torch.bfloat16)

    def step():
        attn.kv_append(d, x, k, v, pos, step_slots, freq, qw, kw, cache, q_out, ws)
        attn.decode(d, q_out, cache, table, new, out2, ws, lse=lse2)

    step()
    torch.cuda.synchronize()
    want = out2.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    out2.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, want)
    new.copy_(torch.tensor([64, 2, 0], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    eager, _ = _run_decode(attn, d, q_out, cache, table, new, ws)
    assert torch.equal(out2, eager) and (out2[2] == 0).all()
    assert attn.device_status(ws) == 0


def test_one_workspace_serves_other_shapes(attn):
    big = attn.dims(64, 2, 256)
    ws = attn.workspace(big)
    for Hq, Hkv, D, fmt in ((64, 2, 256, "bf16"), (4, 4, 64, "e4m3"), (16, 2, 128, "bf16")):
        d = attn.dims(Hq, Hkv, D)
        lens = [900, 3]
        q, cache, table, lens_t, slots, _ = _sequences(attn, d, lens, 16, fmt, 28)
        for _ in range(2):
            out, lse = _run_decode(attn, d, q, cache, table, lens_t, ws)
            _check_decode(attn, d, q, cache, slots, lens, out, lse, 16)


def test_tensors_that_do_not_fit_are_refused_before_a_launch(attn):
    from mxfp4_routed_expert_latentmoe_gb300 import K3MoEError
    d, other = attn.dims(4, 2, 64), attn.dims(4, 2, 128)
    q, cache, table, lens_t, slots, ws = _sequences(attn, d, [20, 5], 16, "e4m3", 30)
    _, k, v = _qkv(2, 4, 2, 64, 31)
    out, lse = torch.full((2, 4, 64), 7.0, device="cuda", dtype=torch.bfloat16), torch.empty(2, 4, device="cuda")
    good = dict(q=q, cache=cache, page_table=table, lens=lens_t, out=out, ws=ws)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:1]), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(page_table=table.long()), dict(page_table=table[:1]), dict(page_table=table[0]),
                dict(page_table=table[:, ::2]), dict(lens=lens_t.cpu()), dict(lens=lens_t[:1]), dict(lens=None),
                dict(out=out.half()), dict(out=out[:, :, :32]), dict(ws=ws.float()), dict(lse=lse.half()),
                dict(lse=lse[:1]), dict(cache=attn.KVCache.empty(other, 2, 16))):
        with pytest.raises(ValueError):
            attn.decode(d, **{**good, **bad})
    with pytest.raises(K3MoEError) as e:
        attn.decode(d, **{**good, "ws": ws[:256]})
    assert e.value.code == 4
    two = torch.tensor([3, 4], device="cuda", dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.kv_write(d, k, v, two.long(), cache, ws)
    with pytest.raises(ValueError):
        attn.kv_write(d, k, v[:1], two, cache, ws)
    with pytest.raises(ValueError):
        attn.kv_read(d, two, cache, out[:, :2], out[:, 2:], ws)  # not dense
    with pytest.raises(K3MoEError) as e:
        attn.kv_write(d, k, v, two, cache, ws[:255])
    assert e.value.code == 4
    w = torch.ones(64, device="cuda")
    freq = attn.rope_frequencies(64)
    args = dict(q=q, k=k, positions=two, inv_freq=freq, q_w=w, k_w=w, q_out=torch.empty_like(out),
                k_out=torch.empty(2, 2, 64, device="cuda", dtype=torch.bfloat16))
    for bad in (dict(positions=two[:1]), dict(inv_freq=freq.float()), dict(inv_freq=None), dict(q_w=w[:32]),
                dict(k_w=w.half()), dict(q_out=out[:1]), dict(k_out=out), dict(k=k[:1])):
        with pytest.raises(ValueError):
            attn.qk_norm_rope(d, **{**args, **bad})
    for wrong in (cache.k[:, :1], cache.k[..., :32], cache.k.to(torch.bfloat16)):
        with pytest.raises(ValueError):
            attn.KVCache(d, wrong, cache.v, cache.k_scale, cache.v_scale)
    with pytest.raises(ValueError):
        attn.KVCache(d, cache.k, cache.v)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and attn.device_status(ws) == 0
    # no tokens, no sequences
    attn.kv_write(d, k[:0], v[:0], two[:0], cache, ws)
    attn.decode(d, q[:0], cache, table[:0], lens_t[:0], out[:0], ws)
