"""The 4-bit (MXFP4) cache on the GPU against its definition: rows written and read back, the append,
the decode attention over it; and the decode attention with sinks, in every format.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of fp16 2^-11, of fp32 2^-24;
of an E2M1 code 1/4, 1/2 or 1 of its scale (below 2, below 4, up to 7 scales)."""
import math

import pytest

from tests import _attn_more_ref as more
from tests import _attn_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16_HALF = 2.0 ** -8
F32_ROWS = 32 * 2.0 ** -24  # fp32 roundings of a normed and rotated element (13 / 2 + 5 + 8 + 3, rounded up)


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


def _randn(*shape, seed, size=1.0):
    return (size * torch.randn(*shape, generator=_gen(seed), device="cuda")).to(torch.bfloat16)


def _close(got, want, tol, what=""):
    off = (got.double().cpu() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off - tol).max()):.3e} over"


def _pools(cache):
    return [x.contiguous().cpu().clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]


def _random(cache, seed):
    """Fills a cache's tensors with random bytes."""
    for i, x in enumerate((cache.k, cache.v, cache.k_scale, cache.v_scale)):
        x.copy_(torch.randint(0, 256, x.shape, generator=_gen(seed + i), device="cuda", dtype=torch.uint8))


def _slots(T, places, seed):
    return torch.randperm(places, generator=_gen(seed), device="cuda")[:T].to(torch.int32)


CACHE_CASES = [  # T, Hkv, D, page, order
    (1, 1, 32, 1, "phtd"), (5, 2, 64, 7, "phtd"), (40, 3, 96, 16, "pthd"), (129, 8, 128, 64, "hptd"),
    (300, 1, 256, 24, "tphd"), (33, 5, 160, 3, "phtd"), (2100, 3, 192, 48, "pthd"), (9, 2, 224, 16, "phtd")]


@pytest.mark.parametrize("T,Hkv,D,page,order", CACHE_CASES)
def test_write_and_read_are_exact(attn, T, Hkv, D, page, order):
    """Written rows equal the definition's bit for bit, all other bytes stay (those behind a row's
    scales too); reading gives code * scale.  Ties, the border of the scales (7 times a power of
    two and next to it), zeros, tiny, huge and non-finite groups among the rows."""
    d = attn.dims(Hkv, Hkv, D, rot_dim=0)
    n_pages = -(-T // page) + 2
    cache = more.empty_cache(attn, d, n_pages, page, "mxfp4", order)
    _random(cache, 5)
    ws = attn.workspace(d)
    x = _randn(T, 2 * Hkv, D, seed=6, size=2.0)
    k, v = x[:, :Hkv], x[:, Hkv:]
    k[0, 0, :32] = 0.0
    v[T // 2, Hkv - 1, :16] *= 1e-38
    v[T - 1, 0] *= 1e37
    v[T - 1, 0, 3] = -3.38e38
    if T > 4:
        k[2, 0, 5], k[2, 0, 6] = float("inf"), float("-inf")
        v[3, 0, 0] = float("nan")
        k[4, 0, 0:16] = torch.tensor([7.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 2, device="cuda")
        v[4, 0, 0:4] = torch.tensor([7.03125, -6.9, 1e-30, -0.0], device="cuda")
        v[4, 0, 4:32] = 0.001
        k[T - 2, 0, :32] = 2.0 ** -126  # (scales stop at 2^-100)
    slots = _slots(T, n_pages * page, 7)
    if T > 1:
        slots[1] = -1
    before = _pools(cache)
    attn.kv_write(d, k, v, slots, cache, ws)
    written = slots >= 0
    pg, at = (slots[written] // page).long().cpu(), (slots[written] % page).long().cpu()
    after = _pools(cache)
    for i, rows in enumerate((k, v)):
        codes, byte = more.quantise_mxfp4(rows[written])
        want, scales = before[i].clone(), before[i + 2].clone()
        got = after[i][pg, :, at]
        nan = (byte == 255).repeat_interleave(16, -1)
        want[pg, :, at] = torch.where(nan, got, codes)  # (a NaN group's codes are any)
        rows_of = scales[pg, :, at]
        rows_of[..., :D // 32] = byte
        scales[pg, :, at] = rows_of
        assert torch.equal(after[i], want) and torch.equal(after[i + 2], scales)
    ko, vo = (torch.full((T, Hkv, D), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    attn.kv_read(d, slots, cache, ko, vo, ws)
    for got, name in ((ko, "k"), (vo, "v")):
        want = more.gather(cache, name, slots[written]).float().to(torch.bfloat16)
        g = got[written].cpu()
        assert ((g == want) | (torch.isnan(g) & torch.isnan(want))).all()
        assert (got[~written] == 0).all()
    assert attn.device_status(ws) == 0


def test_every_scale_is_read(attn):
    """All 256 scale bytes with all codes."""
    d = attn.dims(1, 1, 32, rot_dim=0)
    cache = more.empty_cache(attn, d, 256, 1, "mxfp4")
    _random(cache, 8)
    cache.k[:, 0, 0] = torch.tensor([i * 16 + (15 - i) for i in range(16)], device="cuda", dtype=torch.uint8)
    cache.k_scale[:, 0, 0, 0] = torch.arange(256, device="cuda", dtype=torch.uint8)
    cache.v_scale[:, 0, 0, 0] = torch.arange(256, device="cuda", dtype=torch.uint8).flip(0)
    ws = attn.workspace(d)
    ko, vo = (torch.empty(256, 1, 32, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    slots = torch.arange(256, device="cuda", dtype=torch.int32)
    attn.kv_read(d, slots, cache, ko, vo, ws)
    for got, name in ((ko, "k"), (vo, "v")):
        want = more.gather(cache, name, slots).float().to(torch.bfloat16)
        g = got.cpu()
        assert ((g == want) | (torch.isnan(g) & torch.isnan(want))).all()


def test_slots_outside_the_cache_are_skipped_and_reported(attn):
    d = attn.dims(2, 2, 64, rot_dim=0)
    cache = more.empty_cache(attn, d, 3, 16, "mxfp4")
    _random(cache, 9)
    ws = attn.workspace(d)
    k, v = _randn(4, 2, 64, seed=9), _randn(4, 2, 64, seed=10)
    before = _pools(cache)
    bad = torch.tensor([48, -2, 2 ** 31 - 1, -1], device="cuda", dtype=torch.int32)
    attn.kv_write(d, k, v, bad, cache, ws)
    assert attn.device_status(ws) == attn.DEV_BAD_SLOT
    assert all(torch.equal(a, b) for a, b in zip(_pools(cache), before))
    attn.workspace_init(ws)
    ko, vo = (torch.ones(4, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    attn.kv_read(d, bad, cache, ko, vo, ws)
    assert (ko == 0).all() and (vo == 0).all() and attn.device_status(ws) == attn.DEV_BAD_SLOT


def _half_step(y):
    """Half a step of the codes around the f64 rows y, and their scales."""
    s = more.size_of(more.exponents(y)).repeat_interleave(32, -1)
    z = y.abs() / s
    return s * torch.where(z < 2, 0.25, torch.where(z < 4, 0.5, 1.0)), s


@pytest.mark.parametrize("T,Hq,Hkv,D,R,inter,page", [
    (1, 8, 2, 64, 64, False, 16), (37, 6, 3, 96, 48, True, 5), (40, 6, 3, 96, 48, False, 5), (260, 16, 2, 256, 128, False, 64),
    (64, 12, 4, 128, 128, True, 16), (64, 12, 4, 128, 128, False, 16), (5, 7, 7, 160, 0, False, 7), (70, 4, 1, 192, 32, False, 16),
    (33, 2, 2, 224, 208, False, 8), (3, 1, 1, 32, 16, False, 1), (700, 64, 8, 128, 64, False, 64), (9, 10, 5, 256, 256, False, 4)])
def test_append(attn, T, Hq, Hkv, D, R, inter, page):
    """The fused pass: queries as qk_norm_rope gives them, values as kv_write does (bit for bit), keys
    quantised from their fp32 values: within half a step of the formula's, where the group's scale
    is not next to its border (there the larger one is as right)."""
    d = attn.dims(Hq, Hkv, D, rot_dim=R, rot_interleaved=inter)
    n_pages = -(-T // page) + 1
    cache, plain = (more.empty_cache(attn, d, n_pages, page, "mxfp4") for _ in range(2))
    _random(cache, 11)
    _random(plain, 11)
    ws = attn.workspace(d)
    x = _randn(T, Hq + 2 * Hkv, D, seed=12, size=2.0)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    qw, kw = (1.0 + 0.2 * torch.randn(D, generator=_gen(13 + i), device="cuda") for i in range(2))
    kw[:D // 2] *= 8.0  # groups of a row of different sizes
    pos = torch.randint(0, 100000, (T,), generator=_gen(14), device="cuda", dtype=torch.int32)
    freq = attn.rope_frequencies(R) if R else None
    slots = _slots(T, n_pages * page, 15)
    if T > 2:
        slots[2] = -1
    qo, ko, q1, k1 = (torch.empty(T, h, D, device="cuda", dtype=torch.bfloat16) for h in (Hq, Hkv, Hq, Hkv))
    attn.kv_append(d, q, k, v, pos, slots, freq, qw, kw, cache, qo, ws, k_out=ko)
    attn.qk_norm_rope(d, q, k, pos, freq, qw, kw, q1, k1)
    attn.kv_write(d, k, v, slots, plain, ws)
    assert torch.equal(qo, q1) and torch.equal(ko, k1)
    assert torch.equal(cache.v, plain.v) and torch.equal(cache.v_scale, plain.v_scale)
    assert torch.equal(cache.k_scale[..., D // 32:], plain.k_scale[..., D // 32:])  # never written
    written = slots >= 0
    y, size = ref.norm_rope(k[written], kw, pos[written], freq, 1e-6, inter)
    got = more.gather(cache, "k", slots[written])
    half, s = _half_step(y)
    slack = 4 * F32_ROWS * size.unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
    amax = y.unflatten(-1, (-1, 32)).abs().amax(-1).repeat_interleave(32, -1)
    border = (amax + slack > 7 * s) | (amax - slack <= 3.5 * s)
    _close(got, y, torch.where(border, 2 * s, half) + slack)
    assert border.float().mean() < 0.01
    qo2 = torch.empty_like(qo)
    attn.kv_append(d, q, k, v, pos, slots, freq, qw, kw, plain, qo2, ws)  # without k_out
    assert torch.equal(qo, qo2) and torch.equal(plain.k, cache.k) and torch.equal(plain.k_scale, cache.k_scale)
    assert attn.device_status(ws) == 0


def test_append_of_non_finite_keys(attn):
    """A NaN makes its whole row NaN (the norm), and no other."""
    d = attn.dims(2, 2, 64)
    cache = more.empty_cache(attn, d, 2, 8, "mxfp4")
    ws = attn.workspace(d)
    x = _randn(3, 6, 64, seed=16)
    x[1, 2, 40] = float("nan")
    slots = torch.tensor([3, 9, 0], device="cuda", dtype=torch.int32)
    w, pos = torch.ones(64, device="cuda"), torch.arange(3, device="cuda", dtype=torch.int32)
    qo = torch.empty(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    attn.kv_append(d, x[:, :2], x[:, 2:4], x[:, 4:], pos, slots, attn.rope_frequencies(64), w, w, cache, qo, ws)
    k = more.gather(cache, "k", slots)
    assert torch.isnan(k[1, 0]).all() and torch.isfinite(k[0]).all() and torch.isfinite(k[1, 1]).all()
    assert torch.isfinite(more.gather(cache, "v", slots)).all()


# ------------------------------------------------------------------------------ decode
def _run(attn, s, q, sinks=0, table=None):
    out = torch.full(q.shape, 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    attn.decode(s.d, q, s.cache, s.table if table is None else table, s.lens_t, out, s.ws, lse=lse, sinks=sinks)
    return out, lse


def _check(s, q, out, lse, sinks=0):
    """As the tests of the other formats: weights rounded once (bf16's half step covers fp16's) with the
    logits' fp32 error in their exponents, the result rounded to bf16.

    4 bits hold many zeros, beside which other tokens of the smallest weights show: a weight times its
    row's largest scale is rounded to fp16 with 2^15 for the largest of all tokens, then times its
    group's factor, so that two half steps of 2^-25 at most are lost below fp16's normal numbers, 2^-39
    of that largest, times a code of 6 at most; the largest scale is at most a 3.5th of the row's largest
    value: 2 * 2^-39 max_t(p_t max|v_t|) a token, 2^-38."""
    for b, n in enumerate(s.lens):
        which = more.seen(n, s.d.window, sinks)
        k, v = s.rows(b, which)
        o, z, mean_abs, slack = ref.decode(q[b].double().cpu(), k, v, s.d.softmax_scale)
        count = len(which)
        tol = BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + (64 + count / 8) * 2.0 ** -24)
        if count and s.cache.k.dtype == torch.uint8:
            j = torch.arange(s.d.n_heads) // (s.d.n_heads // s.d.n_kv_heads)
            p = torch.softmax(s.d.softmax_scale * torch.einsum("hd,nhd->hn", q[b].double().cpu(), k[:, j]), -1)
            tol = tol + count * 2.0 ** -38 * (p * v[:, j].abs().amax(-1).t()).amax(-1)[:, None]
        _close(out[b], o, tol, f"sequence {b} of {n}")
        if count == 0:
            assert (lse[b] == -torch.inf).all()
        else:
            _close(lse[b], z, slack + (64 + count / 8) * 2.0 ** -24 + 2.0 ** -22 * z.abs(), f"lse {b}")


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 0, 127, 129, 300, 1000]
DECODE_CASES = [  # Hq, Hkv, D, page, window, sinks, order, lens
    (1, 1, 32, 1, 0, 0, "phtd", [1]), (8, 8, 64, 16, 0, 0, "phtd", LENS), (8, 1, 128, 16, 0, 0, "phtd", LENS),
    (64, 8, 128, 64, 0, 3, "phtd", [1, 700, 0, 5000]), (6, 2, 96, 7, 0, 0, "pthd", LENS),
    (24, 2, 256, 24, 0, 0, "phtd", LENS), (36, 3, 192, 24, 100, 4, "hptd", LENS), (5, 1, 160, 3, 17, 1, "tphd", LENS),
    (16, 1, 64, 128, 0, 0, "phtd", [4097]), (34, 2, 128, 16, 64, 64, "phtd", LENS), (40, 1, 256, 32, 0, 0, "phtd", [77, 513]),
    (7, 7, 32, 16, 1, 1, "phtd", LENS), (2, 1, 128, 32, 0, 0, "phtd", [70001]), (9, 3, 224, 5, 64, 130, "phtd", LENS),
    (8, 2, 128, 64, 0, 0, "phtd", [0, 0, 0]), (16, 8, 64, 16, 0, 0, "phtd", [3 * i % 97 for i in range(400)]),
    (100, 1, 64, 16, 30, 2, "phtd", [200, 0, 1])]


@pytest.mark.parametrize("Hq,Hkv,D,page,window,sinks,order,lens", DECODE_CASES,
                         ids=[f"{c[0]}x{c[1]}x{c[2]}-p{c[3]}-w{c[4]}-s{c[5]}-{c[6]}-{len(c[7])}of{max(c[7])}"
                              for c in DECODE_CASES])
def test_decode(attn, Hq, Hkv, D, page, window, sinks, order, lens):
    d = attn.dims(Hq, Hkv, D, window=window)
    s = more.Sequences(attn, d, lens, page, "mxfp4", 20, order=order)
    q = s.queries(len(lens))
    out, lse = _run(attn, s, q, sinks)
    _check(s, q, out, lse, sinks)
    out2 = torch.empty_like(out)  # again (the workspace is left ready), without lse: the same bits
    attn.decode(d, q, s.cache, s.table, s.lens_t, out2, s.ws, sinks=sinks)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    assert attn.device_status(s.ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 40), (40, 1), (32, 32), (100, 4), (64, 500), (128, 2000), (500, 31)])
@pytest.mark.parametrize("page", [5, 32, 64])
def test_decode_with_sinks(attn, fmt, window, sinks, page):
    """Sinks that end inside a tile, a page, the window, behind the sequence; the token after the last
    of them on the page of the same place, on the same page, or on any other."""
    for Hq, Hkv, D in ((8, 2, 128), (24, 2, 64)):
        d = attn.dims(Hq, Hkv, D, window=window)
        lens = [0, 1, 33, 64 + window, 128 + window, 132, 997, 1060, 64 * 20 + 30, 4000]
        s = more.Sequences(attn, d, lens, page, fmt, 30, room=50)
        q = s.queries(len(lens))
        out, lse = _run(attn, s, q, sinks)
        _check(s, q, out, lse, sinks)
        assert attn.device_status(s.ws) == 0
        s0 = [x.clone() for x in _run(attn, s, q, 0)]
        _check(s, q, *s0)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
def test_sinks_on_pages_that_repeat(attn, fmt):
    """A table that has one page everywhere: sinks and window look alike, and are told apart by where
    they lie on the page."""
    page, D, Hkv = 64, 64, 1
    k, v = _randn(page, Hkv, D, seed=33), _randn(page, Hkv, D, seed=34)
    for window, sinks in ((64, 20), (70, 20), (30, 34), (128, 40), (40, 40)):
        d = attn.dims(4, Hkv, D, window=window, rot_dim=0)
        s = more.Sequences(attn, d, [page], page, fmt, 35, k=k, v=v)
        n = 1000
        s.table = s.table[:, :1].expand(1, 16).contiguous()
        s.slots = [s.slots[0][torch.arange(n) % page]]
        s.lens, s.lens_t = [n], torch.tensor([n], device="cuda", dtype=torch.int32)
        q = s.queries(1)
        _check(s, q, *_run(attn, s, q, sinks), sinks)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 1, 64), (24, 2, 96), (60, 3, 128), (36, 3, 192), (24, 2, 256)])
def test_decode_of_many_query_heads_with_room_in_the_page_table(attn, Hq, Hkv, D):
    d = attn.dims(Hq, Hkv, D)
    for lens in (LENS, [0, 500, 2300]):
        s = more.Sequences(attn, d, lens, 16, "mxfp4", 28)
        q = s.queries(len(lens))
        wide = torch.full((len(lens), 2 ** 16), -1, device="cuda", dtype=torch.int32)
        wide[:, :s.table.shape[1]] = s.table
        for t in (s.table, wide, s.table):
            out, lse = _run(attn, s, q, table=t)
            _check(s, q, out, lse)
        assert attn.device_status(s.ws) == 0


def test_decode_sharp_logits_and_values_of_many_sizes(attn):
    d = attn.dims(16, 2, 128)
    for q_size, spread in ((60.0, 0.5), (2.0, 4.0), (20.0, 4.0), (1e6, 0.5)):
        s = more.Sequences(attn, d, [3, 70, 900], 16, "mxfp4", 21, spread=spread)
        q = s.queries(3, q_size)
        out, lse = _run(attn, s, q)
        if q_size < 1e3:
            _check(s, q, out, lse)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_decode_of_groups_of_many_sizes(attn):
    """Groups of a row that are up to 2^20 apart, other ones in each token: the small ones keep their
    precision (2^25 apart they count as zeros, no more than half of fp32's step of the largest)."""
    d = attn.dims(4, 1, 128, rot_dim=0)
    n = 200
    size = torch.randint(0, 21, (n, 1, 4), generator=_gen(40), device="cuda").float().exp2()
    v = (_randn(n, 1, 128, seed=41).float() * size.repeat_interleave(32, -1)).to(torch.bfloat16)
    s = more.Sequences(attn, d, [n], 16, "mxfp4", 42, v=v)
    q = s.queries(1)
    out, lse = _run(attn, s, q)
    k, vv = s.rows(0, list(range(n)))
    o, z, mean_abs, slack = ref.decode(q[0].double().cpu(), k, vv, d.softmax_scale)
    _close(out[0], o, BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + 2.0 ** -18))
    far = v.clone()
    far[..., :32] *= 2.0 ** 60
    s = more.Sequences(attn, d, [n], 16, "mxfp4", 42, v=far)
    out, _ = _run(attn, s, q)
    _, vv = s.rows(0, list(range(n)))
    o, z, mean_abs, slack = ref.decode(q[0].double().cpu(), k, vv, d.softmax_scale)
    tol = BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + 2.0 ** -18)
    _close(out[0, :, :32], o[:, :32], tol[:, :32])
    largest = vv.abs().amax()
    assert ((out[0, :, 32:].double().cpu() - o[:, 32:]).abs() <= tol[:, 32:] + 2.0 ** -24 * largest).all()


def test_decode_of_rows_with_nan_groups(attn):
    """A key's NaN takes the logits of its head; a value's the 32 dims of its group alone."""
    d = attn.dims(4, 2, 64)
    s = more.Sequences(attn, d, [40, 40], 16, "mxfp4", 22)
    slot = int(s.slots[0][7])
    s.cache.k_scale[slot // 16, 0, slot % 16, 1] = 255
    slot = int(s.slots[1][39])
    s.cache.v_scale[slot // 16, 1, slot % 16, 0] = 255
    q = s.queries(2)
    out, lse = _run(attn, s, q)
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all() and torch.isfinite(out[0, 2:]).all()
    assert torch.isnan(out[1, 2:, :32]).all() and torch.isfinite(out[1, 2:, 32:]).all()
    assert torch.isfinite(out[1, :2]).all() and torch.isfinite(lse[1]).all()


def test_decode_bad_pages_are_left_out_and_reported(attn):
    d = attn.dims(8, 2, 128, window=70)
    s = more.Sequences(attn, d, [200, 64], 16, "mxfp4", 24)
    s.table[0, 0] = -3  # the sinks' page
    s.table[0, 10] = s.cache.n_pages
    s.table[0, 5] = -9  # between sinks and window: not read
    q = s.queries(2)
    out, lse = _run(attn, s, q, 20)
    assert attn.device_status(s.ws) == attn.DEV_BAD_PAGE
    keep = [t for t in more.seen(200, 70, 20) if t // 16 not in (0, 10)]
    k, v = s.rows(0, keep)
    o, z, mean_abs, slack = ref.decode(q[0].double().cpu(), k, v, d.softmax_scale)
    _close(out[0], o, BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + 90 * 2.0 ** -24))


@pytest.mark.parametrize("D", [32, 96, 160, 224])
def test_a_padded_head_dim_is_that_of_heads_with_zeros(attn, D):
    """The same bits, whatever an earlier call (of NaN rows) has left in shared memory and whatever
    lies in the bytes behind a row's scales."""
    wide, Hkv, G = -(-D // 64) * 64, 2, 4
    lens = [300, 1, 77, 0, 33, 2500]
    T = sum(lens)
    k, v = (torch.zeros(T, Hkv, wide, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k[..., :D], v[..., :D] = _randn(T, Hkv, D, seed=41), _randn(T, Hkv, D, seed=42)
    dw, d = attn.dims(Hkv * G, Hkv, wide, rot_dim=0, softmax_scale=D ** -0.5), attn.dims(Hkv * G, Hkv, D, rot_dim=0)
    q = torch.zeros(len(lens), Hkv * G, wide, device="cuda", dtype=torch.bfloat16)
    q[..., :D] = _randn(len(lens), Hkv * G, D, seed=43)
    sw = more.Sequences(attn, dw, lens, 16, "mxfp4", 44, k=k, v=v)
    want, lse = _run(attn, sw, q)
    nan = more.Sequences(attn, dw, lens, 16, "mxfp4", 44, k=torch.full_like(k, float("nan")), v=v)
    s = more.Sequences(attn, d, lens, 16, "mxfp4", 44, k=k[..., :D].contiguous(), v=v[..., :D].contiguous())
    for _ in range(10):
        _run(attn, nan, q)
        out, lse2 = _run(attn, s, q[..., :D].contiguous())
        assert torch.equal(out, want[..., :D]) and torch.equal(lse2, lse)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
def test_windows_and_sinks_of_the_longest_sequences(attn, fmt):
    """Lengths up to 2^31 - 2 over pages that repeat: the window's tokens and the sinks, as a short
    sequence of the same rows gives them."""
    page, wide, D, G = 49981, 42966, 64, 4
    n = page * wide
    k, v = (_randn(2 * page, 1, D, seed=x) for x in (51, 52))
    q = _randn(2, G, D, seed=50)
    for window, sinks in ((100, 7), (257, 300)):
        d = attn.dims(G, 1, D, rot_dim=0, window=window)
        cache = attn.KVCache.empty(d, 2, page, fmt)
        ws = attn.workspace(d)
        attn.kv_write(d, k, v, torch.arange(2 * page, device="cuda", dtype=torch.int32), cache, ws)
        table = torch.zeros(2, wide, device="cuda", dtype=torch.int32)
        table[:, -1] = 1
        got = []
        for t, lens in ((table, [n, n - 30]), (table[:, -2:].contiguous(), [2 * page, 2 * page - 30])):
            out, lse = torch.zeros(2, G, D, device="cuda", dtype=torch.bfloat16), torch.zeros(2, G, device="cuda")
            attn.decode(d, q, cache, t, torch.tensor(lens, device="cuda", dtype=torch.int32), out, ws, lse=lse, sinks=sinks)
            got.append((out, lse))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert torch.isfinite(got[0][1]).all() and attn.device_status(ws) == 0


@pytest.mark.parametrize("log_n,below", [(12, 9.0), (22, 18.0), (26, 22.5)])
def test_decode_of_many_tokens_of_small_weight_beside_a_large_one(attn, log_n, below):
    """One token of weight 1 and 2^log_n - 1 of weight e^-below each, whose sum counts (pages repeat).
    The values 4, -4, 0 and 2, 1 and the key 12 are exact in E2M1."""
    page, D, n = 4096, 64, 1 << log_n
    d = attn.dims(1, 1, D, rot_dim=0)
    cache = attn.KVCache.empty(d, 2, page, "mxfp4")
    ws = attn.workspace(d)
    q = torch.zeros(1, 1, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = below / 12 * math.sqrt(D)
    k = torch.zeros(2 * page, 1, D, device="cuda", dtype=torch.bfloat16)
    k[0, 0, 0] = 12.0
    v = torch.full((2 * page, 1, D), 2.0, device="cuda", dtype=torch.bfloat16)
    v[0, 0, 0::4], v[0, 0, 1::2], v[0, 0, 2::4] = 4.0, -4.0, 0.0
    v[page + 1:, 0, 5::7] = v[1:page, 0, 5::7] = 2.0
    attn.kv_write(d, k, v, torch.arange(2 * page, device="cuda", dtype=torch.int32), cache, ws)
    table = torch.ones(1, n // page, device="cuda", dtype=torch.int32)
    table[0, 0] = 0
    out, lse = torch.zeros(1, 1, D, device="cuda", dtype=torch.bfloat16), torch.zeros(1, 1, device="cuda")
    attn.decode(d, q, cache, table, torch.tensor([n], device="cuda", dtype=torch.int32), out, ws, lse=lse)
    rest = (n - 1) * math.exp(-below)
    first, other = v[0, 0].double().cpu(), v[1, 0].double().cpu()
    want, mean_abs = (first + rest * other) / (1 + rest), (first.abs() + rest * other.abs()) / (1 + rest)
    off = (out[0, 0].double().cpu() - want).abs()
    assert (off <= BF16_HALF * want.abs() + mean_abs * (BF16_HALF + 2.0 ** -10)).all(), (out[0, 0, :4], want[:4])
    assert abs(float(lse) - (below + math.log1p(rest))) <= 2.0 ** -10


def test_a_cache_past_32_bits(attn):
    """Pages whose bytes lie past 2^32 (only the used ones are filled)."""
    d = attn.dims(8, 4, 128)
    page, n_pages = 256, 70000  # 4.6e9 bytes of codes
    k, v = (torch.empty(n_pages, 4, page, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(n_pages, 4, page, 4, device="cuda", dtype=torch.uint8) for _ in range(2))
    cache = attn.KVCache(d, k, v, ks, vs)
    ws, n = attn.workspace(d), 600
    table = torch.tensor([[n_pages - 1, 5, n_pages - 2]], device="cuda", dtype=torch.int32)
    t = torch.arange(n, device="cuda")
    slots = (table[0].long()[t // page] * page + t % page).to(torch.int32)
    kk, vv, q = _randn(n, 4, 128, seed=25), _randn(n, 4, 128, seed=26), _randn(1, 8, 128, seed=27)
    attn.kv_write(d, kk, vv, slots, cache, ws)
    out = torch.empty(1, 8, 128, device="cuda", dtype=torch.bfloat16)
    attn.decode(d, q, cache, table, torch.tensor([n], device="cuda", dtype=torch.int32), out, ws)
    kr, vr = (torch.empty(n, 4, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    attn.kv_read(d, slots, cache, kr, vr, ws)
    rows = [more.values_of(*more.quantise_mxfp4(x)) for x in (kk, vv)]
    assert torch.equal(kr.double().cpu(), rows[0]) and torch.equal(vr.double().cpu(), rows[1])
    o, z, mean_abs, slack = ref.decode(q[0].double().cpu(), *rows, d.softmax_scale)
    _close(out[0], o, BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + 139 * 2.0 ** -24))
    assert attn.device_status(ws) == 0


def test_a_captured_step_replays_with_new_lengths(attn):
    """Append and decode (window and sinks) as a graph, replayed as the sequences grow."""
    d = attn.dims(16, 4, 128, window=64)
    s = more.Sequences(attn, d, [130, 1, 77], 16, "mxfp4", 26, room=4)
    s.table[:, :] = torch.where(s.table < 0, s.table[:, :1], s.table)
    x = _randn(3, 24, 128, seed=27)
    q, k, v = x[:, :16], x[:, 16:20], x[:, 20:]
    w, freq = torch.ones(128, device="cuda"), attn.rope_frequencies(128)
    pos = s.lens_t.clone()
    lens = s.lens_t + 1
    slots = s.table[torch.arange(3, device="cuda"), (pos // 16).long()] * 16 + pos % 16
    qo, out = (torch.empty(3, 16, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    lse = torch.empty(3, 16, device="cuda")

    def step():
        attn.kv_append(d, q, k, v, pos, slots, freq, w, w, s.cache, qo, s.ws)
        attn.decode(d, qo, s.cache, s.table, lens, out, s.ws, lse=lse, sinks=4)

    step()
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    lens.copy_(torch.tensor([64, 2, 0], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    eager = torch.empty_like(out)
    attn.decode(d, qo, s.cache, s.table, lens, eager, s.ws, sinks=4)
    assert torch.equal(out, eager) and (out[2] == 0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(out)
    attn.decode(d, qo, s.cache, s.table, lens, other, s.ws, stream=side, sinks=4)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, eager) and attn.device_status(s.ws) == 0


def test_one_workspace_serves_all_formats(attn):
    ws = attn.workspace(attn.dims(64, 2, 256))
    for Hq, Hkv, D, fmt in ((64, 2, 256, "mxfp4"), (4, 4, 64, "e4m3"), (16, 2, 128, "mxfp4"), (16, 2, 128, "bf16")):
        d = attn.dims(Hq, Hkv, D)
        s = more.Sequences(attn, d, [900, 3], 16, fmt, 28)
        s.ws = ws
        q = s.queries(2)
        for _ in range(2):
            _check(s, q, *_run(attn, s, q))
