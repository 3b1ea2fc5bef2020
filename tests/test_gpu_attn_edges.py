"""The decode attention at its edges: head dims that its tiles pad, lengths next to 2^31, short
sequences at the teams' borders, weights and logits of extreme sizes."""
import math

import pytest

from tests import _attn_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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


def _call(attn, d, q, k, v, lens, page, fmt):
    """Decode over dense rows k, v [sum of lens, Hkv, D] bf16: (out, lse)."""
    pages = [-(-n // page) for n in lens]
    cache = attn.KVCache.empty(d, max(1, sum(pages)), page, fmt)
    table = torch.zeros(len(lens), max(1, max(pages)), device="cuda", dtype=torch.int32)
    slots, first = [], 0
    for b, (n, m) in enumerate(zip(lens, pages)):
        table[b, :m] = torch.arange(first, first + m, device="cuda", dtype=torch.int32)
        slots.append(torch.arange(first * page, first * page + n, device="cuda", dtype=torch.int32))
        first += m
    ws = attn.workspace(d)
    attn.kv_write(d, k, v, torch.cat(slots), cache, ws)
    out = torch.full((len(lens), d.n_heads, d.head_dim), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((len(lens), d.n_heads), 7.0, device="cuda")

    def call():
        attn.decode(d, q, cache, table, torch.tensor(lens, device="cuda", dtype=torch.int32), out, ws, lse=lse)
        return out, lse
    call()
    assert attn.device_status(ws) == 0
    return call


def _cached(x, fmt):
    """Rows [n, H, D] bf16 as the cache holds them, in f64 on the CPU."""
    if fmt == "bf16":
        return x.double().cpu()
    codes, scale = ref.quantise_f32(x)
    return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [16, 32, 48, 80, 112, 144, 176, 208, 240])
def test_decode_of_a_padded_head_dim_is_that_of_heads_with_zeros(attn, D, fmt):
    """Rows of D values and the same rows with zeros up to the tile's width take the same products
    and sums: the same bits, every time, whatever an earlier call (here one of NaN rows) has left
    in shared memory."""
    wide, Hkv, G = -(-D // 64) * 64, 2, 4
    lens = [300, 1, 77, 0, 33, 2500]
    T = sum(lens)
    q, k, v = (torch.zeros(n, h, wide, device="cuda", dtype=torch.bfloat16) for n, h in
               ((len(lens), Hkv * G), (T, Hkv), (T, Hkv)))
    for i, x in enumerate((q, k, v)):
        x[..., :D] = torch.randn(x[..., :D].shape, generator=_gen(40 + i), device="cuda").to(torch.bfloat16)
    dw = attn.dims(Hkv * G, Hkv, wide, rot_dim=0, softmax_scale=D ** -0.5)
    d = attn.dims(Hkv * G, Hkv, D, rot_dim=0)
    want, lse = (x.clone() for x in _call(attn, dw, q, k, v, lens, 16, fmt)())
    assert torch.isfinite(want).all()
    nan = _call(attn, dw, q, torch.full_like(k, float("nan")), torch.full_like(v, float("nan")), lens, 16, fmt)
    call = _call(attn, d, q[..., :D].contiguous(), k[..., :D].contiguous(), v[..., :D].contiguous(), lens, 16, fmt)
    for _ in range(30):
        nan()
        out, lse2 = call()
        assert torch.equal(out, want[..., :D]) and torch.equal(lse2, lse)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [1, 16])
def test_decode_of_windows_at_the_end_of_the_longest_sequences(attn, G, fmt):
    """Lengths up to 2^31 - 2, over pages that repeat: the window's tokens alone, whose last tile
    reaches past 2^31, as a short sequence of the same rows gives them."""
    page, wide, D = 49981, 42966, 64
    n = page * wide
    assert n == 2 ** 31 - 2
    q = torch.randn(3, G, D, generator=_gen(50), device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(2 * page, 1, D, generator=_gen(s), device="cuda").to(torch.bfloat16) for s in (51, 52))
    for window in (100, 1, 257):
        d = attn.dims(G, 1, D, rot_dim=0, window=window)
        cache = attn.KVCache.empty(d, 2, page, fmt)
        ws = attn.workspace(d)
        attn.kv_write(d, k, v, torch.arange(2 * page, device="cuda", dtype=torch.int32), cache, ws)
        table = torch.zeros(3, wide, device="cuda", dtype=torch.int32)
        table[:, -1] = 1
        table[2, -1] = 0
        lens = torch.tensor([n, n - 30, n], device="cuda", dtype=torch.int32)
        out, lse = torch.zeros(3, G, D, device="cuda", dtype=torch.bfloat16), torch.zeros(3, G, device="cuda")
        attn.decode(d, q, cache, table, lens, out, ws, lse=lse)
        short = torch.tensor([[0, 1], [0, 1], [0, 0]], device="cuda", dtype=torch.int32)
        out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
        attn.decode(d, q, cache, short, lens - (n - 2 * page), out2, ws, lse=lse2)
        assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.isfinite(lse).all()
        assert attn.device_status(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("log_n,below", [(12, 9.0), (22, 18.0), (26, 22.5)])
def test_decode_of_many_tokens_of_small_weight_beside_a_large_one(attn, log_n, below, fmt):
    """One token of weight 1 and 2^log_n - 1 of weight e^-below each, whose sum counts: 0.01 to 0.5,
    2^-13 to 2^-32.5 each.  (Pages repeat.)  A weight's rounding takes half a step of bf16 at most
    (2^-8), the result's another; the fp32 sums (a lane's are of 2^26 / 152 / 64 terms at most) and
    powers of two stay below 2^-10."""
    page, D, n = 4096, 64, 1 << log_n
    d = attn.dims(1, 1, D, rot_dim=0)
    cache = attn.KVCache.empty(d, 2, page, fmt)
    ws = attn.workspace(d)
    q = torch.zeros(1, 1, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = below / 12 * math.sqrt(D)
    k = torch.zeros(2 * page, 1, D, device="cuda", dtype=torch.bfloat16)
    k[0, 0, 0] = 12.0
    v = torch.ones(2 * page, 1, D, device="cuda", dtype=torch.bfloat16)
    v[0, 0, 1::2] = -1.0
    v[0, 0, 2::4] = 0.0
    assert float(q[0, 0, 0]) * 12 == below * math.sqrt(D)
    attn.kv_write(d, k, v, torch.arange(2 * page, device="cuda", dtype=torch.int32), cache, ws)
    table = torch.ones(1, n // page, device="cuda", dtype=torch.int32)
    table[0, 0] = 0
    out, lse = torch.zeros(1, 1, D, device="cuda", dtype=torch.bfloat16), torch.zeros(1, 1, device="cuda")
    attn.decode(d, q, cache, table, torch.tensor([n], device="cuda", dtype=torch.int32), out, ws, lse=lse)
    rest = (n - 1) * math.exp(-below)
    first, other = _cached(v[:2], fmt)[:, 0]
    want = (first + rest * other) / (1 + rest)
    mean_abs = (first.abs() + rest * other.abs()) / (1 + rest)
    off = (out[0, 0].double().cpu() - want).abs()
    assert (off <= 2.0 ** -8 * want.abs() + mean_abs * (2.0 ** -8 + 2.0 ** -10)).all(), (out[0, 0, :4], want[:4])
    assert abs(float(lse) - (below + math.log1p(rest))) <= 2.0 ** -10


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D", [(4, 64), (12, 128)])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e7, 1e10, 1e13])
def test_decode_of_logits_of_any_finite_size(attn, size, G, D, fmt):
    """Logits so large that one token takes all (the next one is further off than twice their fp32
    error): the result is that token's value, rounded once to bf16, but for the powers of two and
    quotients of its scale (below 2^-16)."""
    lens, Hkv = [1, 70, 33, 0, 1], 2
    T = sum(lens)
    d = attn.dims(Hkv * G, Hkv, D, rot_dim=0)
    q = (math.sqrt(size) * torch.randn(len(lens), Hkv * G, D, generator=_gen(60), device="cuda")).to(torch.bfloat16)
    k = (math.sqrt(size) * torch.randn(T, Hkv, D, generator=_gen(61), device="cuda")).to(torch.bfloat16)
    v = torch.exp(2 * torch.randn(T, Hkv, 1, generator=_gen(62), device="cuda"))
    v = (v * torch.randn(T, Hkv, D, generator=_gen(63), device="cuda")).to(torch.bfloat16)
    out, lse = _call(attn, d, q, k, v, lens, 16, fmt)()
    kc, vc = _cached(k, fmt), _cached(v, fmt)
    at = seen = 0
    for b, n in enumerate(lens):
        rows, vals = kc[at:at + n], vc[at:at + n]
        at += n
        if n == 0:
            continue
        _, z, _, slack = ref.decode(q[b].double().cpu(), rows, vals, d.softmax_scale)
        for h in range(Hkv * G):
            logits = d.softmax_scale * (rows[:, h // G] @ q[b, h].double().cpu())
            top, where = logits.max(0)
            rest = logits[torch.arange(n) != where]
            if n > 1 and float(top - rest.max()) < 2 * float(slack[h]) + 40:
                continue
            seen += 1
            want = vals[where, h // G]
            off = (out[b, h].double().cpu() - want).abs()
            assert (off <= (2.0 ** -8 + 2.0 ** -16) * want.abs()).all(), (size, b, h)
            assert abs(float(lse[b, h]) - float(z[h])) <= float(slack[h]) + 2.0 ** -22 * abs(float(z[h])) + 2.0 ** -18
    assert seen >= 2 * Hkv * G
