"""Prefill over values that are infinite or NaN, and over finite ones whose sums leave fp32's range on the
way: they show in the tokens and dims that see them, nowhere else, and cost no more than those tokens' share."""
import math

import pytest

from tests import _attn_more_ref as more
from tests import _attn_ref as ref
from tests.test_gpu_attn_prefill import BF16_HALF, FORMATS, Call

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def attn():
    import __graft_entry__ as g
    g.build()
    from mxfp4_routed_expert_latentmoe_gb300 import attn as mod
    torch.cuda.set_device(0)
    return mod


def _spoil(c, b, t, head, what):
    """A value of token t of sequence b, key head `head`: of dim 5 ("dim"; MXFP4 scales have 32 dims each), or all."""
    s, cache = c.s, c.s.cache
    pg, at = int(s.slots[b][t] // s.page), int(s.slots[b][t] % s.page)
    if cache.v.dtype == torch.bfloat16:
        cache.v[pg, head, at, 5 if what == "dim" else slice(None)] = math.inf if what == "dim" else math.nan
    elif cache.v.dtype == torch.uint8:
        cache.v_scale[pg, head, at, 0 if what == "dim" else slice(0, c.d.head_dim // 32)] = 255
    elif what == "dim":
        cache.v.view(torch.uint8)[pg, head, at, 5] = 0xFF  # the code of -NaN
    else:
        cache.v_scale[pg, head, at] = math.inf


def _check(c, most_rows=40, every=()):
    """Every sequence at some of its new tokens: what sees a value that is not finite is not finite, the rest
    as the other tests have it."""
    d, row = c.d, c.before
    out, lse, q = c.out.double().cpu(), c.lse.double().cpu(), c.q.double().cpu()
    for b, (new, n) in enumerate(c.sizes):
        k, v = c.s.rows(b, list(range(n)))
        some = set(range(0, new, max(1, new // most_rows))) | {new - 1} | {i for i in every if 0 <= i < new}
        for i in sorted(some) if new else ():
            which = more.seen(n, d.window, c.sinks, n - new + i)
            vv = v[which]
            bad = ~torch.isfinite(vv).all(0)[torch.arange(d.n_heads) // (d.n_heads // d.n_kv_heads)]
            assert torch.equal(~torch.isfinite(out[row + i]), bad), f"sequence {b} of {new} in {n}, token {i}"
            o, z, mean_abs, slack = ref.decode(q[row + i], k[which], torch.where(torch.isfinite(vv), vv, 0), d.softmax_scale)
            count = len(which)
            tiny = 2.0 ** -125 * count * torch.where(torch.isfinite(vv), vv, 0).abs().amax()
            tol = tiny + BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + (64 + count / 8) * 2.0 ** -24)
            off = (out[row + i] - o).abs()
            assert ((off <= tol) | bad).all(), f"sequence {b} of {new} in {n}, token {i}"
            bound = slack + (64 + count / 8) * 2.0 ** -24 + 2.0 ** -22 * z.abs()
            assert ((lse[row + i] - z).abs() <= bound).all(), f"lse: sequence {b}, token {i}"
        row += new
    assert c.attn.device_status(c.ws) == 0


# Hq, Hkv, D, page, window, sinks
SHAPES = [(8, 1, 128, 16, 0, 0), (4, 4, 64, 16, 0, 0), (16, 2, 96, 7, 0, 0), (24, 2, 256, 24, 0, 0), (6, 2, 192, 16, 100, 4),
          (8, 2, 128, 5, 64, 40), (2, 2, 64, 16, 300, 2), (300, 1, 64, 16, 50, 0), (5, 1, 160, 3, 17, 1)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,D,page,window,sinks", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_values_that_are_not_finite(attn, Hq, Hkv, D, page, window, sinks, fmt):
    """At the ends, at the sinks', the window's and the tiles' borders, in the middle."""
    sizes = [(200, 200), (33, 900), (1, 5), (290, 700), (7, 9000)]
    for what in ("dim", "all"):
        c = Call(attn, sizes, page, fmt, Hq, Hkv, D, window, sinks, before=2, behind=3)
        for b, t in ((0, 0), (0, 131), (0, 199), (1, 870), (1, 899), (3, 3), (3, 411), (3, 530), (4, 8997), (4, 20)):
            _spoil(c, b, t, (b + t) % Hkv, what)
        c.run()
        _check(c, 20, (130, 131, 132, 199, 3, 30, 120, 121))
        c.check_same()


def test_head_dims_of_any_multiple_of_16(attn):
    for D in (16, 48, 80, 112, 144, 176, 208, 240):
        c = Call(attn, [(60, 333)], 16, "bf16", 6, 2, D)
        _spoil(c, 0, 300, 1, "dim")
        _spoil(c, 0, 320, 0, "all")
        _check(c.run(), 60)


def _rising(attn, fmt, spoilt, D=64, H=2):
    """All keys the same but for 20 behind the first 128 with a logit that is 7 (in powers of two; in 4 bits 6)
    higher, values of up to 3e36: the maximum stays the first tile's, and 20 weights of 2^6 or 2^7 times some 2e36
    leave fp32's range; with weights of 1 at most they do not."""
    n, G = 400, 3
    k, v = torch.zeros(n, H, D, device="cuda"), torch.zeros(n, H, D, device="cuda")
    k[128:148, :, 0] = 7.0
    v[:] = 3e36 * (1 + torch.arange(n, device="cuda") % 3)[:, None, None] / 3
    v[:, :, 33:] *= 1e-30
    c = Call(attn, [(40, n)], 16, fmt, G * H, H, D, k=k.to(torch.bfloat16), v=v.to(torch.bfloat16), scale=math.log(2))
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = 1.0
    for t in spoilt:
        _spoil(c, 0, t, 1, "dim")
    return c.run()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("spoilt", [(), (7,), (380,), (7, 399)])
def test_sums_that_leave_fp32_on_the_way(attn, fmt, spoilt):
    """With and without a value that accounts for some of the dims."""
    _check(_rising(attn, fmt, spoilt), 40)


def test_an_infinity_is_no_nan_for_a_hidden_value(attn):
    """Infinities that a token sees stay infinities, whatever keys it does not see hold in the same dims."""
    for window in (0, 90):
        c = Call(attn, [(200, 200)], 16, "bf16", 8, 1, 128, window)
        pg, at = (c.s.slots[0] // 16).long(), (c.s.slots[0] % 16).long()
        c.s.cache.v[pg[100], 0, at[100], 5] = math.inf
        c.s.cache.v[pg[100], 0, at[100], 6] = -math.inf
        c.s.cache.v[pg[150], 0, at[150], 5:8] = math.nan
        c.s.cache.v[pg[199], 0, at[199], 5] = -math.inf
        c.run()
        _check(c, 200)
        out = c.out.float().cpu()
        assert (out[100:150, :, 5] == math.inf).all() and (out[100:150, :, 6] == -math.inf).all()
        assert torch.isnan(out[150:199 if window == 0 else 190, :, 5:8]).all() and torch.isfinite(out[:100]).all()


@pytest.mark.parametrize("where", [[0], range(4000)], ids=["first", "all"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_what_a_value_costs(attn, fmt, where):
    """NaN that all tokens see, in the first token or all, cost them a look (hundreds of times the call, were they
    formed again one by one)."""
    c = Call(attn, [(4000, 4000)], 64, fmt, 32, 4, 128)
    ms = []
    for _ in range(2):
        c.run()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        c.run()
        end.record()
        end.synchronize()
        ms.append(start.elapsed_time(end))
        pg, at = (c.s.slots[0][list(where)] // 64).long(), (c.s.slots[0][list(where)] % 64).long()
        if fmt == "bf16":
            c.s.cache.v[pg, :, at] = math.nan
        else:
            c.s.cache.v_scale[pg, :, at] = math.nan if fmt == "e4m3" else 255
    assert not torch.isfinite(c.out).any() and torch.isfinite(c.lse).all()
    assert ms[1] <= 10 * ms[0], ms


def test_very_long_sequences(attn):
    """A value that all tokens see among 2^24 of them (a page that repeats): in time, and in its dim alone; and a
    NaN that some do not see behind 2^17."""
    page, D, G, new = 4096, 64, 8, 20
    for n, t in ((2 ** 24, 100), (2 ** 17, page - 3)):
        d = attn.dims(G, 1, D, rot_dim=0)
        cache = attn.KVCache.empty(d, 2, page, "bf16")
        ws = attn.workspace(d, prefill=True)
        g = torch.Generator(device="cuda")
        g.manual_seed(9)
        k, v, q = (torch.randn(m, h, D, generator=g, device="cuda").to(torch.bfloat16) for m, h in ((page, 1), (page, 1), (new, G)))
        attn.kv_write(d, k, v, torch.arange(page, device="cuda", dtype=torch.int32), cache, ws)
        attn.kv_write(d, k, v, torch.arange(page, 2 * page, device="cuda", dtype=torch.int32), cache, ws)
        table = torch.zeros(1, n // page, device="cuda", dtype=torch.int32)
        table[0, -1] = 1
        cache.v[0 if t == 100 else 1, 0, t, 5] = math.inf if t == 100 else math.nan
        out, lse = torch.zeros_like(q), torch.zeros(new, G, device="cuda")
        attn.prefill(d, q, torch.tensor([0, new], device="cuda", dtype=torch.int32), cache, table,
                     torch.tensor([n], device="cuda", dtype=torch.int32), out, ws, lse=lse)
        assert attn.device_status(ws) == 0 and torch.isfinite(lse).all()
        bad = torch.zeros(new, G, D, dtype=torch.bool, device="cuda")
        bad[0 if t == 100 else new - 3:, :, 5] = True
        assert torch.equal(~torch.isfinite(out), bad)
        kk, vv, qq = k[:, 0].double().cpu(), v[:, 0].double().cpu(), q.double().cpu()  # (what sees the other value is `bad`)
        # additions one after the other: a tile's products in 8 steps, in 150 parts; formed again, each fourth key
        adds = n / 1024 if t == 100 else n / 4
        for i in (0, new - 4, new - 1):
            times = n // page - (torch.arange(page) > page - new + i).double()  # a key of the page is seen
            for h in range(G):
                logits = d.softmax_scale * (kk @ qq[i, h])
                slack = (D + 8) * 2.0 ** -24 * float((d.softmax_scale * (kk.abs() @ qq[i, h].abs())).amax())
                w = times * torch.exp(logits)
                o, mean_abs = w @ vv / w.sum(), w @ vv.abs() / w.sum()
                tol = BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack + (64 + adds) * 2.0 ** -23)
                off = (out[i, h].double().cpu() - o).abs()
                assert ((off <= tol) | bad[i, h].cpu()).all(), (n, i, h)
