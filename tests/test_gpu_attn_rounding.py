"""Bounds that notice what the other tests' leave room for: values far apart in size between key heads, and
weights rounded to no fewer bits than the interface says.  Each bound is shown to notice on the CPU first."""
import pytest

from tests import _attn_more_ref as more
from tests import _attn_ref as ref

torch = pytest.importorskip("torch")

BF16_HALF, FP16_HALF = 2.0 ** -8, 2.0 ** -11


@pytest.fixture(scope="module")
def attn():
    import __graft_entry__ as g
    g.build()
    from mxfp4_routed_expert_latentmoe_gb300 import attn as mod
    torch.cuda.set_device(0)
    return mod


# ------------------------------------------------------------------------ prefill: heads of very different values
def _head_bound(q, k, v, scale, fmt):
    """Prefill of one token, q [Hq, D] over k, v [n, Hkv, D] in f64: (out, what it may be off by).  A weight is
    rounded to bf16 (E4M3: times its row's scale; what falls below 2^-126, bf16's normal numbers, is lost: times
    a code, 448 at most; else a weight below 2^-126 of 2^0 .. 2^8 times a value of its own head), the result too."""
    o, _, mean_abs, slack = ref.decode(q, k, v, scale)
    n, group = k.shape[0], q.shape[0] // k.shape[1]
    lost = n * 2.0 ** -126 * (448 if fmt == "e4m3" else v.abs().amax((0, 2)).repeat_interleave(group)[:, None])
    return o, lost + BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + (64 + n / 8) * 2.0 ** -24)


def _far_apart(n, D, g):
    v = torch.randn(n, 3, D, generator=g) * torch.tensor([1e30, 1e-28, 1.0])[None, :, None]
    return torch.randn(n, 3, D, generator=g).to(torch.bfloat16), v.to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
def test_the_bound_notices_a_head_that_is_lost(fmt):
    g = torch.Generator()
    g.manual_seed(1)
    k, v = _far_apart(60, 64, g)
    q = 2 * torch.randn(6, 64, generator=g).double()
    o, tol = _head_bound(q, k.double(), v.double(), 0.125, fmt)
    for head in range(6):
        assert (o[head].abs() > 4 * tol[head]).float().mean() > 0.8  # zeros, or 1.25 times the result, would show
        assert ((0.25 * o[head]).abs() > tol[head]).float().mean() > 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (17, 3)])
def test_values_of_very_different_heads(attn, fmt, window, sinks):
    n, new, D = 200, 70, 64
    g = torch.Generator()
    g.manual_seed(2)
    k, v = _far_apart(n, D, g)
    d = attn.dims(6, 3, D, rot_dim=0, window=window)
    s = more.Sequences(attn, d, [n], 16, fmt, 3, k=k.cuda(), v=v.cuda())
    q, ws = s.queries(new), attn.workspace(d, prefill=True)
    out = torch.zeros(new, 6, D, device="cuda", dtype=torch.bfloat16)
    attn.prefill(d, q, torch.tensor([0, new], device="cuda", dtype=torch.int32), s.cache, s.table, s.lens_t, out, ws, sinks=sinks)
    kk, vv = s.rows(0, list(range(n)))
    for i in range(new):
        which = more.seen(n, window, sinks, n - new + i)
        o, tol = _head_bound(q[i].double().cpu(), kk[which], vv[which], d.softmax_scale, fmt)
        assert ((out[i].double().cpu() - o).abs() <= tol).all(), i
    assert attn.device_status(ws) == 0


# --------------------------------------------------------------------- decode over codes: weights of 11 bits
def _weight_bound(q, k, v, scale, fmt):
    """Decode of one token over codes: weights rounded to fp16 (times a group's factor once more, MXFP4),
    powers of two to 2^-22 of exponents whose fp32 error `slack` has; few tokens, of a size, so that what lies
    below fp16's normal numbers (2^-29 of the largest weight times scale) is 2^-30 of it at most."""
    o, _, mean_abs, slack = ref.decode(q, k, v, scale)
    n, group = k.shape[0], q.shape[0] // k.shape[1]
    largest = v.abs().amax((0, 2)).repeat_interleave(group)[:, None]
    rounds = 2 if fmt == "mxfp4" else 1
    return o, n * 2.0 ** -30 * largest + BF16_HALF * o.abs() + mean_abs * (rounds * FP16_HALF + 2 * slack[:, None] + 2.0 ** -17)


def _rounded(q, k, v, scale, dtype):
    """Decode with weights (1 for the largest) rounded to dtype, nothing else."""
    j = torch.arange(q.shape[0]) // (q.shape[0] // k.shape[1])
    logits = scale * torch.einsum("hd,nhd->hn", q, k[:, j])
    w = torch.exp(logits - logits.amax(-1, keepdim=True))
    return torch.einsum("hn,nhd->hd", w.to(dtype).double(), v[:, j]) / w.sum(-1, keepdim=True)


LENS = [3 + i % 4 for i in range(48)]


def _few(seed, n, D):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(n, 2, D, generator=g).to(torch.bfloat16) for _ in range(2))


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp4"])
def test_the_bound_notices_weights_of_8_bits(fmt):
    g = torch.Generator()
    g.manual_seed(5)
    D, over = 128, {torch.bfloat16: 0, torch.float16: 0}
    for b, n in enumerate(LENS):
        k, v = (x.double() for x in _few(b, n, D))
        if fmt == "mxfp4":
            k, v = (more.values_of(*more.quantise_mxfp4(x)) for x in (k, v))
        else:
            k, v = ((lambda c, s: c.view(torch.float8_e4m3fn).double() * s.double()[..., None])(*ref.quantise_f32(x)) for x in (k, v))
        q = torch.randn(16, D, generator=g).double()
        o, tol = _weight_bound(q, k, v, D ** -0.5, fmt)
        for dtype in over:
            over[dtype] += int(((_rounded(q, k, v, D ** -0.5, dtype).to(torch.bfloat16).double() - o).abs() > tol).sum())
    assert over[torch.float16] == 0 and over[torch.bfloat16] > 100, over


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "mxfp4"])
def test_weights_over_codes_have_11_bits(attn, fmt):
    D = 128
    d = attn.dims(16, 2, D, rot_dim=0)
    rows = [tuple(_few(b, n, D)) for b, n in enumerate(LENS)]
    k, v = (torch.cat([r[i] for r in rows]).cuda() for i in range(2))
    s = more.Sequences(attn, d, LENS, 16, fmt, 6, k=k, v=v)
    q = s.queries(len(LENS), 1.0)
    out = torch.zeros(len(LENS), 16, D, device="cuda", dtype=torch.bfloat16)
    attn.decode(d, q, s.cache, s.table, s.lens_t, out, s.ws)
    for b, n in enumerate(LENS):
        kk, vv = s.rows(b, list(range(n)))
        o, tol = _weight_bound(q[b].double().cpu(), kk, vv, d.softmax_scale, fmt)
        assert ((out[b].double().cpu() - o).abs() <= tol).all(), b
    assert attn.device_status(s.ws) == 0
