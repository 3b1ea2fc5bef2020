"""The decode attention at its edges: head dims that its tiles pad, lengths next to 2^31, short
sequences at the teams' borders, weights and logits of extreme sizes."""
import pytest

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
