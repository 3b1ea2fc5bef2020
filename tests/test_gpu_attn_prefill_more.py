"""Prefill calls at their far ends: very long rows that are formed again, as many sequences as a call
takes, a process whose first call is captured."""
import os
import subprocess
import sys

import pytest

from tests import _attn_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16_HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def attn():
    import __graft_entry__ as g
    g.build()
    from mxfp4_routed_expert_latentmoe_gb300 import attn as mod
    torch.cuda.set_device(0)
    return mod


def _randn(*shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def test_infinite_values_in_very_long_sequences(attn):
    """Each row is formed again, over half a million tokens (a page that repeats), while the block's other
    warps wait with the next tile: seconds, which a wait has to outlast."""
    page, wide, D, G, new, B = 256, 2048, 64, 16, 16, 154
    n = page * wide
    d = attn.dims(G, 1, D, rot_dim=0)
    cache = attn.KVCache.empty(d, 1, page, "bf16")
    ws = attn.workspace(d, prefill=True)
    k, v, q = _randn(page, 1, D, seed=1), _randn(page, 1, D, seed=2), _randn(B * new, G, D, seed=3)
    v[100, 0, 5] = float("inf")
    attn.kv_write(d, k, v, torch.arange(page, device="cuda", dtype=torch.int32), cache, ws)
    table = torch.zeros(B, wide, device="cuda", dtype=torch.int32)
    out, lse = torch.zeros_like(q), torch.zeros(B * new, G, device="cuda")
    attn.prefill(d, q, torch.arange(0, B * new + 1, new, device="cuda", dtype=torch.int32), cache, table,
                 torch.full((B,), n, device="cuda", dtype=torch.int32), out, ws, lse=lse)
    assert attn.device_status(ws) == 0
    assert (out[:, :, 5] == torch.inf).all()
    others = torch.arange(D) != 5
    assert torch.isfinite(out[:, :, others.cuda()]).all() and torch.isfinite(lse).all()
    # a sequence's last token sees whole pages: as one page alone
    for b in (0, 77, B - 1):
        i = b * new + new - 1
        o, z, mean_abs, slack = ref.decode(q[i].double().cpu(), k.double().cpu(), v.double().cpu()[..., others], d.softmax_scale)
        # (sums of n terms in fp32, an eighth of them one after the other at most)
        tol = BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + (64 + n / 8) * 2.0 ** -24)
        assert ((out[i].double().cpu()[:, others] - o).abs() <= tol).all()


def test_as_many_sequences_as_a_call_takes(attn):
    B, page, D = 65535, 4, 64
    d = attn.dims(2, 1, D, rot_dim=0)
    ws = attn.workspace(d, prefill=True)
    cache = attn.KVCache.empty(d, 1000, page, "bf16")
    k, v, q = _randn(4000, 1, D, seed=4), _randn(4000, 1, D, seed=5), _randn(B, 2, D, seed=6)
    attn.kv_write(d, k, v, torch.arange(4000, device="cuda", dtype=torch.int32), cache, ws)
    table = (torch.arange(B, device="cuda") * 7 % 1000).to(torch.int32).view(B, 1)
    lens = (1 + torch.arange(B, device="cuda") % 4).to(torch.int32)
    out = torch.zeros_like(q)
    attn.prefill(d, q, torch.arange(B + 1, device="cuda", dtype=torch.int32), cache, table, lens, out, ws)
    kk, vv = (x.double().view(1000, page, D)[table[:, 0].long()] for x in (k, v))
    hidden = torch.arange(page, device="cuda") >= lens.view(B, 1, 1)
    logits = (d.softmax_scale * torch.einsum("bhd,btd->bht", q.double(), kk)).masked_fill(hidden, -torch.inf)
    w = torch.softmax(logits, -1)
    o, mean_abs = torch.einsum("bht,btd->bhd", w, vv), torch.einsum("bht,btd->bhd", w, vv.abs())
    # weights and results rounded to bf16; logits of 64 products in fp32 below 64 in size: 64 * 64 * 2^-24
    tol = BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2.0 ** -11)
    assert ((out.double() - o).abs() <= tol).all() and attn.device_status(ws) == 0


FIRST = """
import torch
from mxfp4_routed_expert_latentmoe_gb300 import attn
fmt, what = {fmt!r}, {what!r}
d = attn.dims(8, 2, 128, rot_dim=0, window=50)
cache = attn.KVCache.empty(d, 8, 16, fmt)
for t in (cache.k, cache.v):
    t.copy_(torch.randn(t.shape, device="cuda").to(t.dtype) if t.dtype == torch.bfloat16 else
            torch.randint(0, 120, t.shape, device="cuda").to(torch.uint8).view(t.dtype))
for t in (cache.k_scale, cache.v_scale):
    if t is not None:
        t.fill_(120 if t.dtype == torch.uint8 else 0.01)
table = torch.randperm(8, device="cuda").to(torch.int32).view(1, 8)
lens = torch.tensor([100], device="cuda", dtype=torch.int32)
q = torch.randn(1 if what == "decode" else 30, 8, 128, device="cuda").to(torch.bfloat16)
starts = torch.tensor([0, q.shape[0]], device="cuda", dtype=torch.int32)
out, ws = torch.zeros_like(q), attn.workspace(d, prefill=True)
def call():
    if what == "decode":
        attn.decode(d, q, cache, table, lens, out, ws, sinks=3)
    else:
        attn.prefill(d, q, starts, cache, table, lens, out, ws, sinks=3)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
g.replay()
torch.cuda.synchronize()
got = out.clone()
out.zero_()
call()
assert torch.equal(got, out) and bool(torch.isfinite(out).all()) and bool(out.any()) and attn.device_status(ws) == 0
print("same")
"""


@pytest.mark.parametrize("what", ["prefill", "decode"])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
def test_a_first_call_inside_a_capture(attn, fmt, what):
    r = subprocess.run([sys.executable, "-c", FIRST.format(fmt=fmt, what=what)], cwd=ROOT, capture_output=True, text=True,
                       timeout=240)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
