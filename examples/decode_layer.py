"""One decoder layer serving a batch: the attention operators, then the routed-expert block.

Per step and sequence: q, k, v from one projection; norms and rotation of q and k, k and v into
the paged cache (one call); attention over the cache; output projection and residual; the
routed-expert block (k3moe_forward) and residual.  The step is captured into a CUDA graph once
and replayed while the sequences grow: lengths, positions and slots live on the device.

    python examples/decode_layer.py --batch 8 --prompt 1000 --steps 32 --format e4m3

The weights are random.  With --check the last step's attention is compared with a plain form
over the rows read back from the cache.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import mxfp4_routed_expert_latentmoe_gb300 as k3  # noqa: E402
from datagen import configs as C  # noqa: E402
from datagen import device as D  # noqa: E402
from mxfp4_routed_expert_latentmoe_gb300 import attn  # noqa: E402


class Layer:
    """Weights, cache and buffers of one layer for `batch` sequences of up to `longest` tokens."""

    def __init__(self, cfg, batch, longest, heads=16, kv_heads=2, head_dim=128, fmt="e4m3", page=16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        H = cfg.hidden

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") / math.sqrt(shape[-1])).to(torch.bfloat16)

        self.cfg, self.batch, self.page = cfg, batch, page
        # attention
        self.d = attn.dims(heads, kv_heads, head_dim)
        self.w_qkv, self.w_o = weight((heads + 2 * kv_heads) * head_dim, H), weight(H, heads * head_dim)
        self.q_w, self.k_w = (torch.ones(head_dim, device="cuda") for _ in range(2))
        self.inv_freq = attn.rope_frequencies(head_dim, 1e6)
        wide = -(-longest // page)
        self.cache = attn.KVCache.empty(self.d, batch * wide, page, fmt)
        self.ws = attn.workspace(self.d)
        # each sequence's pages, scattered over the cache; its places in order
        self.table = torch.randperm(batch * wide, generator=g, device="cuda").to(torch.int32).view(batch, wide)
        self.places = (self.table.unsqueeze(-1) * page + torch.arange(page, device="cuda", dtype=torch.int32)).flatten(1)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.q = torch.empty(batch, heads, head_dim, dtype=torch.bfloat16, device="cuda")
        self.a = torch.empty_like(self.q)
        # the routed-expert block
        self.md = k3.dims(**cfg.dims)
        self.t = D.layer_tensors(cfg, "cuda")
        self.pool, expert_bytes, offsets = D.expert_pool(cfg, "cuda")
        self.experts = k3.ExpertTables.from_pool(self.pool, expert_bytes, offsets)
        self.moe = torch.empty(batch, H, dtype=torch.float32, device="cuda")
        self.moe_ws = torch.empty(k3.workspace_bytes(self.md, batch), dtype=torch.uint8, device="cuda")

    def _qkv(self, x):
        d = self.d
        return (x @ self.w_qkv.t()).view(x.shape[0], -1, d.head_dim).split([d.n_heads, d.n_kv_heads, d.n_kv_heads], 1)

    def prompt(self, x):
        """The prompts' keys and values into the cache: x [batch, n, H] bf16."""
        n = x.shape[1]
        q, k, v = self._qkv(x.flatten(0, 1))
        pos = torch.arange(n, device="cuda", dtype=torch.int32).repeat(self.batch)
        attn.kv_append(self.d, q, k, v, pos, self.places[:, :n].flatten(), self.inv_freq, self.q_w, self.k_w,
                       self.cache, torch.empty(q.shape, dtype=q.dtype, device="cuda"), self.ws)
        self.lens.fill_(n)

    def step(self, x):
        """One new token per sequence: x [batch, H] bf16 -> the layer's output, [batch, H] bf16."""
        t, pos = self.t, self.lens.clone()
        slots = self.places.gather(1, pos.long().unsqueeze(1)).squeeze(1)
        self.lens += 1
        q, k, v = self._qkv(x)
        attn.kv_append(self.d, q, k, v, pos, slots, self.inv_freq, self.q_w, self.k_w, self.cache, self.q, self.ws)
        attn.decode(self.d, self.q, self.cache, self.table, self.lens, self.a, self.ws)
        y = x + self.a.flatten(1) @ self.w_o.t()
        k3.forward(self.md, y, t["wr"], t["bias"], t["wd"], t["wu"], t["gamma"], self.experts, self.moe, self.moe_ws)
        return (y.float() + self.moe).to(torch.bfloat16)

    def attention_error(self):
        """Largest difference of the last step's attention from a plain form over the cache's
        rows, relative to the mean size of the values that it mixes."""
        d, worst = self.d, 0.0
        for b, n in enumerate(self.lens.tolist()):
            k, v = (torch.empty(n, d.n_kv_heads, d.head_dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            attn.kv_read(d, self.places[b, :n].contiguous(), self.cache, k, v, self.ws)
            each = d.n_heads // d.n_kv_heads
            kk, vv = (x.double().repeat_interleave(each, 1) for x in (k, v))
            p = torch.softmax(d.softmax_scale * torch.einsum("hd,nhd->hn", self.q[b].double(), kk), -1)
            off = (self.a[b].double() - torch.einsum("hn,nhd->hd", p, vv)).abs()
            worst = max(worst, float((off / torch.einsum("hn,nhd->hd", p, vv.abs())).max()))
        return worst


def run(cfg=C.MID, batch=8, prompt=1000, steps=32, fmt="e4m3", page=16, check=False):
    layer = Layer(cfg, batch, prompt + steps + 2, fmt=fmt, page=page)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    layer.prompt(torch.randn(batch, prompt, cfg.hidden, generator=g, device="cuda").to(torch.bfloat16))
    x = torch.randn(batch, cfg.hidden, generator=g, device="cuda").to(torch.bfloat16)
    out = layer.step(x)  # a step before the capture, so that everything is loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(x)
        # the output, brought back to size, is the next input
        x.copy_(out * torch.rsqrt(out.float().square().mean(-1, keepdim=True)))
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    status = attn.device_status(layer.ws), k3.device_status(layer.moe_ws)
    if any(status):
        raise RuntimeError(f"device status {status}")
    got = {"us_per_step": start.elapsed_time(end) / steps * 1e3, "lens": layer.lens.tolist(), "out": out}
    if check:
        got["error"] = layer.attention_error()
    return got


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--config", default="mid", choices=sorted(C.LAYER_CONFIGS), help="the routed-expert block's shapes")
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=1000)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--format", default="e4m3", choices=("e4m3", "bf16"))
    p.add_argument("--page", type=int, default=16)
    p.add_argument("--check", action="store_true")
    a = p.parse_args(argv)
    r = run(C.LAYER_CONFIGS[a.config], a.batch, a.prompt, a.steps, a.format, a.page, a.check)
    print(f"{a.batch} sequences from {a.prompt} tokens on, {a.format} cache: {r['us_per_step']:.1f} us a step"
          + (f", attention off by {r['error']:.2e} of the values' mean size" if a.check else ""))


if __name__ == "__main__":
    main()
