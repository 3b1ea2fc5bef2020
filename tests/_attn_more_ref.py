"""Plain 64-bit forms for the tests of the 4-bit cache and of attention with sinks, on the CPU; and
sequences in a cache of any format."""
from __future__ import annotations

import torch

from tests import _attn_ref as ref

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def exponents(rows):
    """rows [..., D] f64 -> the E8M0 bytes [..., D / 32] of the definition."""
    amax = rows.unflatten(-1, (-1, 32)).abs().amax(-1)
    m, e = torch.frexp(torch.where(torch.isfinite(amax), amax, torch.ones_like(amax)))
    byte = (e - 3 + (m > 0.875).int()).clamp_min(-100) + 127  # amax <= 7 * 2^(byte - 127)
    byte = torch.where(amax == 0, torch.full_like(byte, 27), byte)
    return torch.where(torch.isfinite(amax), byte, torch.full_like(byte, 255)).to(torch.uint8)


def size_of(byte):
    return torch.where(byte == 255, torch.full(byte.shape, float("nan"), dtype=torch.float64),
                       torch.ldexp(torch.ones(byte.shape, dtype=torch.float64), byte.int() - 127))


def quantise_mxfp4(rows):
    """rows [..., D] of values exact in f64 -> (codes [..., D / 2] uint8, bytes [..., D / 32] uint8)."""
    x = rows.double().cpu()
    byte = exponents(x)
    z = x.unflatten(-1, (-1, 32)) / size_of(byte)[..., None]
    off = (z.abs()[..., None] - E2M1[:8]).abs()
    best = off.amin(-1, keepdim=True)
    near = off == best  # one, or two neighbours: then the even one
    even = torch.arange(8) % 2 == 0
    near = torch.where(near.sum(-1, keepdim=True) > 1, near & even, near)
    code = near.int().argmax(-1) + 8 * torch.signbit(z).int()
    code = torch.where(torch.isnan(z), torch.zeros_like(code), code).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte


def values_of(codes, byte):
    """f64 values of rows: codes [..., D / 2], bytes [..., D / 32 and more]."""
    codes, byte = codes.cpu(), byte.cpu()
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    return (E2M1[c].unflatten(-1, (-1, 32)) * size_of(byte[..., :c.shape[-1] // 32])[..., None]).flatten(-2)


def gather(cache, name, slots):
    """f64 rows [n, Hkv, D] of a cache's pool ("k" or "v") at slots."""
    pool, scales = getattr(cache, name), getattr(cache, name + "_scale")
    page, at = (slots.long() // cache.page_size).to(pool.device), (slots.long() % cache.page_size).to(pool.device)
    if pool.dtype != torch.uint8:
        return ref.gather(pool, scales, page, at)
    return values_of(pool[page, :, at], scales[page, :, at])


def seen(n, window, sinks, pos=None):
    """The tokens that the query at position pos (the last of n) attends to."""
    pos = n - 1 if pos is None else pos
    return [t for t in range(pos + 1) if not window or t > pos - window or t < sinks]


def empty_cache(attn, d, n_pages, page, fmt, order="phtd", stale=False):
    """A cache over tensors in the given memory order of pages, heads, tokens and the row's values;
    stale: NaN everywhere."""
    D = d.head_dim

    def tensor(width, dtype, fill):
        sizes = dict(p=n_pages, h=d.n_kv_heads, t=page, d=width)
        o = order if width else order.replace("d", "")
        t = torch.empty([sizes[c] for c in o], dtype=dtype, device="cuda")
        t.view(torch.uint8).fill_(fill)
        return t.permute([o.index(c) for c in "phtd" if c in o])

    fill = 0xFF if stale else 0
    if fmt == "bf16":
        return attn.KVCache(d, *(tensor(D, torch.bfloat16, fill) for _ in range(2)))
    if fmt == "e4m3":
        return attn.KVCache(d, *(tensor(D, torch.float8_e4m3fn, fill) for _ in range(2)),
                            *(tensor(0, torch.float32, fill) for _ in range(2)))
    return attn.KVCache(d, *(tensor(D // 2, torch.uint8, fill) for _ in range(2)),
                        *(tensor(attn.mxfp4_scales(D), torch.uint8, fill) for _ in range(2)))


class Sequences:
    """Sequences of the given lengths in a cache, on scattered pages of one that is NaN everywhere
    else; table entries that are not a sequence's point nowhere."""

    def __init__(self, attn, d, lens, page, fmt, seed, order="phtd", spread=0.5, room=0, k=None, v=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        used = [-(-n // page) for n in lens]
        self.d, self.lens, self.page = d, lens, page
        self.cache = empty_cache(attn, d, sum(used) + 2, page, fmt, order, stale=True)
        ids = torch.randperm(sum(used) + 2, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(lens), max(1, max(used)) + room), -7, device="cuda", dtype=torch.int32)
        self.slots, at = [], 0
        for b, (n, m) in enumerate(zip(lens, used)):
            self.table[b, :m] = ids[at:at + m]
            t = torch.arange(n, device="cuda", dtype=torch.int32)
            self.slots.append(ids[at:at + m][(t // page).long()] * page + t % page)
            at += m
        slots = torch.cat(self.slots).to(torch.int32)
        T, H, D = slots.numel(), d.n_kv_heads, d.head_dim
        if k is None:
            k = torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16)
        if v is None:
            v = (torch.randn(T, H, D, generator=g, device="cuda") *
                 torch.exp(spread * torch.randn(T, H, 1, generator=g, device="cuda"))).to(torch.bfloat16)
        self.ws = attn.workspace(d)
        if T:
            attn.kv_write(d, k, v, slots, self.cache, self.ws)
        self.lens_t = torch.tensor(lens, device="cuda", dtype=torch.int32)
        self.generator = g

    def queries(self, T, size=2.0):
        """q [T, Hq, D] bf16 as a slice of a projection's output."""
        d = self.d
        x = size * torch.randn(T, d.n_heads + 2 * d.n_kv_heads, d.head_dim, generator=self.generator, device="cuda")
        return x.to(torch.bfloat16)[:, :d.n_heads]

    def rows(self, b, which):
        """f64 (k, v) of sequence b's tokens `which`."""
        s = self.slots[b].cpu()[which].to("cuda")
        return gather(self.cache, "k", s), gather(self.cache, "v", s)
