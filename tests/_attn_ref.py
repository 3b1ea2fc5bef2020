"""Plain 64-bit forms of the attention operators for their tests, on the CPU."""
from __future__ import annotations

import torch

FP8_MAX, MIN_SCALE = 448.0, 2.0 ** -100


def norm_rope(x, w, pos, inv_freq, eps, inter):
    """x [T, H, D] -> (y f64, size f64): the normed and rotated rows, and for each element the
    sum of the magnitudes that its rotation combines."""
    x, w = x.double().cpu(), w.double().cpu()
    n = w * x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    y, size = n.clone(), n.abs()
    if R:
        a = (pos.double().cpu()[:, None] * inv_freq.double().cpu())[:, None, :]
        i = torch.arange(R // 2)
        i0, i1 = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
        n0, n1 = n[..., i0], n[..., i1]
        y[..., i0] = n0 * torch.cos(a) - n1 * torch.sin(a)
        y[..., i1] = n1 * torch.cos(a) + n0 * torch.sin(a)
        size[..., i0] = size[..., i1] = n0.abs() + n1.abs()
    return y, size


def quantise_f32(rows):
    """The E4M3 row format applied to values that are exact in f32, in the f32 steps of the
    definition: (codes uint8, scales f32)."""
    rows = rows.float().cpu()
    amax = rows.abs().amax(-1)
    scale = (amax / FP8_MAX).clamp_min(MIN_SCALE)
    scale = torch.where(torch.isfinite(rows).all(-1), scale, torch.full_like(scale, float("nan")))
    z = (rows * (1.0 / scale)[..., None]).clamp(-FP8_MAX, FP8_MAX)
    return z.to(torch.float8_e4m3fn).view(torch.uint8), scale


def gather(pool, scales, page, at):
    """f64 rows [n, H, D] of a pool [P, H, S, D] at (page, at)."""
    page, at = page.cpu().long(), at.cpu().long()
    if pool.dtype == torch.float8_e4m3fn:
        rows = pool.cpu().view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn).double()
        return rows * scales.cpu()[page, :, at].double()[..., None]
    return pool.cpu()[page, :, at].double()


def decode(q, k, v, scale):
    """q [Hq, D], k and v [n, Hkv, D] in f64 -> (out, lse, mean_abs, slack): mean_abs is the
    attention's mean of |v|, slack the largest fp32 error of a row's logits (a dot product of
    D terms and a few roundings more), both [Hq, D] / [Hq]."""
    Hq, D = q.shape
    n, Hkv = k.shape[:2]
    if n == 0:
        zero = torch.zeros(Hq, D, dtype=torch.float64)
        return zero, torch.full((Hq,), -torch.inf, dtype=torch.float64), zero, torch.zeros(Hq, dtype=torch.float64)
    j = torch.arange(Hq) // (Hq // Hkv)
    logits = scale * torch.einsum("hd,nhd->hn", q, k[:, j])
    sizes = scale * torch.einsum("hd,nhd->hn", q.abs(), k[:, j].abs())
    p = torch.softmax(logits, -1)
    out = torch.einsum("hn,nhd->hd", p, v[:, j])
    mean_abs = torch.einsum("hn,nhd->hd", p, v[:, j].abs())
    return out, torch.logsumexp(logits, -1), mean_abs, (D + 8) * 2.0 ** -24 * sizes.amax(-1)
