"""The attention operators that stand before the routed-expert block when it serves tokens:
norms of queries and keys per head with the position rotation, the paged key-value cache
(bf16, or E4M3 with a scale per row), and the attention of one new token over its pages.

Thin binding over the C ABI declared in ``include/k3attn.h``, which has the formulas.  Every
function checks its tensors (ValueError), passes pointers and strides, and launches on the
current CUDA stream or on ``stream``; device-detected conditions (DEV_BAD_*) are read with
``device_status(ws)``.

    d = attn.dims(n_heads=64, n_kv_heads=8, head_dim=128, rot_dim=128)
    cache = attn.KVCache.empty(d, n_pages=4096, page_size=64, fmt="e4m3")
    ws = attn.workspace(d)
    attn.kv_append(d, q, k, v, positions, slots, inv_freq, q_w, k_w, cache, q_out, ws)
    attn.decode(d, q_out, cache, page_table, lens, out, ws)
"""
from __future__ import annotations

import ctypes

import torch

from . import K3MoEError, device_status, lib  # noqa: F401  (device_status: the status word of ws)

BF16, E4M3 = 0, 1  # K3ATTN_BF16, K3ATTN_E4M3
MIN_WORKSPACE = 256  # K3ATTN_MIN_WORKSPACE
DEV_BAD_SLOT, DEV_BAD_PAGE, DEV_BAD_LENGTH = 0x1, 0x2, 0x4
_fns = None


class Dims(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("rot_interleaved", ctypes.c_int32), ("rms_eps", ctypes.c_float),
                ("softmax_scale", ctypes.c_float), ("window", ctypes.c_int32)]

    def __init__(self, *args):
        super().__init__(*args)
        self.ref = ctypes.byref(self)


def dims(n_heads, n_kv_heads, head_dim, rot_dim=None, rot_interleaved=False, rms_eps=1e-6, softmax_scale=None,
         window=0) -> Dims:
    """The k3attn_dims struct; rot_dim defaults to head_dim, softmax_scale to 1 / sqrt(head_dim)."""
    return Dims(n_heads, n_kv_heads, head_dim, head_dim if rot_dim is None else rot_dim, int(rot_interleaved), rms_eps,
                head_dim ** -0.5 if softmax_scale is None else softmax_scale, window)


class CacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("format", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("reserved", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("scale_token_stride", ctypes.c_int64)]


def _funcs():
    """The library's attention functions with their signatures set."""
    global _fns
    if _fns is None:
        L = lib()
        p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        D, C = ctypes.POINTER(Dims), ctypes.POINTER(CacheC)
        sigs = {
            "k3attn_workspace_bytes": ([D], sz),
            "k3attn_workspace_init": ([p, sz, p], ctypes.c_int),
            "k3attn_qk_norm_rope": ([D, i32, p, i64, p, i64, p, p, p, p, p, p, p], ctypes.c_int),
            "k3attn_kv_write": ([D, i32, p, i64, p, i64, p, C, p, sz, p], ctypes.c_int),
            "k3attn_kv_append": ([D, i32, p, i64, p, i64, p, i64, p, p, p, p, p, C, p, p, p, sz, p], ctypes.c_int),
            "k3attn_kv_read": ([D, i32, p, C, p, p, p, sz, p], ctypes.c_int),
            "k3attn_decode": ([D, i32, p, i64, C, p, i32, p, p, p, p, sz, p], ctypes.c_int),
        }
        for name, (args, res) in sigs.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _fns = L
    return _fns


def declared_functions() -> list:
    """Function names declared in include/k3attn.h."""
    import re

    from . import _ATTN_HEADER
    return sorted(set(re.findall(r"\b(k3attn_[a-z0-9_]+)\s*\(", open(_ATTN_HEADER).read())))


# ------------------------------------------------------------------------------ checks
# (a decode step's call takes a few microseconds on the GPU: the operators below check in line,
# by comparisons alone, and a message is put together only where one fails)
_bf16, _f32, _i32, _f64, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.float64, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream


def _refuse(t, name, dtype, shape, how=", contiguous"):
    got = f"{list(t.shape)} (strides {list(t.stride())}) of {t.dtype} on {t.device}" if torch.is_tensor(t) else repr(t)
    raise ValueError(f"{name}: a CUDA tensor {list(shape)} of {dtype}{how} is needed, got {got}")


def _rows(t, name, T, heads, D):
    """Pointer and token stride of a [T, heads, D] bf16 tensor whose tokens' rows are dense."""
    sT, sH, sD = t.stride() if t.dim() == 3 else (0, 0, 0)
    if not (t.dtype is _bf16 and t.shape == (T, heads, D) and t.is_cuda and sD == 1 and (sH == D or heads == 1)):
        _refuse(t, name, _bf16, (T, heads, D), ", the heads of a token dense,")
    return t.data_ptr(), sT if T > 1 else heads * D


def _ws(ws):
    if not (ws.dtype is _u8 and ws.is_cuda and ws.is_contiguous()):
        _refuse(ws, "ws", _u8, ("bytes",))
    return ws.data_ptr(), ws.numel()


def _on(t, stream):
    """The stream of a call: `stream`, or the current one of t's device."""
    if stream is None:
        return _raw_stream(t.get_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _fail(code, what):
    raise K3MoEError(code, what)


# ------------------------------------------------------------------------------ what a program keeps
def workspace_bytes(d: Dims) -> int:
    return int(_funcs().k3attn_workspace_bytes(ctypes.byref(d)))


def workspace(d: Dims, device="cuda"):
    """A workspace for calls with these dims (or smaller ones), readied for its first use."""
    n = workspace_bytes(d)
    if n == 0:
        raise ValueError("unsupported dims")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    workspace_init(ws)
    return ws


def workspace_init(ws, stream=None):
    """k3attn_workspace_init: readies a workspace (also clears its status word)."""
    code = _funcs().k3attn_workspace_init(*_ws(ws), _on(ws, stream))
    if code:
        _fail(code, "k3attn_workspace_init")


def rope_frequencies(rot_dim: int, theta: float = 10000.0, device="cuda"):
    """inv_freq [rot_dim / 2] f64: theta^(-2i / rot_dim)."""
    return theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)


class KVCache:
    """A paged cache over the caller's tensors: k, v [n_pages, Hkv, page_size, D], bf16 or
    float8_e4m3fn, with the same strides (any order of pages, heads and tokens; a row's D
    values dense); for E4M3 k_scale, v_scale [n_pages, Hkv, page_size] f32."""

    def __init__(self, d: Dims, k, v, k_scale=None, v_scale=None):
        shape = (k.shape[0], d.n_kv_heads, k.shape[2], d.head_dim) if k.dim() == 4 else ("n_pages", "Hkv", "page", "D")
        fmt = E4M3 if k.dtype is torch.float8_e4m3fn else BF16
        for t, name in ((k, "k"), (v, "v")):
            if not (t.dtype is (torch.float8_e4m3fn if fmt == E4M3 else _bf16) and t.shape == shape and t.is_cuda
                    and t.stride(3) == 1 and t.stride() == k.stride()):
                _refuse(t, name, "bfloat16 or float8_e4m3fn", shape, ", a row's values dense, strides as k's,")
        n, page, ss = shape[0], shape[2], (0, 0, 0)
        if fmt == E4M3:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if t is None or not (t.dtype is _f32 and t.shape == shape[:3] and t.is_cuda
                                     and t.stride() == k_scale.stride()):
                    _refuse(t, name, _f32, shape[:3], ", strides as k_scale's,")
            ss = k_scale.stride()
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.head_shape = n, page, (d.n_kv_heads, d.head_dim)
        self.c = CacheC(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if fmt == E4M3 else None,
                        v_scale.data_ptr() if fmt == E4M3 else None, fmt, n, page, 0, *k.stride()[:3], *ss)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, d: Dims, n_pages: int, page_size: int, fmt: str = "bf16", device="cuda"):
        """A dense cache of zeros; fmt "bf16" or "e4m3"."""
        if fmt not in ("bf16", "e4m3"):
            raise ValueError("fmt is bf16 or e4m3")
        shape = (n_pages, d.n_kv_heads, page_size, d.head_dim)
        if fmt == "bf16":
            return cls(d, *(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        codes = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        return cls(d, *codes, *(torch.ones(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))


def _cache(d, cache):
    if cache.head_shape != (d.n_kv_heads, d.head_dim):
        raise ValueError(f"the cache's (Hkv, D) are {cache.head_shape}, the dims' {(d.n_kv_heads, d.head_dim)}")
    return cache.ref


# ------------------------------------------------------------------------------ the operators
def _norm_args(d, T, D, positions, inv_freq, q_w, k_w):
    """Pointers of what the norms and the rotation read beside the rows."""
    if not (positions.dtype is _i32 and positions.shape == (T,) and positions.is_cuda and positions.is_contiguous()):
        _refuse(positions, "positions", _i32, (T,))
    if not (q_w.dtype is _f32 and q_w.shape == (D,) and q_w.is_cuda and q_w.is_contiguous()):
        _refuse(q_w, "q_w", _f32, (D,))
    if not (k_w.dtype is _f32 and k_w.shape == (D,) and k_w.is_cuda and k_w.is_contiguous()):
        _refuse(k_w, "k_w", _f32, (D,))
    R = d.rot_dim
    if R == 0:
        return positions.data_ptr(), None, q_w.data_ptr(), k_w.data_ptr()
    if not (inv_freq.dtype is _f64 and inv_freq.shape == (R // 2,) and inv_freq.is_cuda and inv_freq.is_contiguous()):
        _refuse(inv_freq, "inv_freq", _f64, (R // 2,))
    return positions.data_ptr(), inv_freq.data_ptr(), q_w.data_ptr(), k_w.data_ptr()


def qk_norm_rope(d: Dims, q, k, positions, inv_freq, q_w, k_w, q_out, k_out, stream=None):
    """k3attn_qk_norm_rope: q [T, Hq, D], k [T, Hkv, D] bf16 (slices of one projection's output
    will do) -> q_out, k_out, dense, normed per head and rotated.  inv_freq may be None when
    d.rot_dim is 0."""
    T, Hq, Hkv, D = q.shape[0], d.n_heads, d.n_kv_heads, d.head_dim
    qp, qs = _rows(q, "q", T, Hq, D)
    kp, ks = _rows(k, "k", T, Hkv, D)
    pos, freq, qw, kw = _norm_args(d, T, D, positions, inv_freq, q_w, k_w)
    if not (q_out.dtype is _bf16 and q_out.shape == (T, Hq, D) and q_out.is_cuda and q_out.is_contiguous()):
        _refuse(q_out, "q_out", _bf16, (T, Hq, D))
    if not (k_out.dtype is _bf16 and k_out.shape == (T, Hkv, D) and k_out.is_cuda and k_out.is_contiguous()):
        _refuse(k_out, "k_out", _bf16, (T, Hkv, D))
    code = _funcs().k3attn_qk_norm_rope(d.ref, T, qp, qs, kp, ks, pos, freq, qw, kw, q_out.data_ptr(),
                                        k_out.data_ptr(), _on(q, stream))
    if code:
        _fail(code, "k3attn_qk_norm_rope")


def kv_write(d: Dims, k, v, slots, cache: KVCache, ws, stream=None):
    """k3attn_kv_write: k, v [T, Hkv, D] bf16 into the cache at slots [T] int32 (-1: not written)."""
    T, Hkv, D = k.shape[0], d.n_kv_heads, d.head_dim
    kp, ks = _rows(k, "k", T, Hkv, D)
    vp, vs = _rows(v, "v", T, Hkv, D)
    if not (slots.dtype is _i32 and slots.shape == (T,) and slots.is_cuda and slots.is_contiguous()):
        _refuse(slots, "slots", _i32, (T,))
    code = _funcs().k3attn_kv_write(d.ref, T, kp, ks, vp, vs, slots.data_ptr(), _cache(d, cache), *_ws(ws),
                                    _on(k, stream))
    if code:
        _fail(code, "k3attn_kv_write")


def kv_append(d: Dims, q, k, v, positions, slots, inv_freq, q_w, k_w, cache: KVCache, q_out, ws, k_out=None,
              stream=None):
    """k3attn_kv_append: qk_norm_rope of q into q_out and of k, and the write of k and v into the
    cache, in one pass; k_out (optional) also receives the keys."""
    T, Hq, Hkv, D = q.shape[0], d.n_heads, d.n_kv_heads, d.head_dim
    qp, qs = _rows(q, "q", T, Hq, D)
    kp, ks = _rows(k, "k", T, Hkv, D)
    vp, vs = _rows(v, "v", T, Hkv, D)
    pos, freq, qw, kw = _norm_args(d, T, D, positions, inv_freq, q_w, k_w)
    if not (slots.dtype is _i32 and slots.shape == (T,) and slots.is_cuda and slots.is_contiguous()):
        _refuse(slots, "slots", _i32, (T,))
    if not (q_out.dtype is _bf16 and q_out.shape == (T, Hq, D) and q_out.is_cuda and q_out.is_contiguous()):
        _refuse(q_out, "q_out", _bf16, (T, Hq, D))
    ko = None
    if k_out is not None:
        if not (k_out.dtype is _bf16 and k_out.shape == (T, Hkv, D) and k_out.is_cuda and k_out.is_contiguous()):
            _refuse(k_out, "k_out", _bf16, (T, Hkv, D))
        ko = k_out.data_ptr()
    code = _funcs().k3attn_kv_append(d.ref, T, qp, qs, kp, ks, vp, vs, pos, slots.data_ptr(), freq, qw, kw,
                                     _cache(d, cache), q_out.data_ptr(), ko, *_ws(ws), _on(q, stream))
    if code:
        _fail(code, "k3attn_kv_append")


def kv_read(d: Dims, slots, cache: KVCache, k_out, v_out, ws, stream=None):
    """k3attn_kv_read: the rows at slots [T] int32 as bf16, k_out and v_out [T, Hkv, D]."""
    T, Hkv, D = slots.shape[0], d.n_kv_heads, d.head_dim
    if not (slots.dtype is _i32 and slots.shape == (T,) and slots.is_cuda and slots.is_contiguous()):
        _refuse(slots, "slots", _i32, (T,))
    if not (k_out.dtype is _bf16 and k_out.shape == (T, Hkv, D) and k_out.is_cuda and k_out.is_contiguous()):
        _refuse(k_out, "k_out", _bf16, (T, Hkv, D))
    if not (v_out.dtype is _bf16 and v_out.shape == (T, Hkv, D) and v_out.is_cuda and v_out.is_contiguous()):
        _refuse(v_out, "v_out", _bf16, (T, Hkv, D))
    code = _funcs().k3attn_kv_read(d.ref, T, slots.data_ptr(), _cache(d, cache), k_out.data_ptr(), v_out.data_ptr(),
                                   *_ws(ws), _on(slots, stream))
    if code:
        _fail(code, "k3attn_kv_read")


def decode(d: Dims, q, cache: KVCache, page_table, lens, out, ws, lse=None, stream=None):
    """k3attn_decode: q [B, Hq, D] bf16, one new token per sequence, over the first lens[b] tokens
    of the pages page_table[b] -> out [B, Hq, D] bf16 and, if given, lse [B, Hq] f32."""
    B, Hq, D = q.shape[0], d.n_heads, d.head_dim
    qp, qs = _rows(q, "q", B, Hq, D)
    width = page_table.shape[-1]
    if not (page_table.dtype is _i32 and page_table.shape == (B, width) and page_table.is_cuda
            and page_table.is_contiguous()):
        _refuse(page_table, "page_table", _i32, (B, "width"))
    if not (lens.dtype is _i32 and lens.shape == (B,) and lens.is_cuda and lens.is_contiguous()):
        _refuse(lens, "lens", _i32, (B,))
    if not (out.dtype is _bf16 and out.shape == (B, Hq, D) and out.is_cuda and out.is_contiguous()):
        _refuse(out, "out", _bf16, (B, Hq, D))
    lp = None
    if lse is not None:
        if not (lse.dtype is _f32 and lse.shape == (B, Hq) and lse.is_cuda and lse.is_contiguous()):
            _refuse(lse, "lse", _f32, (B, Hq))
        lp = lse.data_ptr()
    code = _funcs().k3attn_decode(d.ref, B, qp, qs, _cache(d, cache), page_table.data_ptr(), width, lens.data_ptr(),
                                  out.data_ptr(), lp, *_ws(ws), _on(q, stream))
    if code:
        _fail(code, "k3attn_decode")
