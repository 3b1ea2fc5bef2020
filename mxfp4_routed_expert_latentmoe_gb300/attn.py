"""The attention operators that stand before the routed-expert block when it serves tokens:
norms of queries and keys per head with the position rotation, the paged key-value cache
(bf16, or E4M3 with a scale per row), and the attention of one new token over its pages.

Thin binding over the C ABI declared in ``include/k3attn.h``, which has the formulas.  Every
function checks its tensors (ValueError), which all have to be on one device, passes pointers and
strides, and launches there, on that device's current stream or on ``stream``; device-detected conditions (DEV_BAD_*) are read with
``device_status(ws)``.  The operators' checks and calls are native (csrc/attn/k3attn_binding.cpp):
a decode step's kernels take no longer than they would in Python.

    d = attn.dims(n_heads=64, n_kv_heads=8, head_dim=128, rot_dim=128)
    cache = attn.KVCache.empty(d, n_pages=4096, page_size=64, fmt="e4m3")
    ws = attn.workspace(d)
    attn.kv_append(d, q, k, v, positions, slots, inv_freq, q_w, k_w, cache, q_out, ws)
    attn.decode(d, q_out, cache, page_table, lens, out, ws)
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _stream, lib
from . import device_status as _device_status

BF16, E4M3 = 0, 1  # K3ATTN_BF16, K3ATTN_E4M3
MIN_WORKSPACE = 256  # K3ATTN_MIN_WORKSPACE
DEV_BAD_SLOT, DEV_BAD_PAGE, DEV_BAD_LENGTH = 0x1, 0x2, 0x4
_fns = None
_native = None  # the extension module, loaded by the first operator


class Dims(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("rot_interleaved", ctypes.c_int32), ("rms_eps", ctypes.c_float),
                ("softmax_scale", ctypes.c_float), ("window", ctypes.c_int32)]

    @property
    def addr(self):  # (of this object: a copy has its own)
        return ctypes.addressof(self)


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
            f = getattr(L, name, None)
            if f is None:
                raise RuntimeError(f"libk3moe.so has no {name}: it is older than this package, build() it")
            f.argtypes = args
            f.restype = res
        _fns = L
    return _fns


def _load():
    """The native side, bound to the library's operators."""
    global _native
    if _native is None:
        import importlib.util
        import os
        import shutil

        from . import _stale, attn_binding_path, attn_binding_sources, build_attn_binding
        L, path = _funcs(), attn_binding_path()
        if not os.path.exists(path) or (_stale(path, attn_binding_sources()) and shutil.which("g++")):
            build_attn_binding()
        spec = importlib.util.spec_from_file_location("k3attn_binding", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.bind(*(ctypes.cast(getattr(L, "k3attn_" + n), ctypes.c_void_p).value
                   for n in ("qk_norm_rope", "kv_write", "kv_append", "kv_read", "decode")))
        _native = mod
    return _native


def declared_functions() -> list:
    """Function names declared in include/k3attn.h."""
    import re

    from . import _ATTN_HEADER
    return sorted(set(re.findall(r"\b(k3attn_[a-z0-9_]+)\s*\(", open(_ATTN_HEADER).read())))


# ------------------------------------------------------------------------------ what a program keeps
def workspace_bytes(d: Dims) -> int:
    """Bytes of workspace that decode needs with these dims (0: unsupported); the other operators
    take any of at least MIN_WORKSPACE."""
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
    if ws.dtype != torch.uint8 or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws: a contiguous uint8 CUDA tensor is needed")
    with torch.cuda.device(ws.device):
        _check(_funcs().k3attn_workspace_init(ws.data_ptr(), ws.numel(), _stream(stream)), "k3attn_workspace_init")


def device_status(ws, stream=None) -> int:
    """DEV_BAD_* bits of the calls that used workspace `ws` since it was readied (waits for the
    stream)."""
    with torch.cuda.device(ws.device):
        return _device_status(ws, stream)


def rope_frequencies(rot_dim: int, theta: float = 10000.0, device="cuda"):
    """inv_freq [rot_dim / 2] f64: theta^(-2i / rot_dim)."""
    return theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)


class KVCache:
    """A paged cache over the caller's tensors: k, v [n_pages, Hkv, page_size, D], bf16 or
    float8_e4m3fn, with the same strides (any order of pages, heads and tokens; a row's D
    values dense); for E4M3 k_scale, v_scale [n_pages, Hkv, page_size] f32."""

    def __init__(self, d: Dims, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("k: [n_pages, Hkv, page_size, D] of bfloat16 or float8_e4m3fn is needed")
        fmt = E4M3 if k.dtype == torch.float8_e4m3fn else BF16
        shape = (k.shape[0], d.n_kv_heads, k.shape[2], d.head_dim)
        for t, name in ((k, "k"), (v, "v")):
            if (t.dtype != k.dtype or t.shape != shape or not t.is_cuda or t.device != k.device or t.stride(3) != 1
                    or t.stride() != k.stride()):
                raise ValueError(f"{name}: a CUDA tensor {list(shape)} of {k.dtype}, a row's values dense, with the "
                                 f"strides of k and on its device, is needed, got {list(t.shape)} (strides {list(t.stride())}) of "
                                 f"{t.dtype} on {t.device}")
        n, page, ss = shape[0], shape[2], (0, 0, 0)
        if fmt == E4M3:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if (t is None or t.dtype != torch.float32 or t.shape != shape[:3] or t.device != k.device
                        or t.stride() != k_scale.stride()):
                    raise ValueError(f"{name}: a CUDA tensor {list(shape[:3])} of float32, with the strides of "
                                     "k_scale and on the device of k, is needed for an E4M3 cache")
            ss = k_scale.stride()
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size = n, page
        self.c = CacheC(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if fmt == E4M3 else None,
                        v_scale.data_ptr() if fmt == E4M3 else None, fmt, n, page, 0, *k.stride()[:3], *ss)
        self.addr = ctypes.addressof(self.c)
        self.rows = (k.device.index << 32) + d.n_kv_heads * 65536 + d.head_dim  # what a call compares with its own

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


# ------------------------------------------------------------------------------ the operators
def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def qk_norm_rope(d: Dims, q, k, positions, inv_freq, q_w, k_w, q_out, k_out, stream=None):
    """k3attn_qk_norm_rope: q [T, Hq, D], k [T, Hkv, D] bf16 (slices of one projection's output
    will do) -> q_out, k_out, dense, normed per head and rotated.  inv_freq may be None when
    d.rot_dim is 0."""
    code = (_native or _load()).qk_norm_rope(d.addr, q, k, positions, inv_freq, q_w, k_w, q_out, k_out,
                                             _handle(stream))
    if code:
        _check(code, "k3attn_qk_norm_rope")


def kv_write(d: Dims, k, v, slots, cache: KVCache, ws, stream=None):
    """k3attn_kv_write: k, v [T, Hkv, D] bf16 into the cache at slots [T] int32 (-1: not written)."""
    code = (_native or _load()).kv_write(d.addr, k, v, slots, cache.addr, cache.rows, ws, _handle(stream))
    if code:
        _check(code, "k3attn_kv_write")


def kv_append(d: Dims, q, k, v, positions, slots, inv_freq, q_w, k_w, cache: KVCache, q_out, ws, k_out=None,
              stream=None):
    """k3attn_kv_append: qk_norm_rope of q into q_out and of k, and the write of k and v into the
    cache, in one pass; k_out (optional) also receives the keys."""
    code = (_native or _load()).kv_append(d.addr, q, k, v, positions, slots, inv_freq, q_w, k_w, cache.addr,
                                          cache.rows, q_out, k_out, ws, _handle(stream))
    if code:
        _check(code, "k3attn_kv_append")


def kv_read(d: Dims, slots, cache: KVCache, k_out, v_out, ws, stream=None):
    """k3attn_kv_read: the rows at slots [T] int32 as bf16, k_out and v_out [T, Hkv, D]."""
    code = (_native or _load()).kv_read(d.addr, slots, cache.addr, cache.rows, k_out, v_out, ws, _handle(stream))
    if code:
        _check(code, "k3attn_kv_read")


def decode(d: Dims, q, cache: KVCache, page_table, lens, out, ws, lse=None, stream=None):
    """k3attn_decode: q [B, Hq, D] bf16, one new token per sequence, over the first lens[b] tokens
    of the pages page_table[b] -> out [B, Hq, D] bf16 and, if given, lse [B, Hq] f32.  With more
    than 8 query heads a key head a table just wide enough is faster for few short sequences."""
    code = (_native or _load()).decode(d.addr, q, cache.addr, cache.rows, page_table, lens, out, lse, ws,
                                       _handle(stream))
    if code:
        _check(code, "k3attn_decode")
