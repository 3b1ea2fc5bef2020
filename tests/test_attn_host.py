"""Host-only checks of the attention operators' C ABI and binding: every declared function is
exported, the status bits match the header, and arguments are refused before a device is
touched."""
import ctypes
import re

import pytest

import mxfp4_routed_expert_latentmoe_gb300 as k3
from mxfp4_routed_expert_latentmoe_gb300 import attn

torch = pytest.importorskip("torch")

OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WS, ERR_DEVICE = range(6)
V = ctypes.c_void_p(4096)  # never read: every call below is refused first, or finds no device
GPU = torch.cuda.is_available()


def test_library_exports_every_declared_function_and_the_binding_declares_it():
    names = attn.declared_functions()
    assert {"k3attn_decode", "k3attn_kv_append", "k3attn_qk_norm_rope"} <= set(names)
    L = attn._funcs()
    for n in names:
        assert getattr(L, n).argtypes is not None, n


def test_constants_match_the_header():
    text = open(k3._ATTN_HEADER).read()
    bits = {m.group(1): int(m.group(2), 16) for m in re.finditer(r"#define K3ATTN_DEV_(\w+) (0x[0-9a-f]+)u", text)}
    assert bits == {"BAD_SLOT": attn.DEV_BAD_SLOT, "BAD_PAGE": attn.DEV_BAD_PAGE,
                    "BAD_LENGTH": attn.DEV_BAD_LENGTH}
    assert f"#define K3ATTN_MIN_WORKSPACE {attn.MIN_WORKSPACE}u" in text
    assert f"#define K3ATTN_BF16 {attn.BF16}\n" in text and f"#define K3ATTN_E4M3 {attn.E4M3}\n" in text


BAD_DIMS = [(dict(n_heads=0), ERR_SHAPE), (dict(n_heads=1025, n_kv_heads=1), ERR_SHAPE),
            (dict(n_kv_heads=3), ERR_SHAPE), (dict(n_kv_heads=0), ERR_SHAPE), (dict(head_dim=8, rot_dim=0), ERR_SHAPE),
            (dict(head_dim=100, rot_dim=0), ERR_SHAPE), (dict(head_dim=272), ERR_SHAPE), (dict(rot_dim=8), ERR_SHAPE),
            (dict(rot_dim=144), ERR_SHAPE), (dict(rot_dim=-16), ERR_SHAPE), (dict(rot_interleaved=2), ERR_ARG),
            (dict(rms_eps=-1.0), ERR_ARG), (dict(rms_eps=float("nan")), ERR_ARG), (dict(softmax_scale=0.0), ERR_ARG),
            (dict(softmax_scale=float("inf")), ERR_ARG), (dict(window=-1), ERR_ARG)]


def _dims(**kw):
    return attn.dims(**{**dict(n_heads=8, n_kv_heads=2, head_dim=128), **kw})


def _norm_rope(d, T=1, **kw):
    a = dict(q=V, qs=1024, k=V, ks=256, pos=V, freq=V, qw=V, kw=V, qo=V, ko=V, **{})
    a.update(kw)
    return attn._funcs().k3attn_qk_norm_rope(ctypes.byref(d), T, a["q"], a["qs"], a["k"], a["ks"], a["pos"], a["freq"],
                                             a["qw"], a["kw"], a["qo"], a["ko"], None)


@pytest.mark.parametrize("bad,code", BAD_DIMS, ids=[str(b) for b, _ in BAD_DIMS])
def test_bad_dims_are_refused_everywhere(bad, code):
    d = _dims(**bad)
    assert attn.workspace_bytes(d) == 0
    assert _norm_rope(d) == code
    assert _write(d) == _append(d) == _read(d) == _decode(d) == code


def test_norm_rope_validates_on_the_host():
    d = _dims()
    assert _norm_rope(d, T=0) == OK
    assert _norm_rope(d, T=-1) == ERR_ARG
    for name in ("q", "k", "pos", "freq", "qw", "kw", "qo", "ko"):
        assert _norm_rope(d, **{name: None}) == ERR_ARG, name
    for name in ("q", "k", "qw", "kw", "qo", "ko"):
        assert _norm_rope(d, **{name: ctypes.c_void_p(4104)}) == ERR_ALIGN, name
    assert _norm_rope(d, pos=ctypes.c_void_p(4098)) == ERR_ALIGN
    assert _norm_rope(d, freq=ctypes.c_void_p(4100)) == ERR_ALIGN
    assert _norm_rope(d, qs=1016) == ERR_SHAPE and _norm_rope(d, ks=255) == ERR_SHAPE
    assert _norm_rope(d, qs=1028) == ERR_ALIGN and _norm_rope(d, ks=257) == ERR_ALIGN
    if not GPU:  # valid calls (positions at any 4 bytes; no frequencies without a rotation) reach the device check
        assert _norm_rope(d, pos=ctypes.c_void_p(4100)) == ERR_DEVICE
        assert _norm_rope(_dims(rot_dim=0), freq=None) == ERR_DEVICE


def _cache(fmt=attn.E4M3, **kw):
    a = dict(k=4096, v=4096, k_scale=4096, v_scale=4096, format=fmt, n_pages=10, page_size=16, reserved=0,
             page_stride=4096, head_stride=2048, token_stride=128, scale_page_stride=32, scale_head_stride=16,
             scale_token_stride=1)
    a.update(kw)
    return attn.CacheC(*(a[n] for n, _ in attn.CacheC._fields_))


def _write(d, T=1, cache=None, ws_bytes=256, **kw):
    a = dict(k=V, ks=256, v=V, vs=256, slots=V, ws=V)
    a.update(kw)
    c = ctypes.byref(cache or _cache())
    return attn._funcs().k3attn_kv_write(ctypes.byref(d), T, a["k"], a["ks"], a["v"], a["vs"], a["slots"], c, a["ws"],
                                         ws_bytes, None)


def _append(d, T=1, cache=None, ws_bytes=256, **kw):
    a = dict(q=V, qs=1024, k=V, ks=256, v=V, vs=256, pos=V, slots=V, freq=V, qw=V, kw=V, qo=V, ko=None, ws=V)
    a.update(kw)
    c = ctypes.byref(cache or _cache())
    return attn._funcs().k3attn_kv_append(ctypes.byref(d), T, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                                          a["pos"], a["slots"], a["freq"], a["qw"], a["kw"], c, a["qo"], a["ko"],
                                          a["ws"], ws_bytes, None)


def _read(d, T=1, cache=None, ws_bytes=256, **kw):
    a = dict(slots=V, ko=V, vo=V, ws=V)
    a.update(kw)
    c = ctypes.byref(cache or _cache())
    return attn._funcs().k3attn_kv_read(ctypes.byref(d), T, a["slots"], c, a["ko"], a["vo"], a["ws"], ws_bytes, None)


def _decode(d, B=1, cache=None, width=4, ws_bytes=None, **kw):
    a = dict(q=V, qs=1024, table=V, lens=V, out=V, lse=V, ws=V)
    a.update(kw)
    c = ctypes.byref(cache or _cache())
    n = max(attn.workspace_bytes(d), 256) if ws_bytes is None else ws_bytes
    return attn._funcs().k3attn_decode(ctypes.byref(d), B, a["q"], a["qs"], c, a["table"], width, a["lens"], a["out"],
                                       a["lse"], a["ws"], n, None)


BAD_CACHE = [(dict(k=0), ERR_ARG), (dict(v=0), ERR_ARG), (dict(k_scale=0), ERR_ARG), (dict(v_scale=0), ERR_ARG),
             (dict(format=2), ERR_ARG), (dict(n_pages=0), ERR_ARG), (dict(page_size=0), ERR_ARG),
             (dict(reserved=1), ERR_ARG), (dict(n_pages=1 << 20, page_size=1 << 12), ERR_SHAPE),
             (dict(token_stride=64), ERR_SHAPE), (dict(head_stride=0), ERR_SHAPE), (dict(page_stride=-128), ERR_SHAPE),
             (dict(scale_token_stride=0), ERR_SHAPE), (dict(k=4104), ERR_ALIGN), (dict(v=4104), ERR_ALIGN),
             (dict(token_stride=136), ERR_ALIGN), (dict(head_stride=2056), ERR_ALIGN),
             (dict(page_stride=4104), ERR_ALIGN), (dict(k_scale=4098), ERR_ALIGN)]


@pytest.mark.parametrize("bad,code", BAD_CACHE, ids=[str(b) for b, _ in BAD_CACHE])
def test_bad_caches_are_refused_everywhere(bad, code):
    d, c = _dims(), _cache(**bad)
    assert _write(d, cache=c) == _append(d, cache=c) == _read(d, cache=c) == _decode(d, cache=c) == code
    # without tokens as well
    assert _write(d, T=0, cache=c) == code


def test_bf16_cache_needs_no_scales_and_half_the_alignment_of_strides():
    d = _dims()
    c = _cache(attn.BF16, k_scale=0, v_scale=0, scale_page_stride=0, scale_head_stride=0, scale_token_stride=0,
               token_stride=136, head_stride=2176, page_stride=4352)
    if not GPU:
        assert _write(d, cache=c) == _append(d, cache=c) == _read(d, cache=c) == _decode(d, cache=c) == ERR_DEVICE
    c.token_stride = 132
    assert _write(d, cache=c) == ERR_ALIGN


@pytest.mark.parametrize("call,names", [(_write, ("k", "v", "slots", "ws")),
                                        (_append, ("q", "k", "v", "pos", "slots", "freq", "qw", "kw", "qo", "ws")),
                                        (_read, ("slots", "ko", "vo", "ws")),
                                        (_decode, ("q", "table", "lens", "out", "ws"))])
def test_cache_calls_validate_on_the_host(call, names):
    d = _dims()
    assert call(d, 0) == OK
    assert call(d, -1) == ERR_ARG
    for name in names:
        assert call(d, **{name: None}) == ERR_ARG, name
        bad = 4098 if name in ("slots", "pos", "table", "lens") else 4100
        assert call(d, **{name: ctypes.c_void_p(bad)}) == ERR_ALIGN, name
    for name, width in (("qs", 1024), ("ks", 256), ("vs", 256)):
        if name[0] in names:
            assert call(d, **{name: width - 8}) == ERR_SHAPE, name
            assert call(d, **{name: width + 4}) == ERR_ALIGN, name
    assert call(d, ws_bytes=255) == ERR_WS
    if not GPU:
        assert call(d) == ERR_DEVICE


def test_decode_limits():
    d = _dims()
    assert _decode(d, ws_bytes=attn.workspace_bytes(d) - 1) == ERR_WS
    assert _decode(d, width=-1) == ERR_ARG
    assert _decode(d, width=1 << 28) == ERR_SHAPE  # 2^28 pages of 16 tokens pass int32
    assert _decode(d, B=65536) == ERR_SHAPE
    assert _decode(d, lse=ctypes.c_void_p(4098)) == ERR_ALIGN
    if not GPU:
        assert _decode(d, lse=None) == ERR_DEVICE
        assert _decode(d, width=0, table=None) == ERR_DEVICE


def test_workspace_init_validates_on_the_host():
    L = attn._funcs()
    assert L.k3attn_workspace_init(None, 256, None) == ERR_ARG
    assert L.k3attn_workspace_init(ctypes.c_void_p(4104), 256, None) == ERR_ALIGN
    assert L.k3attn_workspace_init(V, 255, None) == ERR_WS
    if not GPU:
        assert L.k3attn_workspace_init(V, 256, None) == ERR_DEVICE


def test_the_binding_refuses_tensors_that_do_not_fit():
    d = _dims()
    cpu = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q: a CUDA tensor .1, 8, 128. of BFloat16"):  # not on the GPU
        attn.qk_norm_rope(d, cpu, cpu[:, :2], None, None, None, None, None, None)
    for not_a_tensor in (None, 3, [1.0]):
        with pytest.raises(ValueError):
            attn.qk_norm_rope(d, not_a_tensor, cpu[:, :2], None, None, None, None, None, None)
    pool = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attn.KVCache(d, pool, pool)
    with pytest.raises(ValueError):
        attn.KVCache(d, pool.float(), pool.float())
    with pytest.raises(ValueError):
        attn.KVCache.empty(d, 4, 16, fmt="int3")
    with pytest.raises(ValueError):
        attn.workspace(_dims(head_dim=100, rot_dim=0))


def test_the_native_side_checks_its_arguments_count_and_structs():
    native = attn._load()
    for f, n in ((native.qk_norm_rope, 10), (native.kv_write, 8), (native.kv_append, 15), (native.kv_read, 8),
                 (native.decode, 10), (native.bind, 5)):
        with pytest.raises(TypeError):
            f(*[None] * (n - 1))
    with pytest.raises(ValueError):  # no dims at address 0
        native.decode(0, *[None] * 9)
    with pytest.raises(TypeError):  # not an address
        native.decode("x", *[None] * 9)


def test_rope_frequencies():
    f = attn.rope_frequencies(64, 1e6, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    assert f[0] == 1.0 and abs(f[8].item() - 1e6 ** -0.25) < 1e-15
