"""Host-only checks of the attention of many new tokens: what the C ABI and the binding refuse before a
device is touched."""
import ctypes

import pytest

from mxfp4_routed_expert_latentmoe_gb300 import attn
from tests import test_attn_host as base
from tests.test_attn_binding import two_devices  # noqa: F401

torch = pytest.importorskip("torch")

OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WS, ERR_DEVICE = range(6)
GPU = torch.cuda.is_available()
V = base.V


def _prefill(d, B=1, T=1, cache=None, width=4, sinks=0, ws_bytes=None, **kw):
    a = dict(q=V, qs=1024, starts=V, table=V, lens=V, out=V, lse=V, ws=V)
    a.update(kw)
    c = ctypes.byref(cache or base._cache())
    n = max(attn.workspace_bytes(d, prefill=True), 256) if ws_bytes is None else ws_bytes
    return attn._funcs().k3attn_prefill(ctypes.byref(d), sinks, B, T, a["q"], a["qs"], a["starts"], c, a["table"], width,
                                        a["lens"], a["out"], a["lse"], a["ws"], n, None)


@pytest.mark.parametrize("bad,code", base.BAD_DIMS, ids=[str(b) for b, _ in base.BAD_DIMS])
def test_bad_dims_are_refused(bad, code):
    d = base._dims(**bad)
    assert attn.workspace_bytes(d, prefill=True) == 0 and _prefill(d) == code


@pytest.mark.parametrize("bad,code", base.BAD_CACHE, ids=[str(b) for b, _ in base.BAD_CACHE])
def test_bad_caches_are_refused(bad, code):
    c = base._cache(**bad)
    assert _prefill(base._dims(), cache=c) == _prefill(base._dims(), cache=c, B=0) == _prefill(base._dims(), cache=c, T=0) == code


def test_arguments_are_validated_on_the_host():
    d = base._dims()
    assert _prefill(d, B=0) == _prefill(d, T=0) == OK
    assert _prefill(d, B=-1) == _prefill(d, T=-1) == _prefill(d, width=-1) == _prefill(d, sinks=-1) == ERR_ARG
    for name in ("q", "starts", "table", "lens", "out", "ws"):
        assert _prefill(d, **{name: None}) == ERR_ARG, name
    for name in ("q", "out", "ws"):
        assert _prefill(d, **{name: ctypes.c_void_p(4104)}) == ERR_ALIGN, name
    for name in ("starts", "table", "lens", "lse"):
        assert _prefill(d, **{name: ctypes.c_void_p(4098)}) == ERR_ALIGN, name
    assert _prefill(d, qs=1016) == ERR_SHAPE and _prefill(d, qs=1028) == ERR_ALIGN
    assert _prefill(d, B=65536) == ERR_SHAPE and _prefill(d, width=1 << 28) == ERR_SHAPE
    n = attn.workspace_bytes(d, prefill=True)
    assert n >= attn.workspace_bytes(d) and _prefill(d, ws_bytes=n - 1) == ERR_WS
    if not GPU:
        assert _prefill(d) == _prefill(d, lse=None) == _prefill(d, width=0, table=None) == ERR_DEVICE


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_tensors_on_several_devices_are_refused(two_devices):  # noqa: F811
    make, d, T, B = two_devices, base._dims(), 5, 3
    i32, pool = dict(dtype=torch.int32), (4, 2, 16, 128)
    tensors = dict(q=lambda dev: make(T, 8, 128, device=dev), q_starts=lambda dev: make(B + 1, device=dev, **i32),
                   cache=lambda dev: attn.KVCache(d, make(*pool, device=dev), make(*pool, device=dev)),
                   page_table=lambda dev: make(B, 4, device=dev, **i32), lens=lambda dev: make(B, device=dev, **i32),
                   out=lambda dev: make(T, 8, 128, device=dev), ws=lambda dev: make(1 << 20, dtype=torch.uint8, device=dev),
                   lse=lambda dev: make(T, 8, dtype=torch.float32, device=dev))
    for stranger in tensors:
        with pytest.raises(ValueError, match="on cuda:[01], is needed|the cache is on cuda:"):
            attn.prefill(d, **{n: t(int(n == stranger)) for n, t in tensors.items()})
    for bad in (dict(q_starts=make(0, **i32)), dict(q_starts=make(B, **i32)), dict(lse=make(T, 4, dtype=torch.float32))):
        with pytest.raises(ValueError):
            attn.prefill(d, **{**{n: t(0) for n, t in tensors.items()}, **bad})
