"""Host-only checks of the 4-bit cache and of sinks: what the C ABI and the binding refuse before a
device is touched."""
import ctypes

import pytest

import mxfp4_routed_expert_latentmoe_gb300 as k3
from mxfp4_routed_expert_latentmoe_gb300 import attn
from tests import test_attn_host as base

torch = pytest.importorskip("torch")

OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WS, ERR_DEVICE = range(6)
GPU = torch.cuda.is_available()


def _cache(**kw):
    a = dict(page_stride=4096, head_stride=2048, token_stride=128, scale_page_stride=128, scale_head_stride=64,
             scale_token_stride=4)
    a.update(kw)
    return base._cache(attn.MXFP4, **a)


def _everywhere(d, c, code):
    assert base._write(d, cache=c) == base._append(d, cache=c) == base._read(d, cache=c) == base._decode(d, cache=c) == code


def test_the_format_is_the_headers():
    text = open(k3._ATTN_HEADER).read()
    assert f"#define K3ATTN_MXFP4 {attn.MXFP4}\n" in text
    assert [attn.mxfp4_scales(D) for D in (32, 96, 128, 160, 256)] == [4, 4, 4, 8, 8]


BAD = [(dict(k=0), ERR_ARG), (dict(k_scale=0), ERR_ARG), (dict(v_scale=0), ERR_ARG), (dict(token_stride=96), ERR_SHAPE),
       (dict(scale_token_stride=3), ERR_SHAPE), (dict(scale_head_stride=0), ERR_SHAPE), (dict(scale_page_stride=-4), ERR_SHAPE),
       (dict(token_stride=144), ERR_ALIGN), (dict(head_stride=2064), ERR_ALIGN), (dict(page_stride=4112), ERR_ALIGN),
       (dict(scale_token_stride=6), ERR_ALIGN), (dict(scale_head_stride=66), ERR_ALIGN), (dict(scale_page_stride=130), ERR_ALIGN),
       (dict(k=4104), ERR_ALIGN), (dict(v_scale=4098), ERR_ALIGN), (dict(reserved=1), ERR_ARG)]


@pytest.mark.parametrize("bad,code", BAD, ids=[str(b) for b, _ in BAD])
def test_bad_caches_are_refused_everywhere(bad, code):
    _everywhere(base._dims(), _cache(**bad), code)


def test_unknown_formats_and_head_dims_are_refused():
    for fmt in (2, 3, 5, -1):
        _everywhere(base._dims(), _cache(format=fmt), ERR_ARG)
    for D in (16, 48, 80, 240):
        d = base._dims(head_dim=D, rot_dim=0)
        _everywhere(d, _cache(), ERR_SHAPE)
    # a row of more than 128 has two words of scales
    d = base._dims(head_dim=160, rot_dim=0)
    wide = dict(token_stride=160, head_stride=2560, page_stride=5120)
    assert base._read(d, cache=_cache(**wide)) == ERR_SHAPE
    if not GPU:
        assert base._read(d, cache=_cache(scale_token_stride=8, **wide)) == ERR_DEVICE
        _everywhere(base._dims(), _cache(), ERR_DEVICE)  # a valid one reaches the device check


def test_sinks_are_validated_on_the_host():
    d, c, V = base._dims(window=100), _cache(), base.V
    n = attn.workspace_bytes(d)

    def call(sinks, B=1):
        return attn._funcs().k3attn_decode_sinks(ctypes.byref(d), sinks, B, V, 1024, ctypes.byref(c), V, 4, V, V, V, V, n, None)
    assert call(-1) == call(-1, B=0) == ERR_ARG
    assert call(5, B=0) == OK
    if not GPU:
        assert call(0) == call(2 ** 31 - 1) == ERR_DEVICE


@pytest.fixture
def make():
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    mode = fake.FakeTensorMode()

    def tensor(*shape, dtype=torch.uint8, device="cuda:0"):
        with mode:
            return torch.empty(*shape, dtype=dtype, device=device)
    return tensor


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_the_cache_checks_its_tensors(make):
    d = base._dims()
    k, s = make(4, 2, 16, 64), make(4, 2, 16, 4)
    c = attn.KVCache(d, k, make(4, 2, 16, 64), s, make(4, 2, 16, 4)).c
    assert (c.format, c.token_stride, c.head_stride, c.page_stride) == (attn.MXFP4, 128, 2048, 4096)
    assert (c.scale_token_stride, c.scale_head_stride, c.scale_page_stride) == (4, 64, 128)
    f32 = make(4, 2, 16, dtype=torch.float32)
    for bad in ((k, make(4, 2, 16, 128), s, s), (make(4, 2, 16, 128), make(4, 2, 16, 128), s, s), (k, k, None, None),
                (k, k, s, None), (k, k, f32, f32), (k, k, make(4, 2, 16, 3), make(4, 2, 16, 3)),
                (k, k, s, make(4, 2, 16, 8)[..., :4]), (k, k, make(4, 2, 4, 16).transpose(2, 3), make(4, 2, 4, 16).transpose(2, 3)),
                (k, make(4, 2, 16, 64, device="cuda:1"), s, s), (k, k, s, make(4, 2, 16, 4, device="cuda:1")),
                (k, make(4, 2, 16, 64, dtype=torch.int8), s, s)):
        with pytest.raises(ValueError):
            attn.KVCache(d, *bad)
    with pytest.raises(ValueError, match="multiple of 32"):
        attn.KVCache(base._dims(head_dim=80), make(4, 2, 16, 40), make(4, 2, 16, 40), s, s)
    with pytest.raises(ValueError):
        attn.KVCache.empty(d, 1, 1, "fp4")


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_sinks_that_are_no_number_are_refused(make):
    d = base._dims()
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    cache = attn.KVCache(d, make(4, 2, 16, 128, **bf), make(4, 2, 16, 128, **bf))
    args = (d, make(3, 8, 128, **bf), cache, make(3, 4, **i32), make(3, **i32), make(3, 8, 128, **bf), make(1 << 20))
    for bad, error in ((2 ** 31, ValueError), (-2 ** 40, ValueError), ("4", TypeError), (1.5, TypeError)):
        with pytest.raises(error):
            attn.decode(*args, sinks=bad)
