"""Host-only checks of the attention operators' Python side: what a call reads of its dims, which
tensors it refuses, and how its parts are built."""
import copy
import ctypes
import os
import pickle
import sys

import pytest

import mxfp4_routed_expert_latentmoe_gb300 as k3
from mxfp4_routed_expert_latentmoe_gb300 import attn

torch = pytest.importorskip("torch")


def _dims(**kw):
    return attn.dims(**{**dict(n_heads=8, n_kv_heads=2, head_dim=128), **kw})


def test_copies_of_dims_stand_for_themselves():
    """What a call reads is the copy's memory, not that of the original (which may be gone)."""
    d = _dims(window=7)
    for e in (copy.copy(d), copy.deepcopy(d), pickle.loads(pickle.dumps(d)), attn.Dims.from_buffer_copy(d)):
        assert e.addr == ctypes.addressof(e) != d.addr
        assert bytes(e) == bytes(d)
        e.n_heads, e.window = 16, 9
        assert (d.n_heads, d.window) == (8, 7)
        # the native side sees the copy's heads: it asks for queries of them
        with pytest.raises(ValueError, match=r"q: a CUDA tensor .1, 16, 128."):
            attn.qk_norm_rope(e, torch.zeros(1, 8, 128), *[None] * 7)


@pytest.fixture
def two_devices():
    """Tensors that say they are on one of two GPUs (without storage: no call may get past its checks)."""
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    mode = fake.FakeTensorMode()

    def make(*shape, dtype=torch.bfloat16, device=0):
        with mode:
            return torch.empty(*shape, dtype=dtype, device=f"cuda:{device}")
    return make


def _calls(make):
    """Each operator with its tensors on device 0, by their names, and its cache's device."""
    d, T = _dims(), 3
    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)
    q, kv, pool = (T, 8, 128), (T, 2, 128), (4, 2, 16, 128)
    tensors = dict(q=lambda dev: make(*q, device=dev), k=lambda dev: make(*kv, device=dev),
                   v=lambda dev: make(*kv, device=dev), positions=lambda dev: make(T, device=dev, **i32),
                   slots=lambda dev: make(T, device=dev, **i32), lens=lambda dev: make(T, device=dev, **i32),
                   page_table=lambda dev: make(T, 4, device=dev, **i32),
                   inv_freq=lambda dev: make(64, dtype=torch.float64, device=dev),
                   q_w=lambda dev: make(128, device=dev, **f32), k_w=lambda dev: make(128, device=dev, **f32),
                   q_out=lambda dev: make(*q, device=dev), k_out=lambda dev: make(*kv, device=dev),
                   v_out=lambda dev: make(*kv, device=dev), out=lambda dev: make(*q, device=dev),
                   lse=lambda dev: make(T, 8, device=dev, **f32),
                   ws=lambda dev: make(1 << 20, dtype=torch.uint8, device=dev),
                   cache=lambda dev: attn.KVCache(d, make(*pool, device=dev), make(*pool, device=dev)))
    names = {attn.qk_norm_rope: "q k positions inv_freq q_w k_w q_out k_out", attn.kv_write: "k v slots cache ws",
             attn.kv_append: "q k v positions slots inv_freq q_w k_w cache q_out ws k_out",
             attn.kv_read: "slots cache k_out v_out ws", attn.decode: "q cache page_table lens out ws lse"}
    return d, tensors, {f: n.split() for f, n in names.items()}


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_tensors_on_several_devices_are_refused(two_devices):
    """Each tensor of each operator on another device than the others."""
    d, tensors, operators = _calls(two_devices)
    for f, names in operators.items():
        for stranger in names:
            args = {n: tensors[n](int(n == stranger)) for n in names}
            with pytest.raises(ValueError, match="on cuda:[01], is needed|the cache is on cuda:"):
                f(d, **args)


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_a_cache_on_several_devices_is_refused(two_devices):
    d, f8, f32 = _dims(), dict(dtype=torch.float8_e4m3fn), dict(dtype=torch.float32)
    pool, scales = (4, 2, 16, 128), (4, 2, 16)
    for at in range(1, 4):
        x = [two_devices(*pool, device=0, **f8), two_devices(*pool, device=int(at == 1), **f8),
             two_devices(*scales, device=int(at == 2), **f32), two_devices(*scales, device=int(at == 3), **f32)]
        with pytest.raises(ValueError, match="device"):
            attn.KVCache(d, *x)


def test_the_workspace_is_readied_and_read_on_its_own_device(monkeypatch):
    """With another device current: the calls' stream is that of the workspace's device."""
    current, seen = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Library:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, current[0])) or 0

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(attn, "_funcs", Library)
    monkeypatch.setattr(attn, "_stream", lambda s: ("stream of", current[0]))
    monkeypatch.setattr(attn, "_device_status", lambda ws, s: seen.append(("status", current[0])) or 0)

    class Ws:
        dtype, is_cuda, device = torch.uint8, True, torch.device("cuda:1")
        is_contiguous, data_ptr, numel = (lambda self: True), (lambda self: 4096), (lambda self: 256)

    attn.workspace_init(Ws())
    assert attn.device_status(Ws()) == 0
    assert seen == [("k3attn_workspace_init", 1), ("status", 1)] and current == [0]


# ------------------------------------------------------------------------------ the build
@pytest.fixture
def compiled(monkeypatch):
    """The outputs that a build compiles, by their names (nothing is run)."""
    seen = []
    monkeypatch.setattr(k3, "_compile", lambda cmd, out, *_: seen.append(os.path.basename(out)))
    return seen


def test_the_library_is_built_without_torch(compiled, monkeypatch):
    assert k3.build() == k3._SO
    assert sorted(compiled) == sorted(["libk3moe.so", os.path.basename(k3.attn_binding_path())])
    del compiled[:]
    monkeypatch.setitem(sys.modules, "torch", None)  # (import torch raises)
    assert k3.build() == k3._SO and compiled == ["libk3moe.so"]


def test_a_binding_that_does_not_compile_leaves_the_library_built(monkeypatch):
    seen = []

    def compile_(cmd, out, *_):
        if "binding" in out:
            raise RuntimeError("g++ failed: no Python.h")
        seen.append(out)

    monkeypatch.setattr(k3, "_compile", compile_)
    with pytest.raises(RuntimeError, match="Python.h"):
        k3.build()
    assert seen == [k3._SO]


def test_a_binding_belongs_to_one_torch_and_python(monkeypatch):
    import sysconfig
    paths = {k3.attn_binding_path()}
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    paths.add(k3.attn_binding_path())
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399")
    paths.add(k3.attn_binding_path())
    assert len(paths) == 3


def test_a_library_older_than_its_sources_is_built_again(tmp_path, monkeypatch):
    so, nvcc, compiled = tmp_path / "libk3moe.so", tmp_path / "nvcc", []
    with open(k3.build_library(), "rb") as f:
        so.write_bytes(f.read())
    monkeypatch.setattr(k3, "_compile", lambda cmd, out, *_: compiled.append(os.path.basename(out)))
    monkeypatch.setattr(k3, "_SO", str(so))
    monkeypatch.setattr(k3, "_nvcc", lambda: str(nvcc))
    for age, compiler, built in ((10, True, []), (-10, True, ["libk3moe.so"]), (-10, False, [])):
        monkeypatch.setattr(k3, "_lib", None)
        newest = max(os.path.getmtime(f) for f in k3._sources())
        os.utime(so, (newest + age, newest + age))
        nvcc.write_text("") if compiler else nvcc.unlink()
        k3.lib()
        assert compiled == built, (age, compiler)
        del compiled[:]


def test_a_library_without_the_operators_says_so(monkeypatch):
    monkeypatch.setattr(attn, "_fns", None)
    monkeypatch.setattr(attn, "lib", lambda: object())
    with pytest.raises(RuntimeError, match="older than this package"):
        attn.workspace_bytes(_dims())


def test_a_library_without_its_sources_is_loaded_as_it_is(tmp_path, monkeypatch):
    k3.build_library()
    for name in ("_CSRC", "_ATTN", "_HEADER", "_ATTN_HEADER"):
        monkeypatch.setattr(k3, name, str(tmp_path / "not there"))
    monkeypatch.setattr(k3, "_compile", lambda *a: pytest.fail("nothing can be built"))
    monkeypatch.setattr(k3, "_lib", None)
    assert k3.lib().k3moe_abi_version() > 0
    assert not k3._stale(k3._SO, k3._sources())
