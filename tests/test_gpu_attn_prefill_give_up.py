"""A wait inside the prefill kernel that runs out: the kernel ends, says so in the status word, and leaves
the GPU as it was for the next call.  Each warp's waits run out in turn, in blocks with whole tiles, with
the first, a middle and the last part of a tile that is cut."""
import ctypes
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))
TIMEOUT = 0x100


@pytest.fixture(scope="module")
def launch(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("give_up") / "prefill_give_up.so")
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-shared", "-o", so, os.path.join(HERE, "prefill_give_up.cu")], check=True)
    torch.cuda.set_device(0)
    torch.zeros(1, device="cuda")  # (the context)
    lib = ctypes.CDLL(so)
    lib.parts_floats.restype = ctypes.c_size_t
    return lib


# new and cached tokens: whole tiles, one of 6 parts (in blocks 1 to 6 of 20), whole tiles
SIZES = [(70, 70)] * 4 + [(32, 30000)] + [(70, 200)] * 30
HQ, HKV, D, PAGE, GRID = 8, 1, 64, 16, 20


class Call:
    def __init__(self, launch, fmt):
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        self.launch, self.fmt = launch, fmt
        wide = -(-max(n for _, n in SIZES) // PAGE)
        self.pages, self.wide, self.T = wide, wide, sum(n for n, _ in SIZES)
        if fmt == "bf16":
            self.k, self.v = (torch.randn(wide, HKV, PAGE, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
            self.ks = self.vs = torch.zeros(1, device="cuda")
        else:
            self.k, self.v = (torch.randint(0, 256, (wide, HKV, PAGE, D // 2), generator=g, device="cuda").to(torch.uint8)
                              for _ in range(2))
            self.ks, self.vs = (torch.randint(125, 129, (wide, HKV, PAGE, 4), generator=g, device="cuda").to(torch.uint8)
                                for _ in range(2))
        self.q = torch.randn(self.T, HQ, D, generator=g, device="cuda").to(torch.bfloat16)
        self.starts = torch.tensor([0] + [n for n, _ in SIZES], device="cuda").cumsum(0).to(torch.int32)
        self.lens = torch.tensor([n for _, n in SIZES], device="cuda", dtype=torch.int32)
        self.table = torch.arange(wide, device="cuda", dtype=torch.int32).repeat(len(SIZES), 1).contiguous()
        self.status = torch.zeros(1, device="cuda", dtype=torch.int32)
        self.arrived = torch.zeros(1024, device="cuda", dtype=torch.int32)
        self.parts = torch.zeros(launch.parts_floats(), device="cuda")
        self.out = torch.zeros(self.T, HQ, D, device="cuda", dtype=torch.bfloat16)
        self.lse = torch.zeros(self.T, HQ, device="cuda")

    def __call__(self, block=0, warp=0, wait=0):
        """(whether the wait ran out, status)"""
        for t in (self.status, self.arrived, self.out, self.lse):
            t.zero_()
        torch.cuda.synchronize()
        p = [ctypes.c_void_p(t.data_ptr()) for t in (self.q, self.k, self.v, self.ks, self.vs, self.starts, self.table, self.lens,
                                                     self.out, self.lse, self.status, self.arrived, self.parts)]
        got = self.launch.give_up(0 if self.fmt == "bf16" else 4, block, warp, wait, GRID, len(SIZES), self.T, HQ, HKV, 0, 0, self.pages,
                                  PAGE, self.wide, *p)
        assert got in (0, 1), f"launch: {got}"
        return got, int(self.status)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_a_wait_that_runs_out(launch, fmt):
    call = Call(launch, fmt)
    assert call() == (0, 0)
    out, lse = call.out.clone(), call.lse.clone()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all() and (lse != 0).all()
    ran_out = {}
    for block in (0, 1, 4, 6, 12):
        for warp in range(16):
            for wait in (1, 2, 3, 4, 5, 6, 8, 11, 17, 29, 50):
                got, status = call(block, warp, wait)
                assert status == (TIMEOUT if got else 0), (block, warp, wait)
                ran_out[warp] = ran_out.get(warp, 0) + got
                if not got:  # the warp has no such wait
                    assert torch.equal(call.out, out) and torch.equal(call.lse, lse), (block, warp, wait)
                else:  # the other blocks are through: the last sequence is the last block's
                    assert torch.equal(call.out[-70:], out[-70:]), (block, warp, wait)
        assert call() == (0, 0) and torch.equal(call.out, out) and torch.equal(call.lse, lse)
    assert all(ran_out[w] >= 5 for w in range(16)), ran_out
