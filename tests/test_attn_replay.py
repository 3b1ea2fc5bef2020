"""Parts of the decode attention kernel replayed on the host: its own functions, compiled for the
CPU, that decide which thread writes and reads what."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
BF16, E4M3 = 0, 1
CONFIGS = [(f, dp, nt) for f in (BF16, E4M3) for dp in (64, 128, 192, 256) for nt in (1, 2) if (f, dp, nt) != (E4M3, 256, 2)]


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("replay") / "attn_replay.so")
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-shared", "-o", so, os.path.join(HERE, "attn_replay.cu")], check=True)
    return ctypes.CDLL(so)


def _shape(replay, config):
    x = (ctypes.c_int32 * 3)()
    assert replay.replay_config(*config, x)
    return list(x)  # warps, bytes of the rings, tokens of a tile


@pytest.mark.parametrize("config", CONFIGS)
def test_a_warp_clears_its_own_ring_and_no_other(replay, config):
    """Nothing orders one warp's zeros against the rows and masks that another has copied into its
    ring, so that no thread may write outside its own warp's."""
    warps, size, _ = _shape(replay, config)
    for w in range(warps):
        rings = np.full(size, 0xFF, np.uint8)
        for lane in range(32):
            replay.replay_clear(*config, rings.ctypes.data_as(ctypes.c_void_p), w, lane)
        each = size // warps
        assert (rings[w * each:(w + 1) * each] == 0).all()
        assert (rings[:w * each] == 0xFF).all() and (rings[(w + 1) * each:] == 0xFF).all()


@pytest.mark.parametrize("tile", [16, 32])
@pytest.mark.parametrize("first", [0, 2 ** 31 - 101, 2 ** 31 - 2, 12345])
def test_tokens_next_to_the_longest_length_do_not_wrap(replay, first, tile):
    """A sequence of 2^31 - 1 tokens: the rows of its last unit that lie past it stay past it (a
    negative token would count as one of the sequence's, and be looked up in front of the table)."""
    replay.replay_token.restype = ctypes.c_uint32
    n = 2 ** 31 - 1
    for W in (1, 2, 4, 8):
        last = -(-(n - first) // (W * tile)) - 1
        for u in {0, last // 2, last}:
            got = [replay.replay_token(first, u, W, tw, tile, row) for tw in range(W) for row in range(tile)]
            assert got == [first + u * W * tile + i for i in range(W * tile)]
