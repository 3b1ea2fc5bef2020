"""The prefill's work, dealt out on the host as in test_prefill_replay, with a tile's start counted as each
format and head dim has it."""
import ctypes
import os
import random
import subprocess

import pytest

from tests.test_prefill_replay import HERE, _check

STARTS = {(1, 1): 384, (0, 1): 320, (1, 0): 192, (0, 0): 128}  # (bf16, two halves)


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("replay") / "prefill_replay_start.so")
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-shared", "-o", so, os.path.join(HERE, "prefill_replay_start.cu")], check=True)
    return ctypes.CDLL(so)


def test_starts(replay):
    for (bf16, two_halves), start in STARTS.items():
        assert replay.replay_start_of(bf16, two_halves) == start
        L = ctypes.c_int64
        assert replay.replay_start_in(start, L(152 * 512), L(152)) == start
        assert replay.replay_start_in(start, L(152 * 512 - 1), L(152)) == replay.replay_start_in(start, L(1), L(152)) == 512


@pytest.mark.parametrize("two_halves", [1, 0])
@pytest.mark.parametrize("start", [128, 192, 320, 512])
def test_every_tile_is_dealt_out_once(replay, start, two_halves):
    replay.replay_start(start)
    rows = 256 if two_halves else 128
    rng = random.Random(2 * start + two_halves)
    for _ in range(80):
        B = rng.choice([1, 1, 2, 5, 30])
        new = [rng.choice([0, 1, 2, 7, 40, 129, 300, 700]) for _ in range(B)]
        lens = [n + rng.choice([0, 1, 100, 127, 128, 1000, 5000]) for n in new]
        starts = [3 + sum(new[:b]) for b in range(B + 1)]
        G = rng.choice([1, 2, 3, 5, 8, 12, 16, 100, 128, 130, 256, 300, 600])
        window = rng.choice([0, 0, 1, 60, 128, 500])
        sinks = rng.choice([0, 1, 4, 130, 2000]) if window else 0
        _check(replay, starts, lens, starts[-1] + 2, rng.choice([1, 2, 3]), G, window, sinks, rows, max(lens) + 1,
               rng.choice([1, 3, 20, 152]))
    n = 2 ** 31 - 1
    _check(replay, [0, 37, 74], [n, n - 5], 80, 2, 4, 100, 7, rows, n, 5)
    _check(replay, [0, 3], [n], 3, 1, 8, 0, 0, rows, n, 152)
