"""How the prefill kernel deals out its work, replayed on the host by its own functions, compiled for the
CPU: every tile of keys of every tile of rows is some block's, once, and the parts of a tile that is cut
know of one another."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
FIELDS = "end b kvh head0 heads row0 ntok pos0 len f ns keys kt0 kt1 whole c0 parts".split()


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("replay") / "prefill_replay.so")
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-shared", "-o", so, os.path.join(HERE, "prefill_replay.cu")], check=True)
    return ctypes.CDLL(so)


def _items(replay, starts, lens, T, Hkv, G, window, sinks, rows, longest, blocks):
    """Every block's items, as dicts."""
    a, b = np.asarray(starts, np.int32), np.asarray(lens, np.int32)
    p = lambda x: x.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    bn, total, found = (128 if rows == 256 else 64), ctypes.c_int64(), []
    room = np.zeros((100000, 17), np.int32)
    for block in range(blocks):
        n = replay.replay_items(p(a), p(b), len(lens), T, Hkv, G, window, sinks, rows, longest, bn, blocks, block,
                                ctypes.byref(total), p(room), len(room))
        assert n <= len(room)
        found.append([dict(zip(FIELDS, map(int, x))) for x in room[:n]])
    return found, total.value, bn


def _check(replay, starts, lens, T, Hkv, G, window, sinks, rows, longest, blocks):
    found, total, bn = _items(replay, starts, lens, T, Hkv, G, window, sinks, rows, longest, blocks)
    groups = -(-G // rows)
    heads = -(-G // groups)
    tokens = rows // heads
    whole = (ctypes.c_int * 3)()
    replay.replay_constants(whole)
    tiles = {}
    for block, items in enumerate(found):
        load = 0
        for it in items:
            assert it["kt0"] < it["kt1"] and it["ntok"] * it["heads"] <= rows
            tiles.setdefault((it["b"], it["head0"], it["row0"]), []).append((block, it))
            load += (it["kt1"] - it["kt0"]) * bn + whole[0]
        chunk = max(whole[1], -(-total // blocks))
        assert load <= chunk + 2 * (bn + whole[0]) + whole[2] * bn + sum(bn for _ in items), "a block's share"
    expected = set()
    for b, n in enumerate(lens):
        new = starts[b + 1] - starts[b]
        for kvh in range(Hkv):
            for g in range(groups):
                for m in range(-(-new // tokens)):
                    key = (b, kvh * G + g * heads, starts[b] + m * tokens)
                    expected.add(key)
                    parts = tiles[key]
                    it = parts[0][1]
                    p0 = n - new + m * tokens
                    last = min(n, p0 + tokens)
                    f = max(0, p0 - window + 1) if window else 0
                    ns = min(sinks, f)
                    assert (it["kvh"], it["pos0"], it["len"], it["f"], it["ns"]) == (kvh, p0, n, f, ns)
                    assert it["heads"] == min(heads, G - g * heads) and it["ntok"] == last - p0 and it["keys"] == last - f + ns
                    nkt = -(-it["keys"] // bn)
                    at = 0
                    for i, (block, x) in enumerate(parts):  # one after the other, in neighbouring blocks
                        assert x["kt0"] == at and block == parts[0][0] + i
                        at = x["kt1"]
                        assert x["whole"] == (len(parts) == 1)
                        if len(parts) > 1:
                            assert (x["c0"], x["parts"]) == (parts[0][0], len(parts))
                    assert at == nkt
    assert set(tiles) == expected
    # a block has at most one part that goes on from the block before and one that goes on behind
    for items in found:
        assert all(it["kt0"] == 0 for it in items[1:]) and all(it["whole"] or i in (0, len(items) - 1) for i, it in enumerate(items))


def test_places_in_closed_form(replay):
    rng = random.Random(1)
    got = (ctypes.c_int64 * 2)()
    for _ in range(3000):
        n, old, tokens = rng.choice([1, 5, 300, 4000]), rng.choice([0, 3, 777, 100000]), rng.choice([1, 3, 16, 32, 85, 256])
        window = rng.choice([0, 1, 2, 50, 1000, 2 ** 31 - 1])
        sinks = rng.choice([0, 1, 60, 5000, 2 ** 31 - 1]) if window else 0
        L = ctypes.c_int64
        for m in {0, 1, -(-n // tokens) // 2, -(-n // tokens) - 1, -(-n // tokens)}:
            replay.replay_place(L(n), L(old), L(window), L(sinks), tokens, L(m), got)
            assert got[0] == got[1], (n, old, window, sinks, tokens, m)


def test_every_tile_is_dealt_out_once(replay):
    rng = random.Random(2)
    for _ in range(250):
        B = rng.choice([1, 1, 2, 5, 30])
        new = [rng.choice([0, 1, 2, 7, 40, 129, 300, 700]) for _ in range(B)]
        lens = [n + rng.choice([0, 1, 100, 127, 128, 1000, 5000]) for n in new]
        before = rng.choice([0, 3])
        starts = [before + sum(new[:b]) for b in range(B + 1)]
        G = rng.choice([1, 2, 3, 5, 8, 12, 16, 100, 128, 130, 256, 300, 600])
        window = rng.choice([0, 0, 1, 60, 128, 500])
        sinks = rng.choice([0, 1, 4, 130, 2000]) if window else 0
        _check(replay, starts, lens, starts[-1] + 2, rng.choice([1, 2, 3]), G, window, sinks, rng.choice([128, 256]), max(lens) + 1,
               rng.choice([1, 3, 20, 152]))


def test_the_longest_sequences(replay):
    n = 2 ** 31 - 1
    for window, sinks in ((100, 0), (100, 7), (1, 300)):
        _check(replay, [0, 37, 74], [n, n - 5], 80, 2, 4, window, sinks, 256, n, 5)
    _check(replay, [0, 3], [n], 3, 1, 8, 0, 0, 256, n, 152)


def test_bad_starts_and_lengths_stay_inside_the_tensors(replay):
    rng = random.Random(3)
    bad = [-2 ** 31, -5, -1, 0, 1, 7, 60, 100, 129, 130, 2 ** 31 - 1]
    for _ in range(500):
        B, T, longest = rng.choice([1, 3, 6]), 129, rng.choice([0, 64, 200])
        starts, lens = [rng.choice(bad) for _ in range(B + 1)], [rng.choice(bad) for _ in range(B)]
        window = rng.choice([0, 50])
        found, _, bn = _items(replay, starts, lens, T, 2, 8, window, rng.choice([0, 9]) if window else 0, 256, longest, 20)
        for it in sum(found, []):
            assert 0 <= it["b"] < B and 0 <= it["row0"] and it["row0"] + it["ntok"] <= T and it["ntok"] > 0
            assert 0 <= it["len"] <= longest and 0 <= it["kt0"] < it["kt1"] <= -(-it["keys"] // bn)
            assert it["f"] >= 0 and 0 <= it["ns"] <= it["f"] and 0 <= it["c0"] and it["c0"] + it["parts"] <= 20
