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


def _deal(replay, lens, Hkv, groups, window, tile_log, wlog, teams):
    """Every team's units, as the kernel deals them out."""
    unit, start, whole = 1 << (tile_log + wlog), replay.replay_start(wlog), replay.replay_whole(wlog)
    c_lens = (ctypes.c_int32 * len(lens))(*lens)
    nu = [-(-(min(n, window) if window else n) // unit) for n in lens]
    places = [(x + start) * Hkv * groups if x else 0 for x in nu]
    first, total = [sum(places[:b]) for b in range(len(lens))], sum(places)
    chunk = max(1, -(-total // teams))
    most = total + 4
    got, buf = [], (ctypes.c_int32 * (4 * most))()
    for team in range(teams):
        unit0 = team * chunk
        if unit0 >= total:
            got.append([])
            continue
        b = max(i for i in range(len(lens)) if places[i] and first[i] <= unit0)
        n = replay.replay_team(c_lens, len(lens), Hkv, groups, window, 2 ** 31 - 1, tile_log, wlog, whole, start, b,
                               ctypes.c_int64(unit0 - first[b]), min(total - unit0, chunk), buf, most)
        assert n <= most
        got.append([tuple(buf[4 * i:4 * i + 4]) for i in range(n)])
    return got, nu, whole


@pytest.mark.parametrize("wlog", [0, 1, 2, 3])
@pytest.mark.parametrize("kind", ["short", "mixed", "long", "window"])
def test_every_unit_is_dealt_to_one_team(replay, kind, wlog):
    """Random batches: each unit of each (sequence, key head, head group) is taken once, in order;
    a sequence of few units by one team; the teams of a cut one follow each other."""
    rng = np.random.default_rng([11, wlog, len(kind)])
    for it in range(60):
        tile_log = 4 + it % 2
        unit = 1 << (tile_log + wlog)
        B = int(rng.integers(1, 90))
        top = dict(short=unit, mixed=6 * unit, long=40 * unit, window=9 * unit)[kind]
        lens = [int(x) for x in rng.integers(0, top + 1, B)]
        if it % 5 == 0:
            lens = [min(top, unit)] * B  # all alike: borders fall on every place of a start
        window = int(rng.integers(1, 3 * unit)) if kind == "window" else 0
        Hkv, groups = int(rng.integers(1, 5)), int(rng.integers(1, 3))
        teams = int(rng.choice([1, 3, 19, 152, 304, 1216]))
        got, nu, whole = _deal(replay, lens, Hkv, groups, window, tile_log, wlog, teams)
        assert [u for team in got for u in team] == [(b, h, g, u) for b in range(B) for h in range(Hkv)
                                                     for g in range(groups) for u in range(nu[b])], (it, teams)
        for team in got:  # what is not cut comes whole
            for b, h, g, u in team:
                if nu[b] <= whole:
                    assert all((b, h, g, i) in team for i in range(nu[b]))


def test_short_sequences_at_every_border_are_dealt_once(replay):
    """As many one-unit sequences as there are teams, and some more and less: a team's range may
    begin at each place of a start."""
    for wlog in (0, 1, 2, 3):
        unit = 1 << (5 + wlog)
        for B in (50, 200, 402, 700):
            got, _, _ = _deal(replay, [unit] * B, 1, 1, 0, 5, wlog, 304)
            assert sum(len(t) for t in got) == B
