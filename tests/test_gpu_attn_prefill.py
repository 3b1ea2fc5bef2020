"""The attention of many new tokens per sequence on the GPU against a plain 64-bit form.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of fp32 2^-24."""
import math

import pytest

from tests import _attn_more_ref as more
from tests import _attn_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16_HALF = 2.0 ** -8
FORMATS = ["bf16", "e4m3", "mxfp4"]


@pytest.fixture(scope="module")
def attn():
    import __graft_entry__ as g
    g.build()
    from mxfp4_routed_expert_latentmoe_gb300 import attn as mod
    torch.cuda.set_device(0)
    return mod


def _randn(*shape, seed, size=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (size * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


class Call:
    """A prefill call: sequences of (new tokens, cached tokens) in a cache that is NaN everywhere else;
    `before` and `behind`: rows of no sequence."""

    def __init__(self, attn, sizes, page, fmt, Hq, Hkv, D, window=0, sinks=0, seed=70, order="phtd", before=0, behind=0,
                 q_size=2.0, spread=0.5, k=None, v=None, room=0, scale=None):
        self.attn, self.sizes, self.sinks, self.before = attn, sizes, sinks, before
        self.d = attn.dims(Hq, Hkv, D, rot_dim=0, window=window, softmax_scale=scale)
        self.s = more.Sequences(attn, self.d, [n for _, n in sizes], page, fmt, seed, order=order, spread=spread, k=k, v=v,
                                room=room)
        self.ws = attn.workspace(self.d, prefill=True)
        T = before + behind + sum(n for n, _ in sizes)
        self.q = self.s.queries(T, q_size)
        starts = torch.tensor([before] + [n for n, _ in sizes]).cumsum(0)
        self.starts = starts.to(torch.int32).cuda()
        self.out = torch.full((T, Hq, D), 7.0, device="cuda", dtype=torch.bfloat16)
        self.lse = torch.full((T, Hq), 7.0, device="cuda")

    def run(self, **kw):
        a = dict(q=self.q, q_starts=self.starts, cache=self.s.cache, page_table=self.s.table, lens=self.s.lens_t,
                 out=self.out, ws=self.ws, lse=self.lse, sinks=self.sinks)
        a.update(kw)
        self.attn.prefill(self.d, **a)
        return self

    def check(self, most_rows=24):
        """Every sequence at up to `most_rows` of its new tokens (the first and last ones among them)."""
        assert self.attn.device_status(self.ws) == 0
        d, row = self.d, self.before
        assert (self.out[:row] == 7).all() and (self.lse[:row] == 7).all()
        out, lse = self.out.double().cpu(), self.lse.double().cpu()
        q = self.q.double().cpu()
        for b, (new, n) in enumerate(self.sizes):
            k, v = self.s.rows(b, list(range(n)))
            step = max(1, new // most_rows)
            for i in sorted(set(range(0, new, step)) | {new - 1} if new else ()):
                which = more.seen(n, d.window, self.sinks, n - new + i)
                o, z, mean_abs, slack = ref.decode(q[row + i], k[which], v[which], d.softmax_scale)
                count = len(which)
                # weights rounded to bf16 at most with the logits' fp32 error in their exponents (twice),
                # sums in fp32; the result rounded to bf16.  (A weight below fp32's normal numbers, 2^-126,
                # is lost: 4 bits hold zeros beside which it would show)
                tiny = 2.0 ** -125 * count * (v[which].abs().amax() if count else 0)
                tol = tiny + BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + (64 + count / 8) * 2.0 ** -24)
                off = (out[row + i] - o).abs()
                assert (off <= tol).all(), f"sequence {b} of {new} in {n}, token {i}: {float((off - tol).max()):.3e} over"
                if count == 0:
                    assert (lse[row + i] == -torch.inf).all()
                else:
                    bound = slack + (64 + count / 8) * 2.0 ** -24 + 2.0 ** -22 * z.abs()
                    assert ((lse[row + i] - z).abs() <= bound).all(), f"lse: sequence {b}, token {i}"
            row += new
        assert (self.out[row:] == 7).all() and (self.lse[row:] == 7).all()
        return self

    def check_same(self):
        """The same call again: the same bits (the workspace is left ready)."""
        out, lse = torch.zeros_like(self.out), torch.zeros_like(self.lse)
        self.run(out=out, lse=lse)
        r = slice(int(self.starts[0]), int(self.starts[-1]))
        assert torch.equal(out[r].view(torch.int16), self.out[r].view(torch.int16)) and torch.equal(lse[r], self.lse[r])
        out.zero_()
        self.run(out=out, lse=None)
        assert torch.equal(out[r].view(torch.int16), self.out[r].view(torch.int16))


MIXED = [(1, 1), (0, 0), (3, 3), (17, 40), (0, 25), (128, 128), (129, 129), (64, 1000), (1, 777), (300, 300), (31, 32)]
CASES = [  # Hq, Hkv, D, page, window, sinks, order, sizes
    (1, 1, 32, 1, 0, 0, "phtd", [(1, 1)]), (8, 8, 64, 16, 0, 0, "phtd", MIXED), (8, 1, 128, 16, 0, 0, "phtd", MIXED),
    (64, 8, 128, 64, 0, 0, "phtd", [(700, 700), (0, 0), (2, 5000)]), (6, 2, 96, 7, 0, 0, "pthd", MIXED),
    (24, 2, 256, 24, 0, 0, "phtd", MIXED), (36, 3, 192, 24, 100, 4, "hptd", MIXED), (5, 1, 160, 3, 17, 1, "tphd", MIXED),
    (16, 1, 64, 128, 0, 0, "phtd", [(515, 4097)]), (34, 2, 128, 16, 64, 64, "phtd", MIXED),
    (40, 1, 256, 32, 0, 0, "phtd", [(77, 513), (5, 5)]), (7, 7, 32, 16, 1, 1, "phtd", MIXED), (9, 3, 224, 5, 64, 130, "phtd", MIXED),
    (2, 1, 128, 32, 0, 0, "phtd", [(3, 70001)]), (8, 2, 128, 64, 0, 0, "phtd", [(0, 0), (0, 10)]),
    (16, 8, 64, 16, 0, 0, "phtd", [(3 * i % 23, 3 * i % 23 + 5 * i % 97) for i in range(300)]),
    (100, 1, 64, 16, 30, 2, "phtd", [(70, 200), (1, 1)]), (300, 1, 64, 16, 0, 0, "phtd", [(5, 130), (2, 2)]),
    (1024, 2, 32, 16, 0, 0, "phtd", [(3, 50)]), (12, 4, 128, 64, 128, 0, "phtd", [(1300, 1300)]),
    (4, 4, 128, 100, 500, 31, "phtd", [(900, 2500)])]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,D,page,window,sinks,order,sizes", CASES,
                         ids=[f"{c[0]}x{c[1]}x{c[2]}-p{c[3]}-w{c[4]}-s{c[5]}-{c[6]}-{len(c[7])}" for c in CASES])
def test_prefill(attn, Hq, Hkv, D, page, window, sinks, order, sizes, fmt):
    c = Call(attn, sizes, page, fmt, Hq, Hkv, D, window, sinks, order=order, before=2, behind=3)
    c.run().check().check_same()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [16, 48, 80, 112, 144, 176, 208, 240])
def test_head_dims_of_any_multiple_of_16(attn, D, fmt):
    c = Call(attn, [(40, 333), (300, 300)], 16, fmt, 6, 2, D, window=100 if D % 32 else 0, sinks=3)
    nan = Call(attn, [(40, 333), (300, 300)], 16, fmt, 6, 2, 256, seed=71)
    nan.s.cache.k.view(torch.uint8).fill_(0xFF)
    nan.s.cache.v.view(torch.uint8).fill_(0xFF)
    for _ in range(3):  # whatever an earlier call (of NaN rows) has left in shared and tensor memory
        nan.run()
        c.run()
    assert torch.isnan(nan.out).all()
    c.check().check_same()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 40), (40, 1), (128, 128), (100, 4), (64, 500), (257, 3), (500, 31)])
def test_windows_and_sinks(attn, fmt, window, sinks):
    """Sinks that end inside a tile, a page, the window, behind the sequence; windows that end inside a
    tile of queries and of keys."""
    for Hq, Hkv, D, page in ((8, 2, 128, 5), (6, 1, 64, 64)):
        sizes = [(1, 1), (33, 64 + window), (200, 200), (64, 1060), (7, 997), (450, 1500)]
        Call(attn, sizes, page, fmt, Hq, Hkv, D, window, sinks, room=9).run().check().check_same()


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_new_token_is_decode(attn, fmt):
    """Calls of one new token a sequence against the decode operator, as near as two orders of sums
    and two roundings of the weights are."""
    sizes = [(1, n) for n in (1, 2, 17, 64, 129, 1000, 3000)]
    c = Call(attn, sizes, 16, fmt, 16, 2, 128, window=700, sinks=5).run().check()
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    attn.decode(c.d, c.q, c.s.cache, c.s.table, c.s.lens_t, out, c.ws, lse=lse, sinks=5)
    assert ((out.float() - c.out.float()).abs() <= 4 * BF16_HALF * (1 + out.float().abs())).all()
    assert ((lse - c.lse).abs() <= 2.0 ** -12).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_prompt_in_chunks_is_the_prompt(attn, fmt):
    """Each row depends on its own position alone: the prompt at once and in chunks."""
    n = 700
    c = Call(attn, [(n, n)], 16, fmt, 8, 2, 128, window=300, sinks=2).run().check()
    for at, end in ((0, 1), (1, 130), (130, 600), (600, n)):
        out, lse = torch.zeros_like(c.out[at:end]), torch.zeros_like(c.lse[at:end])
        c.run(q=c.q[at:end], q_starts=torch.tensor([0, end - at], device="cuda", dtype=torch.int32),
              lens=torch.tensor([end], device="cuda", dtype=torch.int32), out=out, lse=lse)
        assert ((out.float() - c.out[at:end].float()).abs() <= 4 * BF16_HALF * (1 + out.float().abs())).all()
        assert ((lse - c.lse[at:end]).abs() <= 2.0 ** -12).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_sharp_logits_and_values_of_many_sizes(attn, fmt):
    for q_size, spread in ((60.0, 0.5), (2.0, 4.0), (20.0, 4.0)):
        Call(attn, [(3, 3), (70, 200), (130, 900)], 16, fmt, 16, 2, 128, q_size=q_size, spread=spread).run().check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [1e3, 1e5, 1e7, 1e10, 1e13])
def test_logits_of_any_finite_size(attn, size, fmt):
    """Logits so large that one token takes all (the next one is further off than twice their fp32
    error): the result is that token's value, rounded once (a value's scale may round its weight)."""
    sizes, H, D = [(1, 1), (30, 70), (33, 33)], 2, 64
    T = sum(n for _, n in sizes)
    k = _randn(T, H, D, seed=61, size=size ** 0.5)
    v = (torch.exp(2 * _randn(T, H, 1, seed=62).float()) * _randn(T, H, D, seed=63).float()).to(torch.bfloat16)
    c = Call(attn, sizes, 16, fmt, 8, H, D, q_size=size ** 0.5, k=k, v=v).run()
    q, out, lse, row, seen = c.q.double().cpu(), c.out.double().cpu(), c.lse.double().cpu(), 0, 0
    for b, (new, n) in enumerate(sizes):
        kk, vv = c.s.rows(b, list(range(n)))
        for i in range(new):
            which = n - new + i + 1
            _, z, _, slack = ref.decode(q[row + i], kk[:which], vv[:which], c.d.softmax_scale)
            for h in range(8):
                logits = c.d.softmax_scale * (kk[:which, h // 4] @ q[row + i, h])
                top, where = logits.max(0)
                rest = logits[torch.arange(which) != where]
                if which > 1 and float(top - rest.max()) < 2 * float(slack[h]) + 60:
                    continue
                seen += 1
                want = vv[where, h // 4]
                # (the others' weights, e^-60 each at most, show beside a zero)
                rest = which * math.exp(-60.0) * vv[:which, h // 4].abs().amax()
                assert ((out[row + i, h] - want).abs() <= (2 * BF16_HALF + 2.0 ** -16) * want.abs() + rest).all(), (b, i, h)
                assert abs(float(lse[row + i, h]) - float(z[h])) <= float(slack[h]) + 2.0 ** -22 * abs(float(z[h])) + 2.0 ** -18
        row += new
    assert seen >= 8


def test_rows_without_weight_and_non_finite_tokens(attn):
    c = Call(attn, [(20, 40), (20, 40), (20, 40)], 16, "bf16", 4, 2, 64)
    c.q[:20] = c.q[:20].abs() + 0.1
    at = [(s // 16).long() for s in c.s.slots], [(s % 16).long() for s in c.s.slots]
    c.s.cache.k[at[0][0], :, at[1][0]] = float("-inf")  # sequence 0: every logit is -infinity
    c.s.cache.k[at[0][1][30], 0, at[1][1][30], 0] = float("nan")  # sequence 1: in key head 0, from position 30 on
    c.s.cache.v[at[0][2][25], 1, at[1][2][25], 5] = float("nan")  # sequence 2: dim 5 of value head 1, from 25 on
    c.run()
    out, lse = c.out.float().cpu(), c.lse.cpu()
    assert (out[:20] == 0).all() and (lse[:20] == -torch.inf).all()
    assert torch.isfinite(out[20:30]).all() and torch.isnan(out[30:40, :2]).all() and torch.isnan(lse[30:40, :2]).all()
    assert torch.isfinite(out[30:40, 2:]).all()
    hit = torch.zeros(20, 4, 64, dtype=torch.bool)
    hit[5:, 2:, 5] = True
    assert torch.equal(torch.isnan(out[40:]), hit) and torch.isfinite(lse[40:]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp4"])
def test_scales_that_are_zero_nan_or_extreme(attn, fmt):
    """Values whose scales lie near the ends of fp32's range, zero scales (E4M3), NaN scales."""
    n, H, D = 60, 2, 64
    v = (_randn(n, H, D, seed=64).float() * torch.tensor([1e30, 1e-28], device="cuda")[None, :, None]).to(torch.bfloat16)
    c = Call(attn, [(20, n)], 16, fmt, 4, H, D, v=v).run().check()
    pg, at = (c.s.slots[0] // 16).long(), (c.s.slots[0] % 16).long()
    if fmt == "e4m3":
        c.s.cache.v_scale[pg[:20], :, at[:20]] = 0.0
        c.s.cache.k_scale[pg[5:10], :, at[5:10]] = 0.0
        c.run().check()
        c.s.cache.v_scale[pg[50], 1, at[50]] = float("nan")
    else:
        c.s.cache.v_scale[pg[50], 1, at[50], 1] = 255
    c.run()
    out = c.out.float().cpu()
    hit = torch.zeros(20, 4, D, dtype=torch.bool)
    hit[10:, 2:, (32 if fmt == "mxfp4" else 0):] = True
    assert torch.equal(torch.isnan(out), hit) and torch.isfinite(c.lse).all()


def test_bad_pages_lengths_and_starts_are_reported(attn):
    c = Call(attn, [(60, 100), (64, 64), (5, 50)], 16, "e4m3", 8, 2, 128)
    c.run().check()
    table = c.s.table.clone()
    c.s.table[0, 2], c.s.table[0, 4] = -3, c.s.cache.n_pages
    c.run()
    assert attn.device_status(c.ws) == attn.DEV_BAD_PAGE
    keep = [t for t in range(100) if t // 16 not in (2, 4)]
    k, v = c.s.rows(0, keep)
    o, _, mean_abs, slack = ref.decode(c.q[59].double().cpu(), k, v, c.d.softmax_scale)
    tol = BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + 80 * 2.0 ** -24)
    assert ((c.out[59].double().cpu() - o).abs() <= tol).all()
    attn.workspace_init(c.ws)
    c.s.table = table
    # lengths outside the table, fewer cached tokens than new ones
    table[2] = table[1, 0]
    c.s.lens_t.copy_(torch.tensor([2 ** 31 - 1, -5, 3]))
    table[0] = table[1, 0]
    c.run()
    assert attn.device_status(c.ws) == attn.DEV_BAD_LENGTH
    assert torch.isfinite(c.out[:60]).all()
    assert (c.out[60:126] == 0).all() and (c.lse[60:126] == -torch.inf).all() and torch.isfinite(c.lse[126:]).all()
    # starts that fall, and that leave the rows: nothing outside the tensors is touched
    c.s.lens_t.copy_(torch.tensor([64, 64, 64]))
    for starts in ([0, 60, 30, 129], [-5, 60, 124, 129], [0, 60, 124, 2 ** 31 - 1], [50, 20, 10, 0], [-2 ** 31, 2 ** 31 - 1, 0, 129]):
        attn.workspace_init(c.ws)
        c.run(q_starts=torch.tensor(starts, device="cuda", dtype=torch.int32))
        assert attn.device_status(c.ws) & attn.DEV_BAD_LENGTH
    attn.workspace_init(c.ws)


@pytest.mark.parametrize("fmt", FORMATS)
def test_the_longest_sequences(attn, fmt):
    """Positions up to 2^31 - 3 over pages that repeat: the window's tokens and the sinks, as a short
    sequence of the same rows gives them."""
    page, wide, D, G, new = 49981, 42966, 64, 4, 37
    n = page * wide
    k, v, q = _randn(2 * page, 1, D, seed=51), _randn(2 * page, 1, D, seed=52), _randn(2 * new, G, D, seed=50)
    starts = torch.tensor([0, new, 2 * new], device="cuda", dtype=torch.int32)
    for window, sinks in ((100, 7), (257, 300)):
        d = attn.dims(G, 1, D, rot_dim=0, window=window)
        cache = attn.KVCache.empty(d, 2, page, fmt)
        ws = attn.workspace(d, prefill=True)
        attn.kv_write(d, k, v, torch.arange(2 * page, device="cuda", dtype=torch.int32), cache, ws)
        table = torch.zeros(2, wide, device="cuda", dtype=torch.int32)
        table[:, -1] = 1
        got = []
        for t, lens in ((table, [n, n - 30]), (table[:, -2:].contiguous(), [2 * page, 2 * page - 30])):
            out, lse = torch.zeros(2 * new, G, D, device="cuda", dtype=torch.bfloat16), torch.zeros(2 * new, G, device="cuda")
            attn.prefill(d, q, starts, cache, t, torch.tensor(lens, device="cuda", dtype=torch.int32), out, ws, lse=lse,
                         sinks=sinks)
            got.append((out, lse))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert torch.isfinite(got[0][1]).all() and attn.device_status(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_a_cache_past_32_bits(attn, fmt):
    """Pages whose bytes lie past 2^32 (only the used ones are filled)."""
    d = attn.dims(8, 4, 128)
    page, n = 256, 600
    n_pages = 70000 if fmt == "mxfp4" else 17000
    widths = [64, 64, 4, 4] if fmt == "mxfp4" else [128, 128]
    dtype = torch.uint8 if fmt == "mxfp4" else torch.bfloat16
    cache = attn.KVCache(d, *(torch.empty(n_pages, 4, page, w, dtype=dtype, device="cuda") for w in widths))
    ws = attn.workspace(d, prefill=True)
    table = torch.tensor([[n_pages - 1, 5, n_pages - 2]], device="cuda", dtype=torch.int32)
    t = torch.arange(n, device="cuda")
    slots = (table[0].long()[t // page] * page + t % page).to(torch.int32)
    kk, vv, q = _randn(n, 4, 128, seed=25), _randn(n, 4, 128, seed=26), _randn(40, 8, 128, seed=27)
    attn.kv_write(d, kk, vv, slots, cache, ws)
    out = torch.empty(40, 8, 128, device="cuda", dtype=torch.bfloat16)
    attn.prefill(d, q, torch.tensor([0, 40], device="cuda", dtype=torch.int32), cache, table,
                 torch.tensor([n], device="cuda", dtype=torch.int32), out, ws)
    rows = [more.gather(cache, x, slots) for x in ("k", "v")]
    for i in (0, 39):
        o, _, mean_abs, slack = ref.decode(q[i].double().cpu(), rows[0][:561 + i], rows[1][:561 + i], d.softmax_scale)
        tol = BF16_HALF * o.abs() + mean_abs * (BF16_HALF + 2 * slack[:, None] + 139 * 2.0 ** -24)
        assert ((out[i].double().cpu() - o).abs() <= tol).all()
    assert attn.device_status(ws) == 0


def test_a_captured_call_replays_with_new_starts_and_lengths(attn):
    c = Call(attn, [(30, 130), (1, 1), (7, 77)], 16, "mxfp4", 16, 4, 128, window=64, sinks=4, room=4)
    c.s.table[:, :] = torch.where((c.s.table < 0) | (c.s.table >= c.s.cache.n_pages), c.s.table[:, :1], c.s.table)
    c.run().check()
    want = c.out.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)
    c.starts.copy_(torch.tensor([2, 3, 3, 38], dtype=torch.int32))
    c.s.lens_t.copy_(torch.tensor([64, 0, 40], dtype=torch.int32))
    c.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    out, lse = torch.full_like(c.out, 7.0), torch.empty_like(c.lse)
    c.run(out=out, lse=lse)
    assert torch.equal(c.out, out) and (out[:2] == 7).all() and torch.isfinite(out).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.full_like(c.out, 7.0)
    c.run(out=other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, out) and attn.device_status(c.ws) == 0


def test_two_calls_at_once_with_workspaces_of_their_own(attn):
    a = Call(attn, [(300, 900), (20, 20)], 16, "bf16", 16, 2, 128, seed=80).run().check()
    b = Call(attn, [(5, 4000), (500, 500)], 64, "e4m3", 8, 8, 64, seed=81).run().check()
    want = a.out.clone(), b.out.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        a.run(stream=streams[0])
        b.run(stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_one_workspace_serves_decode_and_prefill_of_other_shapes(attn):
    ws = attn.workspace(attn.dims(64, 2, 256), prefill=True)
    for Hq, Hkv, D, fmt in ((64, 2, 256, "bf16"), (4, 4, 64, "e4m3"), (16, 2, 128, "mxfp4")):
        c = Call(attn, [(5, 3000), (100, 130)], 16, fmt, Hq, Hkv, D)
        c.ws = ws
        for _ in range(2):
            c.run().check()
            out = torch.empty(2, Hq, D, device="cuda", dtype=torch.bfloat16)
            attn.decode(c.d, c.q[[4, 104]], c.s.cache, c.s.table, c.s.lens_t, out, ws)
            assert ((out.float() - c.out[[4, 104]].float()).abs() <= 4 * BF16_HALF * (1 + out.float().abs())).all()


def test_append_prefill_decode_as_a_server_runs_them(attn):
    """A prompt's append and prefill, then steps of append and decode: each step's attention is what
    prefill gives for the same tokens in one call."""
    for fmt in FORMATS:
        d = attn.dims(8, 2, 128, window=90, softmax_scale=0.1)
        n, steps, page = 150, 6, 16
        cache = attn.KVCache.empty(d, 12, page, fmt)
        ws = attn.workspace(d, prefill=True)
        x = _randn(n + steps, 12, 128, seed=90)
        table = torch.randperm(12, device="cuda").to(torch.int32)[:10].view(1, 10)
        t = torch.arange(n + steps, device="cuda", dtype=torch.int32)
        slots = table[0][(t // page).long()] * page + t % page
        w, freq = torch.ones(128, device="cuda"), attn.rope_frequencies(128)
        q = torch.empty(n + steps, 8, 128, device="cuda", dtype=torch.bfloat16)
        out = torch.empty_like(q)

        def tensor(*v):
            return torch.tensor(v, device="cuda", dtype=torch.int32)

        def append(a, b):
            attn.kv_append(d, x[a:b, :8], x[a:b, 8:10], x[a:b, 10:], t[a:b], slots[a:b], freq, w, w, cache, q[a:b], ws)

        append(0, n)
        attn.prefill(d, q[:n], tensor(0, n), cache, table, tensor(n), out[:n], ws, sinks=3)
        for i in range(n, n + steps):
            append(i, i + 1)
            attn.decode(d, q[i:i + 1], cache, table, tensor(i + 1), out[i:i + 1], ws, sinks=3)
        whole = torch.empty_like(out)
        attn.prefill(d, q, tensor(0, n + steps), cache, table, tensor(n + steps), whole, ws, sinks=3)
        assert ((out.float() - whole.float()).abs() <= 4 * BF16_HALF * (1 + out.float().abs())).all()
        assert attn.device_status(ws) == 0


def test_tensors_that_do_not_fit_are_refused_before_a_launch(attn):
    from mxfp4_routed_expert_latentmoe_gb300 import K3MoEError
    c = Call(attn, [(3, 20), (2, 5)], 16, "e4m3", 4, 2, 64)
    for bad in (dict(q=c.q.float()), dict(q=c.q.cpu()), dict(q=c.q[:4]), dict(q_starts=c.starts.long()), dict(q_starts=c.starts[:2]),
                dict(q_starts=c.starts[:0]), dict(q_starts=c.starts.cpu()), dict(page_table=c.s.table[:1]), dict(page_table=c.s.table[0]),
                dict(page_table=c.s.table.long()), dict(lens=c.s.lens_t[:1]), dict(lens=None), dict(out=c.out[:4]), dict(out=c.out.half()),
                dict(lse=c.lse.half()), dict(lse=c.lse[:1]), dict(ws=c.ws.float()), dict(cache=attn.KVCache.empty(attn.dims(4, 2, 128), 2, 16)),
                dict(sinks=2 ** 31)):
        with pytest.raises(ValueError):
            c.run(**bad)
    for bad, code in ((dict(ws=c.ws[:256]), 4), (dict(sinks=-1), 1)):
        with pytest.raises(K3MoEError) as e:
            c.run(**bad)
        assert e.value.code == code
    torch.cuda.synchronize()
    assert (c.out == 7.0).all() and attn.device_status(c.ws) == 0
    c.run(q=c.q[:0], out=c.out[:0], lse=None)  # no tokens
    c.run(q_starts=c.starts[:1], page_table=c.s.table[:0], lens=c.s.lens_t[:0])  # no sequences
    torch.cuda.synchronize()
    assert (c.out == 7.0).all()
