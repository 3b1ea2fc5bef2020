// k3_prefill.cuh -- attention of many new tokens per sequence over the paged key-value cache.
//
// One pass over the keys with a running maximum and sum, on the tensor cores: a tile is 256 rows
// (128 for head dims past 128), the query heads of one key head times some tokens, so that a row of
// keys is read once for all of them.  Per tile of 128 keys (64 past 128 dims) and 128 rows:
//   S = Q K^T       128 x 128 in tensor memory
//   P = 2^(S - m)   rounded to bf16, over S in tensor memory
//   O += P V        128 x D in tensor memory
// Warps: 0-3 and 4-7 the softmax of a tile's two halves, a row a thread (the tensor core works on one
// half while the other's weights are formed); 8-13 bring keys and values, as bf16, into shared
// memory, row by row through the page table (any page size, any strides); 14 says which tile is
// next; 15 issues the products.
//
// The work, tiles times keys, stands in a line (each tile's start counts as some keys, pre_start) and is
// dealt out evenly to the blocks, whatever the lengths and masks; a tile that is cut leaves an
// unnormalised record of each part in the workspace, and the part that arrives last joins them, in
// order.
//
// Codes become bf16 on their way: E2M1 times its power of two is a bf16 number, E4M3 codes are, and a
// row's E4M3 scale multiplies its column of logits, or of weights (in fp32, before they are rounded).
// Rounded to fewer bits: a weight to bf16, whose range takes values of any size (fp16 would need a
// maximum of its own for them); both operands of a product have one type, and the result is rounded
// to bf16 anyway (8192-token prompt: results off by 2.2e-3 in the mean square, 1.65e-3 with fp32 weights).
//
// What bounds it (GB300, clocks a tile of 128 keys and 256 rows of 128 dims, measured with clock reads in
// a copy).  bf16, 8192-token prompt, 64 query and 8 key heads: 1.02 ms, 1075 TFLOP/s, 57% of the burst
// rate; the products take 2048 clocks of 4900, the rest is the chain of a half: from logits to the first
// weights 1500, to the last 2500 (maximum 700, then 32 logits at a time; the two halves' warps share the
// issue slots, neither pipe is full), then its turn at the tensor core; and a tile's start, some 14000 clocks
// (queries once the last products are through, the sums' way out; pre_start).  Codes: the copying warps (a chunk of
// 1500 behind 30001 tokens, MXFP4: 1.91 ms, 42% of the rate; of 6440 clocks 2500 are conversion and 2100 addresses
// and copies; E4M3 in a window of 1000: 0.56 ms), and for few rows (drafts: 200 us) the chain of one half.
// Ten copying warps of 64 registers instead of six of 96 were 6 to 20% slower, rows of codes as bulk
// copies of a row each (some 85 clocks to issue one) 35%.
#pragma once

#include "k3_decode.cuh"
#include "k3_tmem.cuh"

namespace k3 {

// What a tile's start counts as, in keys.  A tile of n tiles of keys (windowed prompts, 8 query heads a key
// head) takes, in us: bf16 of 64 dims 5.5 + 2.33 n, 128 dims 6.7 + 2.69 n, 192 dims 3.6 + 1.86 n, 256 dims 3.2 + 2.31 n;
// E4M3 5.5 + 2.84 n, 6.5 + 3.64 n, 4.7 + 2.65 n, 4.3 + 3.13 n; MXFP4 6.5 + 3.03 n, 9.6 + 3.16 n, 4.7 + 2.97 n, 4.8 + 3.04 n:
// 230 to 390 keys with two halves, 90 to 120 with one.  Measured best: somewhat more, as a block's
// first tile has none of its start hidden (8192-token prompts, 64/8 heads, us: bf16 of 128 dims 1093, 1049,
// 1025, 1027, 1045 at 256, 320, 384, 512, 768 keys, of 192 dims 2866, 2729, 2627, 2642, 2690 at 64, 128, 192, 256, 384;
// E4M3 of 128 dims 1780, 1708, 1713, 1724, 1747 at 128, 256, 320, 384, 512; six E4M3 prompts of up to 3000,
// 192 dims: 873, 809, 844, 859 at 64, 128, 192, 256).
constexpr int PRE_START = 384;
K3_HD constexpr int pre_start(bool bf16, bool two_halves) { return two_halves ? (bf16 ? PRE_START : 320) : (bf16 ? 192 : 128); }
// The fewest keys of a block: where the work gives them less, tiles have a block each, and only what is longer is cut
// (128: 4 tokens behind 8000, 32/8 heads of 128, bf16 87 us, 77 at 512; 1024: 8 single tokens behind 500 34 us, 28).
// Tiles of keys up to which a tile is not cut, as its join would take longer (1: 8192 tokens and less
// as at 2; 4: up to 30% less for tiles of 3 and 4, 700 tokens of 256 dims 62 us instead of 49).
constexpr int PRE_LEAST = 512, PRE_WHOLE = 2;
static_assert(PRE_LEAST >= 128, "a block without a tile of keys in the middle of a tile's");
constexpr int PRE_MAX_BLOCKS = 192;

struct PrefillParams {
  const uint16_t* q;
  int64_t q_stride;
  int32_t B, T, Hq, Hkv, G, D, window, sinks;
  int32_t groups, heads, tokens;  // head groups of a key head, heads of each, tokens of a tile
  float scale;                    // softmax_scale * log2(e): logits in powers of two
  CacheView c;
  const int32_t *starts, *table, *lens;
  int32_t table_width;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  uint32_t* arrived;  // two counters a block, zero between calls
  float* parts;       // two records a block
  int32_t boxes;      // whether rows of bf16 may come in boxes of 8 tokens of a page
  int32_t start = PRE_START;
};
struct PrefillMaps {
  CUtensorMap k, v;  // dims, tokens of a page, heads, pages
};

constexpr int PRE_COPY_WARPS = 6, PRE_THREADS = 256 + 32 * PRE_COPY_WARPS + 64;
// Registers of a thread: at the launch, then of the 256 of the softmax and of the others
constexpr int PRE_REGS = 128, PRE_REGS_SOFTMAX = 160, PRE_REGS_OTHERS = 96;
static_assert(PRE_THREADS == 512 && PRE_REGS_SOFTMAX + PRE_REGS_OTHERS <= 2 * PRE_REGS, "a warp would wait for ever");

// ---------------------------------------------------------------------------- the order of the work
K3_HD int64_t pre_min(int64_t a, int64_t b) { return a < b ? a : b; }
K3_HD int64_t pre_max(int64_t a, int64_t b) { return a > b ? a : b; }

// A sequence's tiles (of one head group): n new tokens behind `old` ones, TT tokens a tile.  Its keys in
// order: the sinks in front of the first token's window, then that window's and the rest.
struct PreSeq {
  int64_t n, old, W, S;
  int32_t TT, start = PRE_START;
  K3_HD int64_t tiles() const { return (n + TT - 1) / TT; }
  K3_HD int64_t keys(int64_t m) const {
    const int64_t p0 = old + m * TT, p1 = old + pre_min(n, (m + 1) * TT), f = W > 0 ? pre_max(0, p0 - W + 1) : 0;
    return p1 - f + pre_min(S, f);
  }
  // the place of tile m's start, counted from tile 0's: the keys of full tiles in closed form (up to
  // tile x the window's first token is no further than the sinks: all tokens are keys)
  K3_HD int64_t place(int64_t m) const {
    if (n <= 0) return 0;
    const int64_t all = tiles(), full = m < all ? m : all - 1;
    int64_t x = full;
    if (W > 0) {
      const int64_t t = S + W - 1 - old;
      x = pre_min(full, t < 0 ? 0 : t / TT + 1);
    }
    int64_t at = x * old + TT * (x * (x + 1) / 2) + (full - x) * (TT - 1 + W + S) + full * start;
    if (m >= all) at += keys(all - 1) + start;
    return at;
  }
};

// sequence b's rows of q and cached tokens, within the tensors; false: they were not
K3_HD bool pre_bounds(const PrefillParams& p, int b, int32_t& s0, int32_t& n, int32_t& len) {
  const int32_t a = p.starts[b], e = p.starts[b + 1], l = p.lens[b];
  const int64_t most = (int64_t)p.table_width * p.c.page_size;
  s0 = a < 0 ? 0 : a > p.T ? p.T : a;
  const int32_t s1 = e < s0 ? s0 : e > p.T ? p.T : e;
  n = s1 - s0;
  len = l < 0 ? 0 : l > most ? (int32_t)most : l;
  return s0 == a && s1 == e && len == l && len >= n;
}
K3_HD PreSeq pre_seq(const PrefillParams& p, int32_t n, int32_t len, int32_t start) {
  return PreSeq{n, len > n ? len - n : 0, p.window, p.sinks, p.tokens, start};
}
K3_HD PreSeq pre_seq(const PrefillParams& p, int32_t n, int32_t len) { return pre_seq(p, n, len, p.start); }
// What a start counts as in a call of `total` places with p.start: a block's least where blocks have less.
K3_HD int32_t pre_start_in(const PrefillParams& p, int64_t total, int64_t blocks) {
  return total < blocks * PRE_LEAST && p.start < PRE_LEAST ? PRE_LEAST : p.start;
}

// One part of a tile, as the block's warps get it.
struct PreItem {
  int32_t end;                          // no more
  int32_t b, kvh, head0, heads;         // sequence, key head, first query head and their number
  int32_t row0, ntok, pos0, len;        // first row of q, tokens, position of the first, cached tokens
  int32_t f, ns, keys;                  // keys: ns sinks, then from token f on, in all
  int32_t kt0, kt1;                     // tiles of keys
  int32_t whole, c0, parts;             // all of them; else the tile's first block, the number of them
};

// The walk through a block's items.
struct PreWalk {
  int64_t x, end, chunk;  // place of the tile's first key, end of the block's range, places of a block
  int64_t m;
  int32_t b, h, kt, s0, n, len, bn, start = 0;  // start: 0 as p has it
  K3_HD int32_t start_of(const PrefillParams& p) const { return start ? start : p.start; }
  K3_HD void seq(const PrefillParams& p) { pre_bounds(p, b, s0, n, len); }
  // the block's first item: its range begins `off` places after sequence b's start
  K3_HD void land(const PrefillParams& p, int64_t off) {
    seq(p);
    const PreSeq s = pre_seq(p, n, len, start_of(p));
    const int64_t all = s.tiles(), each = s.place(all);
    const int64_t hh = off / each, rem = off - hh * each;
    h = (int32_t)hh;
    int64_t lo = 0, hi = all;  // the last tile that starts at or before rem
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (s.place(mid) <= rem)
        lo = mid;
      else
        hi = mid;
    }
    m = lo;
    x = end - chunk - rem + s.place(m) + start_of(p);  // (end - chunk: the block's first place)
    const int64_t first = end - chunk, nkt = (s.keys(m) + bn - 1) / bn;
    kt = 0;
    if (first > x) {
      const int64_t k = (first - x + bn - 1) / bn;
      if (nkt <= PRE_WHOLE || k >= nkt)
        next(p);  // another block's to the end
      else
        kt = (int32_t)k;
    }
  }
  K3_HD void next(const PrefillParams& p) {
    const PreSeq s = pre_seq(p, n, len, start_of(p));
    x += s.keys(m) + start_of(p);
    kt = 0;
    if (++m < s.tiles()) return;
    m = 0;
    if (++h < p.Hkv * p.groups) return;
    h = 0;
    do {
      if (++b >= p.B) return;
      if (x >= end) return;  // (past the range already, whatever it is)
      seq(p);
    } while (n <= 0);
  }
  // the item here; false: there is none
  K3_HD bool item(const PrefillParams& p, PreItem& it) {
    it.end = 1;
    if (b >= p.B || (kt == 0 && x >= end)) return false;
    const PreSeq s = pre_seq(p, n, len, start_of(p));
    const int64_t keys = s.keys(m), nkt = (keys + bn - 1) / bn;
    int64_t k1 = nkt <= PRE_WHOLE ? nkt : pre_min(nkt, (end - x + bn - 1) / bn);
    it.end = 0;
    it.b = b;
    it.kvh = h / p.groups;
    const int32_t grp = h - it.kvh * p.groups;
    it.head0 = it.kvh * p.G + grp * p.heads;
    it.heads = (int32_t)pre_min(p.heads, p.G - grp * p.heads);
    it.row0 = s0 + (int32_t)(m * p.tokens);
    it.ntok = (int32_t)pre_min(p.tokens, n - m * p.tokens);
    it.pos0 = (int32_t)(len - n + m * p.tokens);
    it.len = len;
    it.f = p.window > 0 ? (int32_t)pre_max(0, (int64_t)it.pos0 - p.window + 1) : 0;
    it.ns = (int32_t)pre_min(p.sinks, it.f);
    it.keys = (int32_t)keys;
    it.kt0 = kt;
    it.kt1 = (int32_t)k1;
    it.whole = kt == 0 && k1 == nkt;
    it.c0 = (int32_t)(x / chunk);
    it.parts = (int32_t)((x + (nkt - 1) * bn) / chunk) - it.c0 + 1;
    kt = (int32_t)k1;
    if (k1 == nkt) next(p);
    else b = p.B;  // the rest is the next block's
    return true;
  }
};
// The keys of a tile that a token at position pos attends to: those below hi that are at least lo or below sk.
struct PreSeen {
  int32_t hi, lo, sk;
  K3_DEVI PreSeen(const PrefillParams& p, int32_t pos, int32_t f, int32_t ns, int32_t keys)
      : hi(max(0, min(pos + 1 - f + ns, keys))),
        lo(p.window > 0 ? (pos >= p.window ? pos - p.window + 1 : 0) - f + ns : 0),
        sk(p.window > 0 ? p.sinks : 0) {}
};
// places of a block
K3_HD int64_t pre_chunk(int64_t total, int64_t blocks) { return pre_max(PRE_LEAST, (total + blocks - 1) / blocks); }

// ---------------------------------------------------------------------------- rows one by one
// eight values of a cached row: as they are stored, and as numbers
struct Eight {
  uint4 v;
  uint32_t exp;
};
template <int FMT>
K3_DEVI Eight load8(const uint8_t* row, int chunk, const uint8_t* exps) {
  Eight r{};
  if constexpr (FMT == CF_BF16) {
    r.v = ldg128(row + 16 * chunk);
  } else if constexpr (FMT == CF_E4M3) {
    const uint2 c = ldg64(row + 8 * chunk);
    r.v.x = c.x;
    r.v.y = c.y;
  } else {
    r.v.x = __ldg(reinterpret_cast<const uint32_t*>(row + 4 * chunk));
    r.exp = __ldg(exps + chunk / 4);
  }
  return r;
}
template <int FMT>
K3_DEVI void values8(const Eight& r, float scale, float (&x)[8]) {
  uint4 v = r.v;
  if constexpr (FMT == CF_E4M3) {
    uint32_t h[4];
    e4m3x4_f16x4(v.x, h[0], h[1]);
    e4m3x4_f16x4(v.y, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      x[2 * i] = f.x * scale;
      x[2 * i + 1] = f.y * scale;
    }
    return;
  }
  if constexpr (FMT == CF_MXFP4) v = e2m1x8_bf16(v.x, r.exp);
  float2 y[4];
  unpack8(v, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = y[i].x;
    x[2 * i + 1] = y[i].y;
  }
}

// the low bits of a word: those below x
K3_DEVI uint32_t bits_below(int x) { return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u; }

// A tile's products take every row of values, and weight 0 times a value that is infinite or NaN is NaN.  A
// row of the result that is not finite is right if it has seen a NaN in each dim that is NaN and an infinity in
// each that is infinite.  Else one of its tile's keys has such a value that it does not see, behind its position
// or in front of its window (or infinities of both signs are there, or its weight has vanished), or sums of
// finite values have left fp32's range on the way, with weights of up to 2^8: prefill_again forms the row again,
// over its visible keys alone.
struct PreKeys {
  int32_t b, kvh, f, ns, keys, len;  // as PreItem's
};
struct PreRow {  // a lane's: its visible keys, its place
  PreSeen seen;
  int32_t head;
  int64_t row;
};
K3_HD constexpr int key_lanes(int dp) { return dp <= 64 ? 8 : dp <= 128 ? 16 : 32; }  // lanes a key, eight dims each

// where key v's row begins (-1: there is none), and its scales
K3_DEVI void key_at(const PrefillParams& p, const PreKeys& k, uint32_t v, int64_t& at, int64_t& so) {
  at = -1;
  so = 0;
  const uint32_t t = v < (uint32_t)k.ns ? v : v - k.ns + k.f;
  if (v >= (uint32_t)k.keys || t >= (uint32_t)k.len) return;
  const uint32_t pg = p.c.by_page(t), in_page = t - pg * (uint32_t)p.c.page_size;
  const int32_t entry = __ldg(p.table + (int64_t)k.b * p.table_width + pg);
  if (entry < 0 || entry >= p.c.n_pages) return;
  at = entry * p.c.page + k.kvh * p.c.head + in_page * p.c.tok;
  so = entry * p.c.spage + k.kvh * p.c.shead + in_page * p.c.stok;
}
// which of eight values are NaN (bits 0 .. 7), and infinite (8 .. 15)
template <int FMT>
K3_DEVI uint32_t not_finite_of(const Eight& v, float scale) {
  float x[8];
  values8<FMT>(v, scale, x);
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t m = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    bits |= (uint32_t)(m > 0x7F800000u) << e | (uint32_t)(m == 0x7F800000u) << (8 + e);
  }
  return bits;
}
template <int FMT>
K3_DEVI uint32_t not_finite8(const PrefillParams& p, int64_t at, int64_t so, int chunk) {
  return not_finite_of<FMT>(load8<FMT>(p.c.v + at, chunk, p.c.v_exps() + so), FMT == CF_E4M3 ? __ldg(p.c.vs + so) : 1.f);
}
// which of the keys v0 .. v0 + 31 have a value that is not finite
template <int FMT, int DP>
K3_DEVI uint32_t not_finite32(const PrefillParams& p, const PreKeys& k, uint32_t v0, int lane) {
  constexpr int L = key_lanes(DP), N = 32 / L;
  int64_t at, so;
  key_at(p, k, v0 + lane, at, so);
  uint32_t keys = 0;
  constexpr int AT_ONCE = 8;  // loads on the way
#pragma unroll 1
  for (int j0 = 0; j0 < 32; j0 += AT_ONCE * N) {
    Eight e[AT_ONCE];
    float scale[AT_ONCE];
    bool on[AT_ONCE];
#pragma unroll
    for (int a = 0; a < AT_ONCE; ++a) {
      const int64_t r = __shfl_sync(0xFFFFFFFFu, at, j0 + a * N + lane / L), o = __shfl_sync(0xFFFFFFFFu, so, j0 + a * N + lane / L);
      on[a] = r >= 0 && 8 * (lane % L) < p.D;  // (else any row's: loads without a branch)
      e[a] = load8<FMT>(p.c.v + (on[a] ? r : 0), on[a] ? lane % L : 0, p.c.v_exps() + (on[a] ? o : 0));
      scale[a] = FMT == CF_E4M3 ? __ldg(p.c.vs + (on[a] ? o : 0)) : 1.f;
    }
#pragma unroll
    for (int a = 0; a < AT_ONCE; ++a) {
      const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, on[a] && not_finite_of<FMT>(e[a], scale[a]));
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (lanes >> (n * L) & (0xFFFFFFFFu >> (32 - L))) keys |= 1u << (j0 + a * N + n);
    }
  }
  return keys;
}

// The first four (or fewer) of the rows `which` by a warp, which share the loads: 32 keys at a time, `L` lanes
// a key, then a lane a key for the weights.
template <int FMT, int DP>
K3_DEVI void prefill_rows(const PrefillParams& p, const PreKeys& k, const PreRow& x, uint32_t which, int lane) {
  constexpr int L = key_lanes(DP), N = 32 / L, ROWS = 2, AT_ONCE = 8;  // (loads of keys on the way)
  const int c = lane % L;
  const bool on = 8 * c < p.D;
  int from[ROWS], hi[ROWS], lo[ROWS], most = 0;
  float q[ROWS][8], acc[ROWS][8], m[ROWS], l[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    from[i] = __ffs(which) - 1;
    if (which & (which - 1)) which &= which - 1;  // (else the last one again)
    hi[i] = __shfl_sync(0xFFFFFFFFu, x.seen.hi, from[i]);
    lo[i] = __shfl_sync(0xFFFFFFFFu, x.seen.lo, from[i]);
    most = max(most, hi[i]);
    const int64_t row = __shfl_sync(0xFFFFFFFFu, x.row, from[i]);
    const int head = __shfl_sync(0xFFFFFFFFu, x.head, from[i]);
    float2 y[4];
    unpack8(on ? ldg128(reinterpret_cast<const uint8_t*>(p.q + row * p.q_stride + (int64_t)head * p.D + 8 * c)) : make_uint4(0, 0, 0, 0), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      q[i][e] = e & 1 ? y[e / 2].y : y[e / 2].x;
      acc[i][e] = 0.f;
    }
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
#pragma unroll 1
  for (int64_t v0 = 0; v0 < most; v0 += 32) {
    const int64_t v = v0 + lane;  // the lane's key
    int64_t at, so;
    key_at(p, k, (uint32_t)v, at, so);
    float s[ROWS] = {};
#pragma unroll 1
    for (int j0 = 0; j0 < 32; j0 += AT_ONCE * N) {
      Eight e[AT_ONCE];
      // (loads without a branch: where there is no key, or no dim of the lane's, of any row)
#pragma unroll
      for (int a = 0; a < AT_ONCE; ++a) {
        const int64_t r = pre_max(__shfl_sync(0xFFFFFFFFu, at, j0 + a * N + lane / L), 0), o = __shfl_sync(0xFFFFFFFFu, so, j0 + a * N + lane / L);
        e[a] = load8<FMT>(p.c.k + r, on ? c : 0, p.c.k_exps() + o);
      }
#pragma unroll
      for (int a = 0; a < AT_ONCE; ++a) {
        const int j = j0 + a * N;
        float y[8];
        values8<FMT>(e[a], 1.f, y);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          float d = 0.f;
#pragma unroll
          for (int x8 = 0; x8 < 8; ++x8) d = fmaf(on ? y[x8] : 0.f, q[i][x8], d);
#pragma unroll
          for (int b = L / 2; b; b >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, b);
          d = __shfl_sync(0xFFFFFFFFu, d, (lane - j) * L & 31);  // that of key lane, where it is one of these
          if ((uint32_t)(lane - j) < (uint32_t)N) s[i] = d;
        }
      }
    }
    float w[ROWS];
    const float unit = (FMT == CF_E4M3 && at >= 0 ? p.c.ks[so] : 1.f) * p.scale;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const bool seen = at >= 0 && v < hi[i] && (v >= lo[i] || v < x.seen.sk);
      const float z = seen ? s[i] * unit : -INFINITY;
      float top = z;
#pragma unroll
      for (int a = 16; a; a >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, a));
      const float m1 = fmaxf(m[i], top), base = m1 == -INFINITY ? 0.f : m1, fall = ex2(m[i] - base), e1 = ex2(z - base);
      m[i] = m1;
      l[i] = l[i] * fall + e1;
      w[i] = seen ? e1 : -1.f;  // (not seen: no product with its value)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[i][e] *= fall;
    }
#pragma unroll 1
    for (int j0 = 0; j0 < 32; j0 += AT_ONCE * N) {
      Eight e[AT_ONCE];
      float scale[AT_ONCE];
#pragma unroll
      for (int a = 0; a < AT_ONCE; ++a) {
        const int64_t r = pre_max(__shfl_sync(0xFFFFFFFFu, at, j0 + a * N + lane / L), 0), o = __shfl_sync(0xFFFFFFFFu, so, j0 + a * N + lane / L);
        e[a] = load8<FMT>(p.c.v + r, on ? c : 0, p.c.v_exps() + o);
        scale[a] = FMT == CF_E4M3 ? __ldg(p.c.vs + o) : 1.f;
      }
#pragma unroll
      for (int a = 0; a < AT_ONCE; ++a) {
        float y[8];
        values8<FMT>(e[a], scale[a], y);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const float wj = __shfl_sync(0xFFFFFFFFu, w[i], j0 + a * N + lane / L);
#pragma unroll
          for (int x8 = 0; x8 < 8; ++x8) {
            const float sum = fmaf(wj, y[x8], acc[i][x8]);
            acc[i][x8] = wj >= 0.f ? sum : acc[i][x8];
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
#pragma unroll
    for (int a = 16; a; a >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], a);
    const float r = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int a = L; a < 32; a <<= 1) acc[i][e] += __shfl_xor_sync(0xFFFFFFFFu, acc[i][e], a);
      acc[i][e] *= r;
    }
    const int64_t row = __shfl_sync(0xFFFFFFFFu, x.row, from[i]);
    const int head = __shfl_sync(0xFFFFFFFFu, x.head, from[i]);
    if (lane < L && on) {  // (one row twice: the same numbers)
      const uint2 a = bf16x4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]), b = bf16x4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      *reinterpret_cast<uint4*>(p.out + (row * p.Hq + head) * p.D + 8 * c) = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

// A warp's rows that are not finite (in `rows`, a lane a row; out holds them).
template <int FMT, int DP>
__device__ __noinline__ void prefill_again(const PrefillParams& p, const PreKeys k, const PreRow x, uint32_t rows, int lane) {
  auto seen = [&](int64_t v0) {  // by the lane's row
    return bits_below((int)(x.seen.hi - v0)) & (~bits_below((int)(x.seen.lo - v0)) | bits_below((int)(x.seen.sk - v0)));
  };
  // ---- the rows' dims that are NaN, and infinite, a byte a row, a lane eight dims
  uint32_t dims[2][8];
  int end = 0;  // of the keys that any of them sees
  __syncwarp();  // (what other lanes have written is read, and written again)
#pragma unroll 1
  for (int g = 0; g < 8; ++g) {
    uint32_t nan = 0, inf = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = __shfl_sync(0xFFFFFFFFu, x.row, 4 * g + i);
      const int head = __shfl_sync(0xFFFFFFFFu, x.head, 4 * g + i), hi = __shfl_sync(0xFFFFFFFFu, x.seen.hi, 4 * g + i);
      const bool there = rows >> (4 * g + i) & 1;
      if (there) end = max(end, hi);
      const uint4 v = there && 8 * lane < p.D ? *reinterpret_cast<const uint4*>(p.out + (row * p.Hq + head) * p.D + 8 * lane)
                                              : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t m = w[e / 2] >> (16 * (e & 1)) & 0x7FFFu;
        nan |= (uint32_t)(m > 0x7F80u) << (8 * i + e);
        inf |= (uint32_t)(m == 0x7F80u) << (8 * i + e);
      }
    }
    dims[0][g] = nan;
    dims[1][g] = inf;
  }
  // ---- until a visible value accounts for each
  uint32_t open = rows;
#pragma unroll 1
  for (int64_t v0 = 0; open && v0 < end; v0 += 32) {
    uint32_t keys = not_finite32<FMT, DP>(p, k, (uint32_t)v0, lane);
    const uint32_t mask = seen(v0);
#pragma unroll 1
    for (; keys && open; keys &= keys - 1) {
      const int j = __ffs(keys) - 1;
      int64_t at, so;
      key_at(p, k, (uint32_t)v0 + j, at, so);
      const uint32_t its = 8 * lane < p.D ? not_finite8<FMT>(p, at, so, lane) : 0, sees = __ballot_sync(0xFFFFFFFFu, mask >> j & 1);
      uint32_t left = 0;
#pragma unroll 1
      for (int g = 0; g < 8; ++g) {
        // (a row's bit to each bit of its byte; a byte's any bit to a row's bit)
        const uint32_t bytes = ((sees >> (4 * g) & 15) * 0x00204081u & 0x01010101u) * 255u;
        const uint32_t nan = dims[0][g] & ~((its & 255) * 0x01010101u & bytes), inf = dims[1][g] & ~((its >> 8) * 0x01010101u & bytes);
        dims[0][g] = nan;
        dims[1][g] = inf;
#pragma unroll
        for (int i = 0; i < 4; ++i) left |= (uint32_t)(((nan | inf) >> (8 * i) & 255) != 0) << (4 * g + i);
      }
      open &= __reduce_or_sync(0xFFFFFFFFu, left);
    }
  }
#pragma unroll 1
  for (uint32_t which = open; which;) {
    prefill_rows<FMT, DP>(p, k, x, which, lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) which &= which - 1;
  }
}

// ---------------------------------------------------------------------------- the kernel
template <int FMT, int DP>
struct PreCfg {
  static constexpr int HALVES = DP <= 128 ? 2 : 1;  // 128 rows each
  static constexpr int ROWS = 128 * HALVES;
  static constexpr int BN = DP <= 128 ? 128 : 64;  // keys of a tile
  static constexpr int Q_HALF = 128 * DP * 2;
  static constexpr int TILE = BN * DP * 2;  // bytes of a tile's keys, or values
  // A copying warp has its rows of each tile, 8 at a time (a lane a quarter of the 16-byte pieces of one):
  // up to EIGHTS times.  Rows in codes come through a ring of each warp's own and are turned into bf16 from
  // there, RAWS tiles of keys or values later: rows, then words of scales.
  static constexpr int EIGHTS = (BN / 8 + PRE_COPY_WARPS - 1) / PRE_COPY_WARPS, OWN = 8 * EIGHTS;
  static constexpr int PIECES = FMT == CF_BF16 ? 0 : FMT == CF_E4M3 ? DP / 64 : (DP + 127) / 128;
  static constexpr int RAW_ROW = FMT == CF_MXFP4 ? DP / 2 : DP, WORDS = FMT == CF_E4M3 ? 2 : (DP + 127) / 128;
  static constexpr int RAW = FMT == CF_BF16 ? 0 : OWN * (RAW_ROW + 4 * WORDS);
  // masks and scales of RING tiles: those of a tile are read until its weights are formed, and the copies are
  // SLOTS tiles and one ahead of that (two with one half)
  static constexpr int RING = FMT == CF_BF16 || DP <= 64 ? 8 : 4;
  static constexpr int SCALES = FMT == CF_E4M3 ? RING * 2 * BN * 4 : 0;
  static constexpr int OTHERS = 1024 + HALVES * Q_HALF + 512 + 4 * 128 + RING * 16 + 64 + SCALES;  // barriers, items, masks
  static constexpr int ROOM = 227 * 1024 - OTHERS;
  // tiles of keys, and of values, as bf16 (codes: no more than leaves each warp's ring two and more)
  static constexpr int SLOTS = FMT == CF_BF16 ? (ROOM / (2 * TILE) > 4 ? 4 : ROOM / (2 * TILE)) : DP <= 64 ? 3 : 2;
  static constexpr int V_SLOTS = FMT == CF_E4M3 && (DP == 128 || DP == 256) ? 1 : SLOTS;
  static constexpr int RAWS_FIT = FMT == CF_BF16 ? 0 : (ROOM - (SLOTS + V_SLOTS) * TILE) / (PRE_COPY_WARPS * (RAW + 8));
  static constexpr int RAWS = RAWS_FIT > 6 ? 6 : RAWS_FIT;
  static constexpr int SMEM = OTHERS + (SLOTS + V_SLOTS) * TILE + PRE_COPY_WARPS * RAWS * (RAW + 8);
  static constexpr int REC = ROWS * (DP + 2);  // floats of a record
  // columns of tensor memory: a half's logits (with one half two buffers), its weights over them (with one
  // half behind the sums), its sums
  static constexpr uint32_t S_AT = BN, O_AT = DP <= 128 ? 256 : 128, P_AT = DP <= 128 ? 0 : 384, P_STEP = DP <= 128 ? BN : BN / 2;
  static_assert(SLOTS >= 2 && SLOTS + 2 <= RING && (FMT == CF_BF16 || RAWS >= 2) && SMEM <= 227 * 1024 && sizeof(PreItem) <= 128, "does not fit");
};

K3_DEVI float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
K3_DEVI uint32_t bf16x2_of(float2 x) {
  const __nv_bfloat162 h = __float22bfloat162_rn(x);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// a byte pair's E4M3 codes as bf16 (exact)
K3_DEVI void e4m3x4_bf16(uint32_t w, uint32_t& a, uint32_t& b) {
  uint32_t h[2];
  e4m3x4_f16x4(w, h[0], h[1]);
  a = bf16x2_of(__half22float2(*reinterpret_cast<const __half2*>(&h[0])));
  b = bf16x2_of(__half22float2(*reinterpret_cast<const __half2*>(&h[1])));
}
K3_DEVI uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Eight E2M1 codes times 2^(b - 127) as bf16, in order: a code's sign and low bits placed at bits 15 and
// 8..6 are the value times 2^-126 (one product puts them there), which is scaled by 2^(b - 1), in two
// steps where that is no bf16 number.  Exact.
K3_DEVI uint4 e2m1x8_scaled(uint32_t w, uint32_t b) {
  const uint32_t w8 = w >> 8;
  uint32_t o[4] = {((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, ((w & 0x00F000F0u) * 0x104u) & 0x81C081C0u,
                   ((w8 & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, ((w8 & 0x00F000F0u) * 0x104u) & 0x81C081C0u};
  const uint32_t e = b == 255 ? 0x7FC0u : b <= 128 ? (b + 126) << 7 : 254u << 7, s = e | e << 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = mul_bf16x2(o[i], s);
  if (b > 128 && b != 255) {
    const uint32_t e2 = (b - 1) << 7, s2 = e2 | e2 << 16;  // 2^(b - 128)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mul_bf16x2(o[i], s2);
  }
  return make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410), __byte_perm(o[0], o[1], 0x7632),
                    __byte_perm(o[2], o[3], 0x7632));
}
K3_DEVI void sts128(uint32_t a, uint4 v) { *reinterpret_cast<uint4*>(__cvta_shared_to_generic(a)) = v; }

template <int FMT, int DP>
__global__ void __launch_bounds__(PRE_THREADS, 1)
    k3_prefill_kernel(const __grid_constant__ PrefillMaps maps, const PrefillParams p) {
  using C = PreCfg<FMT, DP>;
  constexpr int BN = C::BN, SLOTS = C::SLOTS, V_SLOTS = C::V_SLOTS, HALVES = C::HALVES, ITEMS = 4, RING = C::RING;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up;
  __shared__ int64_t s_sum[PRE_THREADS / 32], s_off;
  __shared__ uint32_t s_tiles[PRE_THREADS / 32];
  __shared__ int32_t s_b, s_last[2];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_at = base, k_at = q_at + HALVES * C::Q_HALF, v_at = k_at + SLOTS * C::TILE, bars = v_at + V_SLOTS * C::TILE;
  const uint32_t items_at = bars + 512, masks_at = items_at + ITEMS * 128, scales_at = (masks_at + RING * 16 + 63u) & ~63u,
                 raw_at = scales_at + C::SCALES, raw_notes = raw_at + PRE_COPY_WARPS * C::RAWS * C::RAW;
  auto k_full = [&](int s) { return bars + 8 * s; };
  auto k_empty = [&](int s) { return bars + 8 * (4 + s); };
  auto v_full = [&](int s) { return bars + 8 * (8 + s); };
  auto v_empty = [&](int s) { return bars + 8 * (12 + s); };
  auto q_full = [&](int h) { return bars + 8 * (16 + h); };
  auto q_empty = [&](int h) { return bars + 8 * (18 + h); };
  auto s_full = [&](int h) { return bars + 8 * (20 + h); };  // of a half, or with one half of a buffer
  auto p_full = [&](int h) { return bars + 8 * (22 + h); };  // likewise
  // of a half's tile n, two in turn: a wait that earlier tiles have left out cannot take one phase for another
  auto o_done = [&](int h, int n) { return bars + 8 * (24 + 2 * h + (n & 1)); };
  auto i_full = [&](int i) { return bars + 8 * (28 + i); };
  auto i_empty = [&](int i) { return bars + 8 * (32 + i); };
  auto p_rest = [&](int h) { return bars + 8 * (36 + h); };  // the second half of a tile's weights
  const uint32_t done = bars + 8 * 38;
  // of a half's cut tile, one that goes on from the block before (0) or on behind (1), of which a block has one
  // each: the four warps' rows of the record are there; s_last says whether it is the last one
  auto r_there = [&](int h, int which) { return bars + 8 * (39 + 2 * h + which); };
  auto r_last = [&](int h, int which) { return bars + 8 * (43 + 2 * h + which); };
  volatile int* const gave_up = &s_gave_up;

  if (threadIdx.x == 0) {
    s_gave_up = 0;
    for (int i = 0; i < 4; ++i) {
      mb_init(k_full(i), PRE_COPY_WARPS);
      mb_init(v_full(i), PRE_COPY_WARPS);
      mb_init(k_empty(i), 1);
      mb_init(v_empty(i), 1);
      mb_init(i_full(i), 1);
      mb_init(i_empty(i), 8 + PRE_COPY_WARPS + 1);
    }
    for (int h = 0; h < 2; ++h) {
      mb_init(q_full(h), PRE_COPY_WARPS);
      mb_init(q_empty(h), 1);
      mb_init(s_full(h), 1);
      mb_init(p_full(h), 4);
      mb_init(p_rest(h), 4);
      mb_init(o_done(h, 0), 1);
      mb_init(o_done(h, 1), 1);
      for (int i = 0; i < 2; ++i) {
        mb_init(r_there(h, i), 4);
        mb_init(r_last(h, i), 1);
      }
    }
    mb_init(done, 1);
    mb_init_fence();
  }
  if (warp == PRE_THREADS / 32 - 1) tm_alloc(smem_u32(&s_tmem), 512);

  grid_dep_wait();

  // ---- this block's range: every thread counts its sequences' places
  const int HR = p.Hkv * p.groups;
  const int each = (p.B + PRE_THREADS - 1) / PRE_THREADS, b_lo = min(p.B, (int)threadIdx.x * each), b_hi = min(p.B, b_lo + each);
  int64_t mine = 0;
  uint32_t tiles_mine = 0;  // (used where there are few: they may wrap)
  bool bad = false;
  for (int b = b_lo; b < b_hi; ++b) {
    int32_t s0, n, len;
    bad |= !pre_bounds(p, b, s0, n, len);
    const PreSeq s = pre_seq(p, n, len);
    mine += s.place(s.tiles()) * HR;
    tiles_mine += (uint32_t)s.tiles() * HR;
  }
  if (bad && blockIdx.x == 0) flag_status(p.status, K3ATTN_DEV_BAD_LENGTH);
  int64_t upto = mine;
  uint32_t tiles_upto = tiles_mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, tiles_upto, o);
    if (lane >= o) {
      upto += v;
      tiles_upto += n;
    }
  }
  if (lane == 31) {
    s_sum[warp] = upto;
    s_tiles[warp] = tiles_upto;
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  // (not before the block has its tensor memory: the next kernel's could take it and wait for this one)
  grid_dep_launch();
  const uint32_t tmem = s_tmem;
  int64_t total = 0;
  uint32_t tiles_total = 0;
  for (int w = 0; w < PRE_THREADS / 32; ++w) {
    if (w == warp) {
      upto += total;
      tiles_upto += tiles_total;
    }
    total += s_sum[w];
    tiles_total += s_tiles[w];
  }
  const int32_t start = pre_start_in(p, total, gridDim.x);
  if (start != p.start) {
    mine += tiles_mine * (start - p.start);
    upto += tiles_upto * (start - p.start);
    total += tiles_total * (start - p.start);
  }
  const int64_t chunk = pre_chunk(total, gridDim.x), first = blockIdx.x * chunk;
  if (mine > 0 && first >= upto - mine && first < upto) {
    int64_t before = upto - mine;
    for (int b = b_lo;; ++b) {
      int32_t s0, n, len;
      pre_bounds(p, b, s0, n, len);
      const PreSeq s = pre_seq(p, n, len, start);
      const int64_t here = s.place(s.tiles()) * HR;
      if (first < before + here) {
        s_b = b;
        s_off = first - before;
        break;
      }
      before += here;
    }
  }
  __syncthreads();

  // ---- roles.  An item goes to all of them: `take` waits for the next one and copies it.
  int taken = 0;
  auto take = [&](PreItem& it) {
    const int i = taken % ITEMS;
    if (!__all_sync(0xFFFFFFFFu, mb_wait(i_full(i), (taken / ITEMS) & 1, gave_up))) return false;
    it = *reinterpret_cast<const PreItem*>(__cvta_shared_to_generic(items_at + i * 128));
    __syncwarp();
    if (lane == 0) mb_arrive(i_empty(i));
    ++taken;
    return !it.end;
  };

  if (warp < 8) {
    regs_more<PRE_REGS_SOFTMAX>();
    const int half = warp / 4, r = half * 128 + (warp % 4) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16);
    const uint32_t o_at = lanes + C::O_AT + half * 128;
    int n_s = 0, n_tile = 0;  // tiles of keys of this half so far, and of the block
    const float unit = FMT == CF_E4M3 ? 1.f : p.scale;  // (E4M3: in the keys' scales)
    bool ok = half < HALVES;
    PreItem it{};
    while (ok && take(it)) {
      const int nkt = it.kt1 - it.kt0, tile0 = n_tile;
      n_tile += nkt;
      if (it.ntok * it.heads <= half * 128) continue;
      const int tok = r / it.heads, head = it.head0 + (r - tok * it.heads);
      const bool valid = tok < it.ntok;
      const int32_t pos = it.pos0 + min(tok, it.ntok - 1);
      const PreSeen keys_seen(p, pos, it.f, it.ns, it.keys);
      // the maximum, in units of 2^unit; the sum of weights
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < nkt; ++j) {
        const int buf = HALVES == 2 ? half : n_s & 1;
        const uint32_t par = HALVES == 2 ? n_s & 1 : (n_s >> 1) & 1;
        if (!(ok = __all_sync(0xFFFFFFFFu, mb_wait(s_full(buf), par, gave_up)))) break;
        tm_fence_after();
        const uint32_t s_at = lanes + buf * C::S_AT;
        const int ring = (tile0 + j) % RING, v0 = (it.kt0 + j) * BN;
        const float* const ks = reinterpret_cast<const float*>(__cvta_shared_to_generic(scales_at + ring * 2 * BN * 4));
        const float* const vs = ks + BN;
        const uint4 ok4 = *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(masks_at + ring * 16));
        const int hi = keys_seen.hi - v0, lo = keys_seen.lo - v0, sk = keys_seen.sk - v0;
        const bool all_rows = (ok4.x & ok4.y & (BN > 64 ? ok4.z & ok4.w : ~0u)) == ~0u;
        const bool masked = !__all_sync(0xFFFFFFFFu, all_rows && hi >= BN && (lo <= 0 || sk >= BN));
        // Logits are read twice, for the maximum and for the weights: tensor memory is as near as registers,
        // and a row of 128 does not leave the other warps registers enough.  raw: 32 of them, from 32 c on
        auto logits_of = [&](int c, const uint32_t* raw, float2 (&s)[16]) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            s[i] = make_float2(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1]));
          }
          if constexpr (FMT == CF_E4M3) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {  // (with p.scale)
              const float4 x = *reinterpret_cast<const float4*>(ks + 32 * c + 2 * i);
              s[i] = mul2(s[i], make_float2(x.x, x.y));
              s[i + 1] = mul2(s[i + 1], make_float2(x.z, x.w));
            }
          }
          if (masked) {
            const uint32_t there = c < 2 ? (c == 0 ? ok4.x : ok4.y) : (c == 2 ? ok4.z : ok4.w);
            const uint32_t see = bits_below(hi - 32 * c) & (~bits_below(lo - 32 * c) | bits_below(sk - 32 * c)) & there;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (!(see >> (2 * i) & 1)) s[i].x = -INFINITY;
              if (!(see >> (2 * i + 1) & 1)) s[i].y = -INFINITY;
            }
          }
        };
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int part = 0; part < BN / 64; ++part) {
          uint32_t raw[64];
          tm_ld32(s_at + 64 * part, raw);
          tm_ld32(s_at + 64 * part + 32, raw + 32);
          tm_ld_wait<64>(raw);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float2 s[16];
            logits_of(2 * part + c, raw + 32 * c, s);
#pragma unroll
            for (int i = 0; i < 16; ++i) tops[i & 3] = max3(tops[i & 3], s[i].x, s[i].y);
          }
        }
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        // the maximum moves where a row's is more than 2^8 above it (weights up to 2^8 are as exact), and
        // the sums with it
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xFFFFFFFFu, (top - m) * unit > 8.f)) {
          const float m1 = (top - m) * unit > 8.f ? top : m, fall = m1 == m ? 1.f : ex2((m - m1) * unit);
          m = m1;
          l *= fall;
          if (!(ok = __all_sync(0xFFFFFFFFu, mb_wait(o_done(half, n_s - 1), (n_s - 1) >> 1 & 1, gave_up)))) break;
          tm_fence_after();
#pragma unroll 1
          for (int c = 0; c < p.D; c += 16) {
            uint32_t o[16];
            tm_ld16(o_at + c, o);
            tm_ld_wait<16>(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fall);
            tm_st16(o_at + c, o);
            tm_st_wait();
            tm_keep16(o);
          }
        }
        const float down = m == -INFINITY ? 0.f : -m;
        float2 sum[4] = {};
        const uint32_t p_at = lanes + C::P_AT + buf * C::P_STEP;
        auto weights_of = [&](int c, const uint32_t* raw, uint32_t (&w)[16]) {
          float2 s[16];
          logits_of(c, raw, s);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            // (the difference first: with the products first, sums and products become one, which does not round
            // the product, and beside a large maximum nothing is left of a weight)
            float2 x = add2(s[i], make_float2(down, down));
            if (FMT != CF_E4M3) x = mul2(x, make_float2(unit, unit));
            float2 e = make_float2(ex2(x.x), ex2(x.y));
            sum[i & 3] = add2(sum[i & 3], e);
            if constexpr (FMT == CF_E4M3) e = mul2(e, *reinterpret_cast<const float2*>(vs + 32 * c + 2 * i));
            w[i] = bf16x2_of(e);
          }
          tm_st16(p_at + 16 * c, w);  // (over logits that are read)
        };
        // (of BN 64 a part is 32 logits, of 128 two times 32, the second ones read while the first are at work)
        constexpr int IN_PART = BN / 64;
        uint32_t raw[2][32];
        tm_ld32(s_at, raw[0]);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {  // the product begins with the first part's weights
          uint32_t w[IN_PART][16];
          tm_ld_wait<32>(raw[0]);
          if (IN_PART == 2) tm_ld32(s_at + 64 * part + 32, raw[1]);
          weights_of(IN_PART * part, raw[0], w[0]);
          if (IN_PART == 2) tm_ld_wait<32>(raw[1]);
          if (part == 0) tm_ld32(s_at + 32 * IN_PART, raw[0]);
          if (IN_PART == 2) weights_of(2 * part + 1, raw[1], w[IN_PART - 1]);
          tm_st_wait();
#pragma unroll
          for (int c = 0; c < IN_PART; ++c) tm_keep16(w[c]);
          tm_fence_before();
          __syncwarp();
          if (lane == 0) mb_arrive(part ? p_rest(buf) : p_full(buf));
        }
        const float2 both = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += both.x + both.y;
        ++n_s;
      }
      if (!ok || !(ok = __all_sync(0xFFFFFFFFu, mb_wait(o_done(half, n_s - 1), (n_s - 1) >> 1 & 1, gave_up)))) break;
      tm_fence_after();
      const int64_t row = it.row0 + tok;
      float* rec = p.parts + (2 * (int64_t)blockIdx.x + (it.kt0 == 0)) * C::REC;
      float inv = l == 0.f ? 0.f : 1.f / l, base = m == -INFINITY ? 0.f : m * unit;
      uint16_t* const out = p.out + (row * p.Hq + head) * p.D;
      uint32_t largest = 0;  // a result that is not finite shows
      bool final = it.whole;
      if (it.whole) {
#pragma unroll 1
        for (int c = 0; c < p.D; c += 16) {
          uint32_t o[16];
          tm_ld16(o_at + c, o);
          tm_ld_wait<16>(o);
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            largest = max(largest, max(o[2 * i] & 0x7FFFFFFFu, o[2 * i + 1] & 0x7FFFFFFFu));
            w[i] = bf16x2_of(make_float2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv));
          }
          if (valid) {
            *reinterpret_cast<uint4*>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      } else {
        // a record: quads of dims of all rows, then each row's maximum and sum
#pragma unroll 1
        for (int c = 0; c < p.D; c += 16) {
          uint32_t o[16];
          tm_ld16(o_at + c, o);
          tm_ld_wait<16>(o);
          if (valid)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(rec + ((c / 4 + i) * C::ROWS + r) * 4) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        if (valid) *reinterpret_cast<float2*>(rec + C::ROWS * DP + 2 * r) = make_float2(m * unit, l);
        // (waits that end, no barrier of the half's warps: one of them may have given up, or not have
        // come this far)
        __syncwarp();
        if (lane == 0) mb_arrive(r_there(half, it.kt0 == 0));
        if (warp % 4 == 0) {
          if (!(ok = __all_sync(0xFFFFFFFFu, mb_wait(r_there(half, it.kt0 == 0), 0, gave_up)))) break;
          if (lane == 0) {
            const bool last = arrive(p.arrived + 2 * it.c0 + half) == (uint32_t)(it.parts - 1);
            if (last) p.arrived[2 * it.c0 + half] = 0;
            s_last[half] = last;  // (read by all warps before they arrive at the next r_there)
            mb_arrive(r_last(half, it.kt0 == 0));
          }
        }
        if (!(ok = __all_sync(0xFFFFFFFFu, mb_wait(r_last(half, it.kt0 == 0), 0, gave_up)))) break;
        final = *reinterpret_cast<volatile int32_t*>(&s_last[half]);
        if (final && valid) {
          // block c0's part is its second record, the others' their first
          auto part = [&](int i) { return p.parts + (2 * (int64_t)(it.c0 + i) + (i == 0)) * C::REC; };
          float top = -INFINITY, sum = 0.f;
          for (int i = 0; i < it.parts; ++i) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(part(i) + C::ROWS * DP + 2 * r));
            const float t1 = fmaxf(top, x.x), b0 = t1 == -INFINITY ? 0.f : t1;
            sum = sum * ex2(top - b0) + x.y * ex2(x.x - b0);
            top = t1;
          }
          l = sum;
          inv = l == 0.f ? 0.f : 1.f / l;
          base = top == -INFINITY ? 0.f : top;
#pragma unroll 1
          for (int c = 0; c < p.D; c += 8) {
            float2 o[4] = {};
            for (int i = 0; i < it.parts; ++i) {
              const float* const y = part(i);
              const float f = ex2(__ldcg(y + C::ROWS * DP + 2 * r) - base);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(y + ((c / 4 + e) * C::ROWS + r) * 4));
                o[2 * e] = fma2(make_float2(v.x, v.y), make_float2(f, f), o[2 * e]);
                o[2 * e + 1] = fma2(make_float2(v.z, v.w), make_float2(f, f), o[2 * e + 1]);
              }
            }
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              largest = max(largest, max(__float_as_uint(o[i].x) & 0x7FFFFFFFu, __float_as_uint(o[i].y) & 0x7FFFFFFFu));
              w[i] = bf16x2_of(mul2(o[i], make_float2(inv, inv)));
            }
            *reinterpret_cast<uint4*>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (final) {
        if (valid && p.lse) p.lse[row * p.Hq + head] = lse_of(base, l);
        const uint32_t again = __ballot_sync(0xFFFFFFFFu, valid && largest >= 0x7F800000u && l < INFINITY);
        if (__builtin_expect(again != 0, 0))
          prefill_again<FMT, DP>(p, PreKeys{it.b, it.kvh, it.f, it.ns, it.keys, it.len}, PreRow{keys_seen, head, row}, again, lane);
      }
    }
    if (half >= HALVES)
      while (take(it)) {
      }
  } else {
    regs_fewer<PRE_REGS_OTHERS>();
    if (warp < 8 + PRE_COPY_WARPS) {
      // ---- copies
      const int w = warp - 8, row_in = lane / 4, piece = lane % 4;
      const int chunks = p.D / 8;  // 16-byte pieces of a row of bf16
      int tiles = 0, q_taken[2] = {0, 0};
      bool ok = true;
      PreItem it{};
      // Copies on the way, oldest first: the barriers that wait for them.  A copy is announced when it has
      // landed and a fence of the thread that made it has made it visible to the tensor core, at the latest
      // before the warp waits for anything.
      uint32_t late[4] = {0, 0, 0, 0};
      int n_late = 0;
      auto landed = [&]() {
        if (n_late == 1)
          cp_async_wait<0>();
        else if (n_late == 2)
          cp_async_wait<1>();
        else if (n_late == 3)
          cp_async_wait<2>();
        else
          cp_async_wait<3>();
        fence_smem_async();
        __syncwarp();
        if (lane == 0) mb_arrive(late[0]);
        late[0] = late[1];
        late[1] = late[2];
        late[2] = late[3];
        --n_late;
      };
      auto on_the_way = [&](uint32_t bar) {
        cp_async_commit();
        if (n_late == 0) late[0] = bar;
        if (n_late == 1) late[1] = bar;
        if (n_late == 2) late[2] = bar;
        if (n_late == 3) late[3] = bar;
        ++n_late;
      };
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (n_late > 0) {
          if (n_late < 4 && __all_sync(0xFFFFFFFFu, mb_test(bar, parity))) return true;
          while (n_late > 0) landed();
        }
        return (bool)__all_sync(0xFFFFFFFFu, mb_wait(bar, parity, gave_up));
      };
      // a piece's place in eight rows of a tile
      auto piece_at = [&](int c, int block) { return row_in * 128 + (c / 8) * block + (((c & 7) ^ row_in) << 4); };
      // a row of a tile or of the queries, bf16, its pieces 4 lanes apart
      auto copy = [&](const uint8_t* from, bool there, uint32_t to, int block) {
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) {
          const int c = piece + 4 * i;
          if (c < chunks) cp_async16_or_zero(to + piece_at(c, block), from + (there ? 16 * c : 0), there ? 16 : 0);
        }
      };
      // A warp's eights of `all`: the first `more` warps have one more than the others; of the values the
      // last ones (so that tiles whose eights the warps do not divide are even over keys and values).
      auto first_of = [&](int all, bool values) {
        const int least = all / PRE_COPY_WARPS, more = all - least * PRE_COPY_WARPS;
        return least * w + (values ? max(0, w - (PRE_COPY_WARPS - more)) : min(w, more));
      };
      auto count_of = [&](int all, bool values) {
        const int least = all / PRE_COPY_WARPS, more = all - least * PRE_COPY_WARPS;
        return least + ((values ? w >= PRE_COPY_WARPS - more : w < more) ? 1 : 0);
      };
      const int k_first = first_of(BN / 8, false), k_count = count_of(BN / 8, false);
      const int v_first = first_of(BN / 8, true), v_count = count_of(BN / 8, true);
      // the warp's rows of the queries of half h
      auto queries = [&](const PreItem& x, int h, int taken_before) {
        if (!wait(q_empty(h), (taken_before & 1) ^ 1)) return false;
        const int q_first = first_of(16, false), q_count = count_of(16, false);
#pragma unroll 1
        for (int g = q_first; g < q_first + q_count; ++g) {
          const int rr = 128 * h + 8 * g + row_in, tok = rr / x.heads, head = x.head0 + (rr - tok * x.heads);
          const bool there = tok < x.ntok;
          const uint16_t* const src = p.q + (there ? (int64_t)(x.row0 + tok) * p.q_stride + (int64_t)head * p.D : 0);
          copy(reinterpret_cast<const uint8_t*>(src), there, q_at + h * C::Q_HALF + g * 1024, 128 * 128);
        }
        on_the_way(q_full(h));
        return true;
      };
      // The warp's rows of the keys or values of a tile, one a lane: page and place in it (-1: there is no such
      // row).  The page table is read a step ahead of the rows' use.
      int32_t entry = -1, in_page = 0, entry_next = -1, in_page_next = 0;
      uint32_t rows = 0;  // those that are there
      auto look_up = [&](int kt, bool values) {  // the next ones
        entry_next = -1;
        in_page_next = -1;
        // (v may be past 2^31)
        const uint32_t v = (uint32_t)kt * BN + 8 * (values ? v_first : k_first) + lane, t = v < (uint32_t)it.ns ? v : v - it.ns + it.f;
        if (lane < 8 * (values ? v_count : k_count) && v < (uint32_t)it.keys && t < (uint32_t)it.len) {
          const uint32_t pg = p.c.by_page(t);
          in_page_next = (int32_t)(t - pg * (uint32_t)p.c.page_size);
          entry_next = __ldg(p.table + (int64_t)it.b * p.table_width + pg);
        }
      };
      auto use_next = [&]() {
        entry = entry_next;
        in_page = in_page_next;
        if (in_page >= 0 && (entry < 0 || entry >= p.c.n_pages)) {
          flag_status(p.status, K3ATTN_DEV_BAD_PAGE);
          entry = -1;
        }
        rows = __ballot_sync(0xFFFFFFFFu, entry >= 0);
      };
      auto set_mask = [&](int tile, uint32_t x) {  // (for all lanes to see after __syncwarp)
        if (lane < k_count)
          *reinterpret_cast<uint8_t*>(__cvta_shared_to_generic(masks_at + tile % RING * 16 + k_first + lane)) = (uint8_t)(x >> (8 * lane));
      };
      if constexpr (FMT == CF_BF16) {
        const int blocks = (p.D + 63) / 64;
        // Rows into a tile: eights that follow one another on a page in boxes, any others row by row.
        auto rows_to = [&](const CUtensorMap* map, const uint8_t* from, uint32_t tile_at, int first, int count, uint32_t full) {
          const int32_t e0 = __shfl_sync(0xFFFFFFFFu, entry, lane & ~7), at0 = __shfl_sync(0xFFFFFFFFu, in_page, lane & ~7);
          const bool follows = entry >= 0 && entry == e0 && in_page == at0 + (lane & 7);
          const uint32_t line = p.boxes ? __ballot_sync(0xFFFFFFFFu, follows) : 0u;
          const int32_t be = __shfl_sync(0xFFFFFFFFu, entry, 8 * lane & 31), bat = __shfl_sync(0xFFFFFFFFu, in_page, 8 * lane & 31);
          const bool box = lane < count && (line >> (8 * lane) & 0xFF) == 0xFF;  // of the lane's eight
          const uint32_t boxed = __ballot_sync(0xFFFFFFFFu, box);
          if (lane == 0 && boxed) mb_expect(full, __popc(boxed) * blocks * 1024);
          __syncwarp();
          if (box)
            for (int c = 0; c < blocks; ++c)
              tma_box(tile_at + c * (BN * 128) + (first + lane) * 1024, map, 64 * c, bat, it.kvh, be, full);
          if (__popc(boxed) == count) {
            if (lane == 0) mb_arrive(full);
            return;
          }
#pragma unroll 1
          for (int g = 0; g < count; ++g) {
            if (boxed >> g & 1) continue;
            const int32_t e = __shfl_sync(0xFFFFFFFFu, entry, 8 * g + row_in), at = __shfl_sync(0xFFFFFFFFu, in_page, 8 * g + row_in);
            const bool there = e >= 0;
            copy(from + (there ? it.kvh * p.c.head + e * p.c.page + at * p.c.tok : 0), there, tile_at + (first + g) * 1024, BN * 128);
          }
          on_the_way(full);
        };
        while (ok) {
          if (n_late > 0 && !__all_sync(0xFFFFFFFFu, mb_test(i_full(taken % ITEMS), (taken / ITEMS) & 1)))
            while (n_late > 0) landed();
          if (!take(it)) break;
          look_up(it.kt0, false);
#pragma unroll 1
          for (int j = it.kt0; j < it.kt1; ++j, ++tiles) {
            use_next();
            look_up(j, true);
            const int ks = tiles % SLOTS, vs = tiles % V_SLOTS;
            if (!(ok = wait(k_empty(ks), (tiles / SLOTS & 1) ^ 1))) break;
            set_mask(tiles, rows);
            __syncwarp();
            rows_to(&maps.k, p.c.k, k_at + ks * C::TILE, k_first, k_count, k_full(ks));
            if (j == it.kt0)
#pragma unroll 1
              for (int h = 0; h < HALVES && ok && it.ntok * it.heads > h * 128; ++h) ok = queries(it, h, q_taken[h]++);
            use_next();
            if (j + 1 < it.kt1) look_up(j + 1, false);
            if (!ok || !(ok = wait(v_empty(vs), (tiles / V_SLOTS & 1) ^ 1))) break;
            rows_to(&maps.v, p.c.v, v_at + vs * C::TILE, v_first, v_count, v_full(vs));
          }
        }
        while (n_late > 0) landed();
      } else {
        // Rows in codes: begun (their copies are on the way into the ring) and finished (in place as bf16), in
        // the order of the products: an item's first keys, its queries, their values, the next keys ..
        static_assert(C::RAW % 16 == 0, "copies of 16 bytes");
        constexpr int RAWS = C::RAWS;
        const uint32_t raws = raw_at + w * (RAWS * C::RAW), notes = raw_notes + w * (RAWS * 8);
        const uint32_t row_bytes = FMT == CF_E4M3 ? p.D : p.D / 2;
        constexpr int KEYS = 0, QUERIES = 1, VALUES = 2, NEW_ITEM = 3, NO_MORE = 4;
        int state = NEW_ITEM, j = 0, front = 0, back = 0, slot_front = 0, slot_back = 0;
#pragma unroll 1
        while (ok) {
          if (front - back == RAWS || (state == NO_MORE && front != back) || state == QUERIES) {
            // ---- finish the oldest; before an item's queries all of it that was begun
            if (state == QUERIES && front == back) {
              for (int h = 0; h < HALVES && ok && it.ntok * it.heads > h * 128; ++h) ok = queries(it, h, q_taken[h]++);
              while (n_late > 0) landed();
              state = VALUES;
              continue;
            }
            if (state == QUERIES || state == NO_MORE)
              cp_async_wait<0>();
            else
              cp_async_wait<RAWS - 1>();
            __syncwarp();
            const uint2 note = lds64(notes + 8 * (back % RAWS));
            const int tile = (int)note.x;
            const uint32_t raw = raws + slot_back;
            ++back;
            slot_back = slot_back + C::RAW == RAWS * C::RAW ? 0 : slot_back + C::RAW;
            const bool keys = !(note.y >> 31);
            const int slot = keys ? tile % SLOTS : tile % V_SLOTS;
            const uint32_t full = keys ? k_full(slot) : v_full(slot);
            if (!(ok = wait(keys ? k_empty(slot) : v_empty(slot), ((keys ? tile / SLOTS : tile / V_SLOTS) & 1) ^ 1))) break;
            const int first = keys ? k_first : v_first, count = keys ? k_count : v_count;
            const uint32_t to0 = (keys ? k_at : v_at) + slot * C::TILE + first * 1024;
#pragma unroll
            for (int g = 0; g < C::EIGHTS; ++g) {
              if (g >= count) break;
              const uint32_t to = to0 + g * 1024, row = raw + (8 * g + row_in) * C::RAW_ROW;
              const uint32_t words = raw + C::OWN * C::RAW_ROW + 4 * (8 * g + row_in);  // C::OWN words apart
#pragma unroll
              for (int i = 0; i < C::PIECES; ++i) {
                // (rows of whole 128 bytes: odd ones from their second 64 on, so that two rows are in different banks)
                const int k = C::RAW_ROW % 128 == 0 ? i ^ (row_in & 1) : i;
                const uint4 v = lds128(row + 16 * (piece + 4 * k));
                if constexpr (FMT == CF_E4M3) {
                  const int c = 2 * (piece + 4 * k);
                  if (c >= chunks) continue;
                  uint4 a, b;
                  e4m3x4_bf16(v.x, a.x, a.y);
                  e4m3x4_bf16(v.y, a.z, a.w);
                  e4m3x4_bf16(v.z, b.x, b.y);
                  e4m3x4_bf16(v.w, b.z, b.w);
                  sts128(to + piece_at(c, BN * 128), a);
                  sts128(to + piece_at(c + 1, BN * 128), b);
                } else {
                  const int c = 4 * (piece + 4 * k);
                  if (c >= chunks) continue;
                  const uint32_t e = lds32(words + k * (4 * C::OWN)) >> (8 * piece) & 255, x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int q = 0; q < 4; ++q) sts128(to + piece_at(c + q, BN * 128), e2m1x8_scaled(x[q], e));
                }
              }
              if (FMT == CF_E4M3 && keys && piece < 2) {
                // (the softmax reads both scales with the logits)
                const float scale = lds_f32(words + piece * (4 * C::OWN));
                sts32(scales_at + tile % RING * 2 * BN * 4 + piece * (BN * 4) + 4 * (8 * (first + g) + row_in),
                      __float_as_uint(piece == 0 ? scale * p.scale : scale));
              }
            }
            if (keys) set_mask(tile, note.y);
            fence_smem_async();
            __syncwarp();
            if (lane == 0) mb_arrive(full);
            continue;
          }
          if (state == NO_MORE) break;
          if (state == NEW_ITEM) {
            if (!take(it)) {
              ok = !*gave_up;
              state = NO_MORE;
              continue;
            }
            j = it.kt0;
            state = KEYS;
            look_up(j, false);
          }
          // ---- begin a tile's keys or values
          const bool keys = state == KEYS;
          use_next();
          if (keys || j + 1 < it.kt1) look_up(keys ? j : j + 1, keys);
          {
            const uint8_t *const from = keys ? p.c.k : p.c.v, *const exps = keys ? p.c.k_exps() : p.c.v_exps();
            const bool mine = lane < 8 * (keys ? k_count : v_count), there = entry >= 0;
            const uint32_t word = raws + slot_front + C::OWN * C::RAW_ROW + 4 * lane;
            const int64_t so = there ? it.kvh * p.c.shead + entry * p.c.spage + in_page * p.c.stok : 0;
            const uint64_t row = (uint64_t)(uintptr_t)(from + (there ? it.kvh * p.c.head + entry * p.c.page + in_page * p.c.tok : 0));
            constexpr int IN_ROW = C::RAW_ROW / 16;  // pieces of a row: consecutive lanes
#pragma unroll
            for (int i = 0; i < (C::OWN * IN_ROW + 31) / 32; ++i) {
              const int r = (32 * i + lane) / IN_ROW, c = (32 * i + lane) % IN_ROW;
              const uint64_t src = __shfl_sync(0xFFFFFFFFu, row, r & 31);
              const uint32_t n = rows >> r & 1 && 16 * c < row_bytes ? 16 : 0;
              if (r < C::OWN)
                cp_async16_or_zero(raws + slot_front + 16 * (32 * i + lane), reinterpret_cast<const uint8_t*>(src) + (n ? 16 * c : 0), n);
            }
            if (mine) {
              if constexpr (FMT == CF_MXFP4) {
#pragma unroll
                for (int k = 0; k < C::WORDS; ++k) {
                  const uint32_t n = there && 128 * k < p.D ? 4 : 0;
                  cp_async4_or_zero(word + k * (4 * C::OWN), exps + (n ? so + 4 * k : 0), n);
                }
              } else if (keys) {
                cp_async4_or_zero(word, p.c.ks + so, there ? 4 : 0);
                cp_async4_or_zero(word + 4 * C::OWN, p.c.vs + so, there ? 4 : 0);
              }
            }
          }
          if (lane == 0) sts64(notes + 8 * (front % RAWS), (uint32_t)tiles, keys ? rows : 0x80000000u);
          __syncwarp();
          cp_async_commit();
          ++front;
          slot_front = slot_front + C::RAW == RAWS * C::RAW ? 0 : slot_front + C::RAW;
          if (keys) {
            state = j == it.kt0 ? QUERIES : VALUES;
          } else {
            ++tiles;
            state = ++j < it.kt1 ? KEYS : NEW_ITEM;
          }
        }
        cp_async_commit();
        cp_async_wait<0>();
      }
    } else if (warp == 8 + PRE_COPY_WARPS) {
      // ---- the block's items
      if (lane == 0) {
        PreWalk walk;
        walk.bn = BN;
        walk.start = start;
        walk.chunk = chunk;
        walk.end = first + chunk;
        walk.b = p.B;
        walk.kt = 0;
        walk.x = walk.end;
        if (first < total) {
          walk.b = s_b;
          walk.land(p, s_off);
        }
        PreItem it;
        it.end = 0;
        for (int n = 0; !it.end; ++n) {
          const int i = n % ITEMS;
          walk.item(p, it);
          if (!mb_wait(i_empty(i), (n / ITEMS & 1) ^ 1, gave_up)) break;
          *reinterpret_cast<PreItem*>(__cvta_shared_to_generic(items_at + i * 128)) = it;
          mb_arrive(i_full(i));
        }
      }
    } else {
      // ---- the products.  All lanes go through this together, so that descriptors and addresses are the
      // warp's; one of them issues (lane 0 alone going through all of it issued wrong ones when the compiler
      // kept them in the warp's registers).
      const uint32_t kind_s = mma_kind(128, BN, false), kind_o = mma_kind(128, p.D, true);
      const int steps = p.D / 16;
      const bool issues = elect_one();
      int tiles = 0, q_taken[2] = {0, 0}, n_p[2] = {0, 0}, n_s = 0;
      PreItem it{};
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        ok = ok && __all_sync(0xFFFFFFFFu, mb_wait(bar, parity, gave_up));
        return ok;
      };
      auto logits = [&](int h, int tile, int buf) {
        const uint64_t a = rows_desc(q_at + h * C::Q_HALF), b = rows_desc(k_at + tile % SLOTS * C::TILE);
        const uint32_t d = tmem + buf * C::S_AT;
        if (issues) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            if (k < steps) mma_ss(d, a + ((k / 4) * 1024 + (k & 3) * 2), b + ((k / 4) * (BN * 8) + (k & 3) * 2), kind_s, k > 0);
          tm_commit(s_full(buf));
        }
      };
      // the product of half of a tile's weights
      auto values = [&](int buf, int h, int tile, bool add, int part) {
        const uint64_t b = rows_desc(v_at + tile % V_SLOTS * C::TILE, BN * 128);
        const uint32_t d = tmem + C::O_AT + h * 128, a = tmem + C::P_AT + buf * C::P_STEP;
        if (issues)
#pragma unroll
          for (int i = 0; i < BN / 32; ++i) {
            const int k = part * (BN / 32) + i;
            mma_ts(d, a + 8 * k, b + k * 128, kind_o, add || k > 0);
          }
      };
      auto commit = [&](uint32_t bar) {
        if (issues) tm_commit(bar);
      };
      auto keys_there = [&](int tile) {
        if (!wait(k_full(tile % SLOTS), tile / SLOTS & 1)) return false;
        tm_fence_after();
        return true;
      };
      auto rows_of_item = [&]() {
        const int nkt = it.kt1 - it.kt0, halves = HALVES == 2 && it.ntok * it.heads > 128 ? 2 : 1;
        // the first logits
        if (!keys_there(tiles)) return;
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
          if (!wait(q_full(h), q_taken[h] & 1)) return;
          tm_fence_after();
          logits(h, tiles, HALVES == 2 ? h : n_s & 1);
          if (nkt == 1) commit(q_empty(h));
          ++q_taken[h];
        }
        commit(k_empty(tiles % SLOTS));
#pragma unroll 1
        for (int j = 0; j < nkt; ++j, ++tiles) {
          const bool more = j + 1 < nkt;
          if (HALVES == 1 && more) {  // the next logits, into the other buffer
            if (!keys_there(tiles + 1)) return;
            logits(0, tiles + 1, (n_s + 1) & 1);
            commit(k_empty((tiles + 1) % SLOTS));
            if (j + 2 == nkt) commit(q_empty(0));
          }
          if (!wait(v_full(tiles % V_SLOTS), tiles / V_SLOTS & 1)) return;
#pragma unroll 1
          for (int h = 0; h < halves; ++h) {
            const int buf = HALVES == 2 ? h : n_s & 1;
            const uint32_t parity = HALVES == 2 ? n_p[h] & 1 : n_s >> 1 & 1;
            if (!wait(p_full(buf), parity)) return;
            tm_fence_after();
            values(buf, h, tiles, j > 0, 0);
            if (!wait(p_rest(buf), parity)) return;
            tm_fence_after();
            values(buf, h, tiles, j > 0, 1);
            commit(o_done(h, HALVES == 2 ? n_p[h] : n_s));
            ++n_p[h];
            if (HALVES == 2 && more) {
              if (h == 0 && !keys_there(tiles + 1)) return;
              logits(h, tiles + 1, h);
              if (j + 2 == nkt) commit(q_empty(h));
            }
          }
          commit(v_empty(tiles % V_SLOTS));
          if (HALVES == 2 && more) commit(k_empty((tiles + 1) % SLOTS));
          ++n_s;
        }
      };
      while (ok && take(it)) rows_of_item();
      commit(done);  // all products have ended before the memory goes
      volatile int never = 0;
      mb_wait(done, 0, &never, MB_LOOKS);
      __syncwarp();
    }
  }
  if (*gave_up)  // copies that nobody has waited for are long over before the block's memory is another's
    for (const long long t0 = clock64(); clock64() - t0 < (1ll << 21);) {
    }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (threadIdx.x == 0 && s_gave_up) flag_status(p.status, K3ATTN_TIMEOUT);
  if (warp == PRE_THREADS / 32 - 1) tm_free(tmem, 512);
}

}  // namespace k3
