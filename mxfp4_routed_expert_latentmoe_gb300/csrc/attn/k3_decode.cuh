// k3_decode.cuh -- attention of one new token over a paged key-value cache.
//
// One pass over the cached rows with a running maximum and sum.  The query heads of one key
// head (8 or 16 of them at a time) are the N side of the matrix instructions and the tokens
// the M side, so that a key head with few query heads wastes no rows:
//   S^T [16 tokens x 8 heads]  = K  [16 tokens x D]  Q^T
//   O^T [16 dims x 8 heads]   += V^T [16 dims x 16 tokens]  P^T
// Each warp streams its own tiles of 16 or 32 tokens through a ring in shared memory with
// cp.async, row by row through the page table (any page size, any strides), and joins its
// team's other warps only at the end of a sequence's part.
//
// What bounds it (GB300, copy rate 6789 GB/s).  Up to 8 query heads a key head, HBM: 2 x 262143
// tokens, 8 E4M3 key heads of 128: 126 us, 90% of the copy rate; 64 sequences of up to 8192
// tokens, bf16: 168 us, 88% (the copies alone reach 95%; the rest is the join at the 3 or 4
// sequence ends of a block).  Up to 16 query heads: twice the matrix instructions and weights a
// tile with the registers of 8 warps an SM used up, so that a warp's own instruction latency
// bounds it: 201 sequences in a window of 1000, 12 heads on E4M3 rows of 192: 64 us, 43%.  MXFP4 rows are
// half as many bytes and as many values: instructions bound them (some 900 a warp for 32 tokens of 128
// dims; issue slots 45%, two warps a scheduler waiting for their own results): 2 x 262143 tokens 145 us,
// 40% of the copy rate, 64 up to 8192 107 us, 37%.  Few
// short sequences: the chain of dependent reads (lengths, page table, rows, joined records),
// 4.7 us for one token, 7.9 us for one sequence of 347.
// mma.sync rather than tcgen05: the products are 2 G flops a cached byte (under 100 TFLOP/s at
// the copy rate with 8 heads), E4M3 rows have to pass through registers on their way to fp16
// anyway, and the softmax stays in the registers that the products leave it in.
//
// MXFP4: codes become fp16 operands exactly, a group's two steps of a key have sums of their own, which
// the group's scale multiplies in fp32; a value's largest scale goes into its weight's exponent like an
// E4M3 row's, and each group's weights are the row's times the power of two that is left (prepare_scales).
//
// E4M3 rows become fp16 operands exactly; a key's scale multiplies its logit, a value's scale
// goes into its weight's exponent, with a maximum of its own, so that weights of values of any
// size keep fp16's full precision.  bf16 rows are multiplied as they are.
//
// Logits, maxima and sums are fp32.  Rounded to fewer bits: a weight to the type of the rows that it
// multiplies, as both operands of a product have one type (bf16, half a step 2^-8 of the weight; fp16,
// 2^-11, and 2^-40 of the largest): a second product with what the rounding left would double the
// second half of the matrix work, and the result is rounded to bf16 anyway (64 sequences up to 8192,
// bf16: results off by 1.75e-3 in the mean square, 1.65e-3 with fp32 weights; E4M3 1.65e-3 both ways;
// the sum of weights is of the unrounded ones).  A query for E4M3 rows to fp16 after a power of two: exact but for elements below 2^-31 of
// its row's largest.  ex2.approx and lg2.approx (2^-22) stand in for exp2f and log2f in weights and
// scales: one instruction each, with an error far below a weight's rounding.
//
// The work is cut into units (W tiles of one (sequence, key head, head group), one for each of
// the W warps of a team), and the units, in a line, are dealt out evenly to all teams, whatever
// the lengths; a sequence's start counts as one or two more, and a sequence of at most DEC_WHOLE tiles
// stays with the team that the first place of its start falls to.  A team joins its warps' sums at the end
// of a sequence's part; a part that is not a whole sequence leaves an unnormalised record in the
// workspace, and the team that arrives last joins a sequence's records, in order.  Long
// sequences have teams of a whole block (few records), short ones of 4, 2 or 1 warps (a warp
// has its own sequence, and waits for nobody).
#pragma once

#include <type_traits>

#include "k3_qkv.cuh"

namespace k3 {

#define K3_HD __host__ __device__ __forceinline__  // also called by a test on the host

struct DecodeParams {
  const uint16_t* q;
  int64_t q_stride;
  int32_t B, Hq, Hkv, G, D, window, sinks;
  int32_t groups;  // head groups of a key head: ceil(G / (8 NT))
  float scale;     // softmax_scale * log2(e): logits in powers of two
  CacheView c;
  const int32_t *table, *lens;
  int32_t table_width;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  uint32_t* arrived;  // one counter a team, zero between calls
  float* parts;       // two records a team
};

// most teams of a launch (the workspace holds their counters and records)
constexpr int DEC_MAX_WARPS = 8;
constexpr int DEC_MAX_BLOCKS = 192;
constexpr int DEC_MAX_TEAMS = DEC_MAX_BLOCKS * DEC_MAX_WARPS;

// Shapes of one instance: the warps of a block, the tokens of a warp's tile, the ring's depth
// (192 KB of rows in all: two or more tiles a warp in flight, 128 KB an SM).
template <int FMT, int DP, int NT>
struct DecCfg {
  static constexpr int ROW = FMT == CF_MXFP4 ? DP / 2 : FMT == CF_E4M3 ? DP : 2 * DP;  // bytes of a row in shared memory
  // 32 tokens a tile where eight warps' rings hold two of them, else 16: a tile's fixed work
  // counts for more than the ring's depth (E4M3, D 192, 12 KB a tile: 201 windowed sequences 64 us,
  // 70 at 16 tokens and a ring of 4; 16 x 20000 tokens 56, 62); and eight warps for the same
  // reason (bf16, D 192: 16 x 10000 tokens 49 us, 55 with four warps and a ring of 4)
  static constexpr int MT = 2 * ROW * 32 <= 12288 ? 2 : 1;
  static constexpr int TW = 16 * MT, TLOG = 3 + MT;
  static constexpr int KV = 2 * TW * ROW;
  static constexpr int WARPS = KV <= 12288 ? 8 : 4;
  // (MXFP4: 6 at most, 160 KB an SM in flight at D 128)
  static constexpr int STAGES = FMT == CF_MXFP4 && 196608 / (WARPS * KV) > 6 ? 6 : 196608 / (WARPS * KV);
  static constexpr int SW = FMT == CF_MXFP4 ? (DP > 128 ? 8 : 4) : FMT == CF_E4M3 ? 4 : 0;  // bytes of a row's scales
  static constexpr int STAGE = KV + 2 * SW * TW + 16;  // rows, scales, mask
  static constexpr int HEADS = 8 * NT;
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int ML = WARPS * HEADS * 2 * 4;
  // MXFP4: what a warp makes of a tile's scales (ScalesAt)
  static constexpr int NG = DP / 32;
  static constexpr int PREP = FMT == CF_MXFP4 ? TW * (4 * NG + 2 * NG + 4) : 0;
  static constexpr int SMEM = RING + ML + 1024 + WARPS * PREP;
  // n-tiles whose sums fit the stage of a tile that is read out (the join of a team's warps)
  static constexpr int PN = HEADS * DP * 4 <= KV ? NT : 1;
  static constexpr int REC = HEADS * (DP + 2);  // floats of a record: sums, and each head's maximum and sum of weights
  static_assert(STAGES >= 2 && SMEM <= 227 * 1024 && PN * 8 * DP * 4 <= KV, "does not fit");
};

// zeros in a warp's ring, by its 32 lanes
template <typename C>
K3_HD void clear_ring(uint8_t* rings, int warp, int lane) {
  uint4* const x = reinterpret_cast<uint4*>(rings + warp * (C::RING / C::WARPS));
  for (int i = lane; i < C::RING / C::WARPS / 16; i += 32) x[i] = make_uint4(0, 0, 0, 0);
}

// D += A B on pairs of sums
K3_DEVI void mma2_bf16(float2 (&d)[2], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  float c[4] = {d[0].x, d[0].y, d[1].x, d[1].y};
  mma_bf16(c, a, b[0], b[1], c);
  d[0] = make_float2(c[0], c[1]);
  d[1] = make_float2(c[2], c[3]);
}
K3_DEVI void mma2_f16(float2 (&d)[2], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  float c[4] = {d[0].x, d[0].y, d[1].x, d[1].y};
  mma_f16(c, a, b[0], b[1], c);
  d[0] = make_float2(c[0], c[1]);
  d[1] = make_float2(c[2], c[3]);
}
K3_DEVI float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&r);
}
K3_DEVI float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
K3_DEVI float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// copies that read nothing and fill with zeros where n is 0
K3_DEVI void cp_async16_or_zero(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n));
}
K3_DEVI void cp_async4_or_zero(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(n));
}
K3_DEVI void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
K3_DEVI void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
K3_DEVI uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// four E4M3 codes -> two words of two fp16
K3_DEVI void e4m3x4_f16x4(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.rn.f16x2.e4m3x2 %0, lo;\ncvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
      : "=r"(a), "=r"(b)
      : "r"(w));
}
K3_DEVI uint4 lds128(uint32_t a) { return *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(a)); }
K3_DEVI float lds_f32(uint32_t a) { return *reinterpret_cast<const float*>(__cvta_shared_to_generic(a)); }

// Byte offset of 16-byte chunk c of a tile's row r: rows are packed, and the chunks of a row
// permuted so that the eight rows of a matrix load, and for E4M3 also the two rows that a
// quarter warp reads 64 bytes of, lie in different banks.
template <int FMT, int ROW>
K3_DEVI uint32_t chunk_at(int r, int c) {
  if constexpr (FMT == CF_MXFP4) {
    constexpr int SHIFT = ROW == 128 ? 0 : ROW == 64 ? 1 : 2, MASK = ROW == 128 ? 7 : ROW == 64 ? 3 : 1;
    return r * ROW + ((c ^ ((r >> SHIFT) & MASK)) << 4);
  } else if constexpr (ROW % 128 == 0) {
    if constexpr (FMT == CF_E4M3) {
      const int f = ((r & 1) << 2) | ((r >> 1) & 3);
      return r * ROW + ((c ^ f) << 4);
    }
    return r * ROW + ((c ^ (r & 7)) << 4);
  } else {  // an odd number of 64-byte pieces a row
    return r * ROW + ((c ^ ((r >> 1) & 3)) << 4);
  }
}

// a / b of non-negative numbers (that are nearly always short)
K3_HD int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
// sum of a warp's non-negative numbers below 2^48
K3_DEVI int64_t warp_sum(int64_t v) {
  return ((int64_t)__reduce_add_sync(0xFFFFFFFFu, (uint32_t)(v >> 24)) << 24) +
         __reduce_add_sync(0xFFFFFFFFu, (uint32_t)v & 0xFFFFFFu);
}
// barrier of one team's threads
K3_DEVI void team_sync(int team, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(team + 1), "r"(threads) : "memory");
}
// counts an arrival: what the team has written (before its barrier) is visible to the team that
// sees the count, and the other way round
K3_DEVI uint32_t arrive(uint32_t* counter) {
  uint32_t before;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;\n" : "=r"(before) : "l"(counter) : "memory");
  return before;
}

// length of sequence b within what its table can hold
K3_HD int32_t seq_len(const DecodeParams& p, int b, bool& bad) {
#ifdef __CUDA_ARCH__
  const int32_t n = __ldg(p.lens + b);
#else
  const int32_t n = p.lens[b];
#endif
  const int64_t most = (int64_t)p.table_width * p.c.page_size;
  bad = n < 0 || n > most;
  return n < 0 ? 0 : (n > most ? (int32_t)most : n);
}

// Units that a sequence's start counts as (its queries, its join): for teams of 4 and 8 warps two
// (64 sequences up to 4000 tokens, 12 query heads a key head, E4M3: 42.0 us, 43.7 at one), for
// smaller ones one (200 sequences up to 100 tokens: 14.9 us, 17.7 at two)
K3_HD int dec_start(int wlog) { return wlog >= 2 ? 2 : 1; }

// Tiles of a sequence that is never cut: joining its records would take longer than they do (200
// sequences up to 100 tokens, D 128, E4M3: 14.9 us, 17.7 if they are cut)
constexpr int DEC_WHOLE = 4;

// A place in the order of the units: sequence b, key head kvh and group grp of its query heads,
// unit u of nu (2^ulog tokens each); x: its number from the team's first one, a sequence's start
// (of each group) counted in front of its units.
struct DecAt {
  int32_t b, kvh, grp, u, nu, first, n, x;
  K3_HD bool open(const DecodeParams& p, int ulog) {  // sequence b's tokens and units; false: a bad length
    bool bad;
    n = seq_len(p, b, bad);
    first = p.window > 0 && n > p.window ? n - p.window : 0;
    first -= first < p.sinks ? first : p.sinks;  // the sinks stand in front of the window's tokens
    nu = (int32_t)(((uint32_t)(n - first) + (1u << ulog) - 1) >> ulog);
    return !bad;
  }
  // the token of a row of the tile that a team's warp tw takes of the unit: past the sequence's last
  // one it may be up to a unit more than n, which passes int32 next to the longest length
  template <int TW>
  K3_HD uint32_t token(int W, int tw, int row) const {
    return (uint32_t)first + ((uint32_t)u * W + tw) * TW + row;
  }
  // what token() stands for where it is one of the sinks: those come first of all
  K3_HD uint32_t seen(const DecodeParams& p, uint32_t t) const {
    return t - (uint32_t)first < (uint32_t)p.sinks ? t - (uint32_t)first : t;
  }
  // whether the unit is the team's whose range ends in front of `end`
  K3_HD bool in(int32_t end, int32_t whole, int start) const { return (nu <= whole ? x - u - start : x) < end; }
  K3_HD void next(const DecodeParams& p, int ulog, int32_t end, int start) {
    ++x;
    if (++u < nu) return;
    x += start;
    u = 0;
    if (x - start >= end) return;  // (its start is past the range already, whatever it is)
    if (++grp < p.groups) return;
    grp = 0;
    if (++kvh < p.Hkv) return;
    kvh = 0;
    do {
      if (++b >= p.B) return;
      open(p, ulog);
    } while (nu == 0);
  }
  // the team's first unit: its range begins `off` places after the first one of sequence b (open)
  K3_HD void land(const DecodeParams& p, int ulog, int64_t off, int32_t end, int32_t whole, int start) {
    const int32_t hr = (int32_t)div64(off, nu + start);
    kvh = hr / p.groups;
    grp = hr - kvh * p.groups;
    u = (int32_t)(off - (int64_t)hr * (nu + start)) - start;
    x = 0;
    if (nu <= whole && u != -start) {  // behind the start's first place: another team's
      x = nu - 1 - u;
      u = nu - 1;
      next(p, ulog, end, start);
    } else if (u < 0) {  // at a start
      x = -u;
      u = 0;
    }
  }
};
// A lane's row of a tile, on its way to be copied: its page (an entry of the page table, still
// being read), its place there, its key head; whether the tile and the row are there at all.
struct DecRow {
  int32_t entry, in_page, kvh;
  bool tile, in;
};
// A part that is not a whole sequence, until its team asks who arrived last.
struct DecPart {
  int64_t i0;           // the sequence's first unit of all
  int64_t row;          // its first row of the output
  int32_t c0, parts;    // its first team, the number of them
  int32_t heads, there;
};

// four values to bf16
K3_DEVI uint2 bf16x4(float a, float b, float c, float d) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
// log-sum-exp from the maximum and the sum of powers of two
K3_DEVI float lse_of(float base, float sum) {
  return sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
}

// MXFP4: a tile's scales as the products take them, one token a lane.  At prep: the keys' scales, f32
// [TW][NG]; the values' factors, f16 [TW / 2][NG][2], 2^(b - largest) with the largest b of the row's
// groups (a group 2^25 and more below it counts as zeros: less than half of fp32's step of the row's
// largest); f32 [TW], the largest as a power of two, for the weight's exponent.  255 gives NaN.
K3_DEVI void sts32(uint32_t a, uint32_t v) { *reinterpret_cast<uint32_t*>(__cvta_shared_to_generic(a)) = v; }
K3_DEVI void sts64(uint32_t a, uint32_t x, uint32_t y) { *reinterpret_cast<uint2*>(__cvta_shared_to_generic(a)) = make_uint2(x, y); }
K3_DEVI void sts16(uint32_t a, uint32_t v) { *reinterpret_cast<uint16_t*>(__cvta_shared_to_generic(a)) = (uint16_t)v; }
K3_DEVI uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <typename C>
K3_DEVI void prepare_scales(uint32_t raw, uint32_t prep, int lane, int D) {
  static_assert(C::TW == 32, "a token a lane");
  constexpr int NG = C::NG, TW = C::TW;
  const int groups = D / 32;
  uint32_t kw[C::SW / 4], vw[C::SW / 4];
#pragma unroll
  for (int i = 0; i < C::SW / 4; ++i) {
    kw[i] = lds32(raw + C::SW * lane + 4 * i);
    vw[i] = lds32(raw + C::SW * TW + C::SW * lane + 4 * i);
  }
  int top = 0;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int b = vw[g / 4] >> (8 * (g % 4)) & 255;
    if (g < groups && b != 255) top = max(top, b);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int b = vw[g / 4] >> (8 * (g % 4)) & 255, below = top - b;
    const uint32_t f = b == 255 ? 0x7E00u : below < 15 ? (uint32_t)(15 - below) << 10 : below < 25 ? 1u << (24 - below) : 0u;
    sts16(prep + 4 * NG * TW + 4 * NG * (lane / 2) + 4 * g + 2 * (lane & 1), g < groups ? f : 0u);
  }
#pragma unroll
  for (int g = 0; g < NG; g += 2) {
    const uint32_t k0 = kw[g / 4] >> (8 * (g % 4)) & 255, k1 = kw[(g + 1) / 4] >> (8 * ((g + 1) % 4)) & 255;
    sts64(prep + 4 * NG * lane + 4 * g, g < groups ? __float_as_uint(ue8m0_to_f32(k0)) : 0u,
          g + 1 < groups ? __float_as_uint(ue8m0_to_f32(k1)) : 0u);
  }
  sts32(prep + 6 * NG * TW + 4 * lane, __float_as_uint((float)(top - 127)));
  __syncwarp();
}

// The largest weight of E4M3 and MXFP4 values is 2^15 (fp16's largest number is 65504), so that weights down to
// 2^-40 of it count: 2^31 tokens of less weight each are lost with less than 2^-9 of the result.
constexpr float TOP = 15.f;

template <int FMT, int DP, int NT>
__global__ void __launch_bounds__(DecCfg<FMT, DP, NT>::WARPS * 32, 1) k3_decode_kernel(const DecodeParams p) {
  using C = DecCfg<FMT, DP, NT>;
  constexpr int WARPS = C::WARPS, THREADS = WARPS * 32, TW = C::TW, MT = C::MT, STAGES = C::STAGES, ROW = C::ROW;
  constexpr int HEADS = C::HEADS, KSTEPS = DP / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ring = smem_u32(smem) + warp * STAGES * C::STAGE;
  float* const s_ml = reinterpret_cast<float*>(smem + C::RING);  // [WARPS][HEADS] maxima, sums
  int64_t* const s_sum = reinterpret_cast<int64_t*>(smem + C::RING + C::ML);               // [WARPS]
  int64_t* const s_off = s_sum + DEC_MAX_WARPS;                                            // [teams]
  int32_t* const s_b = reinterpret_cast<int32_t*>(s_off + DEC_MAX_WARPS);                  // [teams]
  volatile int32_t* const s_last = s_b + DEC_MAX_WARPS;                                    // [teams]
  int64_t* const s_count = reinterpret_cast<int64_t*>(smem + C::RING + C::ML + 256);       // [WARPS][4]
  DecPart* const s_part = reinterpret_cast<DecPart*>(smem + C::RING + C::ML + 512);        // [teams][2]
  const uint32_t prep = smem_u32(smem) + C::RING + C::ML + 1024 + warp * C::PREP;
  static_assert(2 * DEC_MAX_WARPS * sizeof(DecPart) <= 512 && DEC_MAX_WARPS * 32 <= 256, "shared layout");

  // dims past D: zero in every stage, and again wherever a join has written.  A warp clears its
  // own ring: no other warp's zeros can land on rows or masks that it has copied by then
  if (p.D < DP) {
    clear_ring<C>(smem, warp, lane);
    __syncwarp();
  }

  grid_dep_wait();
  grid_dep_launch();

  // ---- the teams' size, and the units of this team: every thread counts its sequences' tiles as
  // teams of 1, 2, 4 and 8 warps would take them (with the idle warps of a sequence's last unit).
  // Up to 32 sequences: a lane has one, every warp has them all; more: the block has them.
  const int32_t HR = p.Hkv * p.groups;
  const bool few = p.B <= 32;
  const int seqs = few ? 1 : (p.B + THREADS - 1) / THREADS, first_b = few ? lane : (int)threadIdx.x * seqs;
  const int b_lo = min(p.B, first_b), b_hi = min(p.B, b_lo + seqs);
  DecAt at;
  int64_t count[4] = {0, 0, 0, 0}, some = 0;
  bool any_bad = false;
  at.nu = at.n = at.first = 0;
  for (at.b = b_lo; at.b < b_hi; ++at.b) {
    any_bad |= !at.open(p, C::TLOG);
#pragma unroll
    for (int i = 0; i < 4; ++i) count[i] += (at.nu + (1 << i) - 1) >> i << i;
    some += at.nu > 0;
  }
  if (any_bad && blockIdx.x == 0) flag_status(p.status, K3ATTN_DEV_BAD_LENGTH);
  int64_t sums[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) sums[i] = warp_sum(count[i]);
  if (!few) {
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_count[warp * 4 + i] = sums[i];
    __syncthreads();
    int64_t v = lane < 4 * WARPS ? s_count[lane] : 0;  // lane i: of warp i / 4, of size i % 4; then of all warps
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[i] = __shfl_sync(0xFFFFFFFFu, v, i);
  }
  int wlog = -1;
#pragma unroll
  for (int i = 3; i >= 0; --i)  // the largest that wastes at most a quarter, or leaves warps idle anyway
    if (wlog < 0 && (1 << i) <= WARPS && (4 * sums[i] <= 5 * sums[0] || sums[i] * HR <= (int64_t)gridDim.x * WARPS))
      wlog = i;
  // teams of half a block, where there are sequences enough for all (HR a sequence) with work for
  // more than a moment, and their ends are frequent (at most 24 units of a block each): while one
  // team joins, the other streams.  201 windowed sequences, D 192: 64 us, 76 with whole blocks;
  // 128 up to 2000, D 64: 50, 54; but 64 up to 8192 (64 units each) 170, 167.
  const int64_t parts_all = (int64_t)p.B * HR, warps_all = (int64_t)gridDim.x * WARPS;
  if (wlog == 3 && 10 * parts_all >= 8 * (int64_t)gridDim.x && sums[0] * HR >= 4 * warps_all &&
      sums[3] * HR <= 24 * 8 * parts_all)
    wlog = 2;
  const int W = 1 << wlog, ulog = C::TLOG + wlog, teams = WARPS >> wlog, team = warp >> wlog, tw = warp & (W - 1);
  const int whole_units = DEC_WHOLE >> wlog, start = dec_start(wlog);
  const int tthreads = 32 << wlog, tthread = threadIdx.x & (tthreads - 1);

  const int64_t mine = ((wlog == 0 ? count[0] : wlog == 1 ? count[1] : wlog == 2 ? count[2] : count[3]) >> wlog) + start * some;
  int64_t upto = mine, total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  if (few) {
    total = __shfl_sync(0xFFFFFFFFu, upto, 31);
  } else {
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    total = 0;
    for (int w = 0; w < WARPS; ++w) {
      if (w == warp) upto += total;
      total += s_sum[w];
    }
  }
  total *= HR;
  const int64_t workers = (int64_t)gridDim.x * teams, chunk = max((int64_t)1, div64(total + workers - 1, workers));
  const int64_t worker = (int64_t)blockIdx.x * teams + team, unit0 = worker * chunk;
  const int64_t lo = (upto - mine) * HR, hi = upto * HR;  // this thread's units
  int64_t off = 0;  // the team's first unit, from the first one of its sequence
  if (few) {
    const uint32_t has = __ballot_sync(0xFFFFFFFFu, mine > 0 && unit0 >= lo && unit0 < hi);
    const int from = has ? __ffs(has) - 1 : 0;
    off = unit0 - __shfl_sync(0xFFFFFFFFu, lo, from);
    at.b = from;
    at.n = __shfl_sync(0xFFFFFFFFu, at.n, from);
    at.first = __shfl_sync(0xFFFFFFFFu, at.first, from);
    at.nu = (int32_t)(((uint32_t)(at.n - at.first) + (1u << ulog) - 1) >> ulog);
  } else {
    if (mine > 0) {
      for (int i = 0; i < teams; ++i) {
        const int64_t x = ((int64_t)blockIdx.x * teams + i) * chunk;
        if (x < lo || x >= hi) continue;
        int64_t before = lo;
        for (at.b = b_lo;; ++at.b) {
          at.open(p, ulog);
          const int64_t here = at.nu > 0 ? (int64_t)(at.nu + start) * HR : 0;
          if (x < before + here) break;
          before += here;
        }
        s_b[i] = at.b;
        s_off[i] = x - before;
      }
    }
    __syncthreads();
    if (unit0 < total) {
      at.b = s_b[team];
      off = s_off[team];
      at.open(p, ulog);
    }
  }

  const int32_t end = (int32_t)max((int64_t)0, min(min(total - unit0, chunk), (int64_t)INT32_MAX));
  if (tthread < 2) s_part[2 * team + tthread].there = 0;
  if (end > 0) {
    at.land(p, ulog, off, end, whole_units, start);
    DecAt ahead = at;  // the next tile whose page entries are to be read
    uint32_t got[2] = {0, 0};  // arrivals before this team's (of its first thread)
    bool cut = false;          // there is a part that is not a whole sequence

    // a copy takes LR 16-byte chunks (128 or 64 bytes) of each of 32 / LR rows
    constexpr int CPR = ROW / 16, LR = CPR % 8 == 0 ? 8 : CPR % 4 == 0 ? 4 : 2, RPI = 32 / LR;
    const int cpr = FMT == CF_MXFP4 ? p.D / 32 : FMT == CF_E4M3 ? p.D / 16 : p.D / 8;
    // reads the page entries of the tile at `ahead` (if it is the team's) and moves on
    auto fetch = [&]() {
      DecRow r{0, 0, ahead.kvh, ahead.in(end, whole_units, start), false};
      if (r.tile) {
        uint32_t t = ahead.token<TW>(W, tw, lane & (TW - 1));
        r.in = t < (uint32_t)ahead.n;
        if (r.in) {
          // (without sinks nothing to do: 201 windowed sequences, 12 heads on E4M3 rows of 192: 64.6 us, 65.9 with
          // the arithmetic always; MXFP4 the other way round, 64 sequences up to 8192: 107.6 us always, 108.8)
          if (FMT == CF_MXFP4 || p.sinks > 0) t = ahead.seen(p, t);
          const uint32_t pg = p.c.by_page(t);
          r.entry = __ldg(p.table + (int64_t)ahead.b * p.table_width + pg);
          r.in_page = (int32_t)(t - pg * (uint32_t)p.c.page_size);
        }
        ahead.next(p, ulog, end, start);
      }
      return r;
    };
    auto issue = [&](int stage, const DecRow& x) {  // the copies of a tile
      const uint32_t st = ring + stage * C::STAGE;
      const bool ok = x.in && x.entry >= 0 && x.entry < p.c.n_pages;
      if (x.in && !ok) flag_status(p.status, K3ATTN_DEV_BAD_PAGE);
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
      if (lane == 0) *reinterpret_cast<uint32_t*>(__cvta_shared_to_generic(st + C::STAGE - 16)) = mask;
      if (mask == 0) return;
      const int64_t off = ok ? x.entry * p.c.page + x.kvh * p.c.head + x.in_page * p.c.tok : 0;
      if constexpr (FMT == CF_E4M3) {
        const int64_t so = ok ? x.entry * p.c.spage + x.kvh * p.c.shead + x.in_page * p.c.stok : 0;
        const uint32_t dst = st + C::KV + 4 * (lane & (TW - 1));
        if (TW == 32 || lane < 16) cp_async4_or_zero(dst, p.c.ks + so, ok ? 4 : 0);
        if (TW == 32 || lane >= 16) cp_async4_or_zero(dst + 4 * TW, p.c.vs + so, ok ? 4 : 0);
      }
      if constexpr (FMT == CF_MXFP4) {
        const int64_t so = ok ? x.entry * p.c.spage + x.kvh * p.c.shead + x.in_page * p.c.stok : 0;
        const uint32_t dst = st + C::KV + C::SW * (lane & (TW - 1));
#pragma unroll
        for (int i = 0; i < C::SW; i += 4) {
          const uint32_t n = ok && 32 * i < p.D ? 4 : 0;  // (a row's words: those that D has)
          cp_async4_or_zero(dst + i, p.c.k_exps() + (n ? so + i : 0), n);
          cp_async4_or_zero(dst + C::SW * TW + i, p.c.v_exps() + (n ? so + i : 0), n);
        }
      }
      // the rows follow one another, the last one on the first one's page (sinks: the window's first
      // token need not be next to the last of them)
      auto in_line = [&]() {
        const int32_t at0 = __shfl_sync(0xFFFFFFFFu, x.in_page, 0);
        if (at0 + TW > p.c.page_size) return false;
        return p.sinks == 0 || (__shfl_sync(0xFFFFFFFFu, x.in_page, TW - 1) == at0 + TW - 1 &&
                                __shfl_sync(0xFFFFFFFFu, x.entry, TW - 1) == __shfl_sync(0xFFFFFFFFu, x.entry, 0));
      };
      if (mask == 0xFFFFFFFFu && p.D == DP && in_line()) {
        // all rows there, on one page: they lie a token's stride apart
        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, 0) + (lane / LR) * p.c.tok + 16 * (lane % LR);
        const int64_t step = RPI * p.c.tok;
        const uint8_t *kp = p.c.k + o, *vp = p.c.v + o;
#pragma unroll
        for (int i = 0; i < TW / RPI; ++i) {
          const uint32_t dst = st + chunk_at<FMT, ROW>(i * RPI + lane / LR, lane % LR);
#pragma unroll
          for (int c = 0; c < CPR / LR; ++c) {
            cp_async16(dst + 16 * LR * c, kp + 16 * LR * c);
            cp_async16(dst + TW * ROW + 16 * LR * c, vp + 16 * LR * c);
          }
          kp += step;
          vp += step;
        }
        return;
      }
#pragma unroll
      for (int i = 0; i < TW / RPI; ++i) {
        const int r = i * RPI + lane / LR;
        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r) + 16 * (lane % LR);
        const uint32_t n = (mask >> r) & 1u ? 16u : 0u;  // (a row that is not there: its place is zeroed)
        const uint8_t *kp = p.c.k + (n ? o : 0), *vp = p.c.v + (n ? o : 0);
        const uint32_t dst = st + chunk_at<FMT, ROW>(r, lane % LR);
#pragma unroll
        for (int c = 0; c < CPR / LR; ++c)
          if (LR * c + lane % LR < cpr) {
            cp_async16_or_zero(dst + 16 * LR * c, n ? kp + 16 * LR * c : kp, n);
            cp_async16_or_zero(dst + TW * ROW + 16 * LR * c, n ? vp + 16 * LR * c : vp, n);
          }
      }
    };
    // the ring's first tiles: the page entries of all are read before the first copy waits for its
    // own (one read's latency in front of the copies, not one a tile)
    DecRow first[STAGES - 1];
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) first[i] = fetch();
    DecRow ready = fetch();  // the tile to be copied next
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      if (first[i].tile) issue(i, first[i]);
      cp_async_commit();
    }

    float2 acc[KSTEPS][NT][2], m[NT], l[NT], vm[NT], qs[NT];  // pairs: of two heads
    uint32_t qf[KSTEPS][NT][2];
    // a part's queries as they are, bf16 (step 4 j + i of an E4M3 contraction holds dims
    // 64 j + 16 (lane % 4) + 4 i .. + 3, step 2 g + i of an MXFP4 one dims 32 g + 8 (lane % 4) + 4 i .. + 3).  bf16: loaded while the part before is joined (128
    // sequences up to 2000 tokens, D 64: 50.2 us, 52.8 without; 32 x 5000, 5 heads of 96: 48, 51);
    // E4M3, and 16 bf16 heads of 256 dims: at the part's start, as the registers' longer life costs
    // the inner loop more (2 x 262143 tokens, E4M3: 125 us, 141 early; 16 x 8000, D 256: 49.5, 52.3)
    constexpr bool EARLY = FMT == CF_BF16 && KSTEPS * NT < 32;
    auto load_queries = [&](const DecAt& a) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = a.grp * HEADS + nt * 8 + lane / 4;
        const uint16_t* q = p.q + a.b * p.q_stride + ((int64_t)a.kvh * p.G + h) * p.D;
        const bool on = h < p.G;
#pragma unroll
        for (int c = 0; c < KSTEPS; ++c) {
          if constexpr (FMT == CF_BF16) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = 16 * c + 8 * e + 2 * (lane & 3);
              qf[c][nt][e] = on && d < p.D ? __ldg(reinterpret_cast<const uint32_t*>(q + d)) : 0u;
            }
          } else {
            const int d = FMT == CF_MXFP4 ? 32 * (c / 2) + 8 * (lane & 3) + 4 * (c & 1)
                                          : 64 * (c / 4) + 16 * (lane & 3) + 4 * (c & 3);
            const uint2 w = on && d < p.D ? ldg64(q + d) : make_uint2(0, 0);
            qf[c][nt][0] = w.x;
            qf[c][nt][1] = w.y;
          }
        }
      }
    };
    if (EARLY) load_queries(at);
    int32_t part_u0 = 0, part_slot = 0;
    int stage = 0;
    for (bool begun = false; at.in(end, whole_units, start); begun = true) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      if (ready.tile) {
        issue(stage == 0 ? STAGES - 1 : stage - 1, ready);
        ready = fetch();
      }
      cp_async_commit();
      const int32_t heads = min(HEADS, p.G - at.grp * HEADS);  // of this group
      const int64_t head0 = (int64_t)at.kvh * p.G + at.grp * HEADS;

      if (!begun || at.u == 0) {  // a new part: its queries, empty sums
        if (!EARLY) load_queries(at);
        part_u0 = at.u;
        part_slot = at.u == 0 && at.x > start;  // not the team's first place of all
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          qs[nt] = make_float2(p.scale, p.scale);
          if constexpr (FMT != CF_BF16) {
            // to fp16, scaled by the power of two that brings the row's largest into [2^14, 2^15)
            uint32_t mx = 0;
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c)
              mx = __vmaxu2(mx, __vmaxu2(qf[c][nt][0] & 0x7FFF7FFFu, qf[c][nt][1] & 0x7FFF7FFFu));
            mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            const int pw = act_exp_from_max(max(mx & 0xFFFF0000u, mx << 16));
            const float f1 = pow2f(pw >> 1), f2 = pow2f(pw - (pw >> 1));
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t w = qf[c][nt][e];
                const float2 x = mul2(mul2(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)),
                                           make_float2(f1, f1)),
                                      make_float2(f2, f2));
                const __half2 hh = __float22half2_rn(x);
                qf[c][nt][e] = *reinterpret_cast<const uint32_t*>(&hh);
              }
            // the scale's inverse, for the two heads whose logits this lane holds
            // (not below the normal numbers: a masked logit's -infinity times it stays one)
            const float inv = fmaxf(p.scale * pow2f(-(pw >> 1)) * pow2f((pw >> 1) - pw), 0x1p-126f);
            qs[nt].x = __shfl_sync(0xFFFFFFFFu, inv, 4 * (2 * (lane & 3)));
            qs[nt].y = __shfl_sync(0xFFFFFFFFu, inv, 4 * (2 * (lane & 3) + 1));
          }
          m[nt] = vm[nt] = make_float2(-INFINITY, -INFINITY);
          l[nt] = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < KSTEPS; ++c) acc[c][nt][0] = acc[c][nt][1] = make_float2(0.f, 0.f);
        }
      }

      const uint32_t st = ring + stage * C::STAGE;
      const uint32_t mask = lds32(st + C::STAGE - 16);
      if (mask != 0) {
        if constexpr (FMT == CF_MXFP4) prepare_scales<C>(st + C::KV, prep, lane, p.D);
        // ---- logits: lane holds tokens lane / 4 and + 8 of each 16, heads 2 (lane % 4) and + 1
        float2 s[MT][NT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[mt][nt][e] = make_float2(0.f, 0.f);
          if constexpr (FMT == CF_BF16) {
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c) {
              uint32_t a[4];
              ldsm4(a, st + chunk_at<FMT, ROW>(16 * mt + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma2_bf16(s[mt][nt], a, qf[c][nt]);
            }
          } else if constexpr (FMT == CF_MXFP4) {
            // a group's two steps, then its sums times the group's scale of each of the lane's rows
            float ks[2][C::NG];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int g = 0; g < C::NG; g += 2) {
                const uint2 x = lds64(prep + C::NG * 4 * (16 * mt + 8 * e + lane / 4) + 4 * g);
                ks[e][g] = __uint_as_float(x.x);
                ks[e][g + 1] = __uint_as_float(x.y);
              }
#pragma unroll
            for (int g = 0; g < C::NG; ++g) {
              uint32_t w[2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e)
                e2m1x8_to_f16x8(lds32(st + chunk_at<FMT, ROW>(16 * mt + 8 * e + lane / 4, g) + 4 * (lane & 3)), w[e]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float2 x[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t a[4] = {w[0][2 * i], w[1][2 * i], w[0][2 * i + 1], w[1][2 * i + 1]};
                  mma2_f16(x, a, qf[2 * g + i][nt]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  s[mt][nt][e] = g == 0 ? mul2(x[e], make_float2(ks[e][0], ks[e][0]))
                                        : fma2(x[e], make_float2(ks[e][g], ks[e][g]), s[mt][nt][e]);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < DP / 64; ++j) {
              const uint4 r0 = lds128(st + chunk_at<FMT, ROW>(16 * mt + lane / 4, 4 * j + (lane & 3)));
              const uint4 r1 = lds128(st + chunk_at<FMT, ROW>(16 * mt + 8 + lane / 4, 4 * j + (lane & 3)));
              const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t a[4];
                e4m3x4_f16x4(w0[i], a[0], a[2]);
                e4m3x4_f16x4(w1[i], a[1], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma2_f16(s[mt][nt], a, qf[4 * j + i][nt]);
              }
            }
          }
        }
        // ---- weights: 2^(logit - maximum), the logits (in powers of two) rounded before the maximum
        // is taken off, so that the largest weight is 1 whatever their size.  E4M3: a value's scale is
        // added to its weight's exponent, next to the maximum (beside a large logit it would have no
        // digits left), and the sums of values have a maximum of their own (vm, on top of m)
        float lvs[MT][2];  // log2 of the values' scales
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 16 * mt + lane / 4 + 8 * e;
            float ks = 1.f;
            if constexpr (FMT == CF_MXFP4) lvs[mt][e] = lds_f32(prep + 6 * C::NG * TW + 4 * r);
            if constexpr (FMT == CF_E4M3) {
              ks = lds_f32(st + C::KV + 4 * r);
              lvs[mt][e] = lg2(lds_f32(st + C::KV + 4 * (TW + r)));
            }
            const bool ok = (mask >> r) & 1u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (FMT == CF_E4M3) s[mt][nt][e] = mul2(s[mt][nt][e], make_float2(ks, ks));
              s[mt][nt][e] = mul2(s[mt][nt][e], qs[nt]);
              if (mask != 0xFFFFFFFFu && !ok) s[mt][nt][e] = make_float2(-INFINITY, -INFINITY);
            }
          }
        uint32_t pf[MT][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          auto warp_max = [&](float2 t) {  // of the largest of s
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 2; ++e) t = make_float2(fmaxf(t.x, s[mt][nt][e].x), fmaxf(t.y, s[mt][nt][e].y));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              t.x = fmaxf(t.x, __shfl_xor_sync(0xFFFFFFFFu, t.x, o));
              t.y = fmaxf(t.y, __shfl_xor_sync(0xFFFFFFFFu, t.y, o));
            }
            return t;
          };
          // a maximum moved to what is here now; f: what old sums shrink by, d: the exponents' base, negated
          auto rebase = [](float& top, float now, float& f, float& d) {
            const float m1 = fmaxf(top, now), base = m1 == -INFINITY ? 0.f : m1;
            f = ex2(top - base);
            top = m1;
            d = -base;
          };
          const float2 t = warp_max(s[0][nt][0]), old = m[nt];
          float2 fall, down;
          rebase(m[nt].x, t.x, fall.x, down.x);
          rebase(m[nt].y, t.y, fall.y, down.y);
          l[nt] = mul2(l[nt], fall);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 x = add2(s[mt][nt][e], down), pr = make_float2(ex2(x.x), ex2(x.y));
              l[nt] = add2(l[nt], pr);  // (a masked token's logit is -infinity: weight 0)
              if constexpr (FMT != CF_BF16) {
                s[mt][nt][e] = add2(x, make_float2(lvs[mt][e], lvs[mt][e]));
              } else {
                const __nv_bfloat162 hh = __float22bfloat162_rn(pr);
                pf[mt][nt][e] = movm(*reinterpret_cast<const uint32_t*>(&hh));
              }
            }
          if constexpr (FMT != CF_BF16) {
            const float2 tv = warp_max(s[0][nt][0]);
            float2 vdown;
            vm[nt] = add2(vm[nt], add2(old, down));
            rebase(vm[nt].x, tv.x - TOP, fall.x, vdown.x);
            rebase(vm[nt].y, tv.y - TOP, fall.y, vdown.y);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float2 y = add2(s[mt][nt][e], vdown);
                const __half2 hh = __floats2half2_rn(ex2(y.x), ex2(y.y));
                pf[mt][nt][e] = movm(*reinterpret_cast<const uint32_t*>(&hh));
              }
          }
          if (__any_sync(0xFFFFFFFFu, fall.x != 1.f || fall.y != 1.f))
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e) acc[c][nt][e] = mul2(acc[c][nt][e], fall);
        }
        // ---- values: lane holds dims lane / 4 and + 8 of each 16 (E4M3: 2 (lane / 4) and + 1)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint32_t vt = st + TW * ROW;
          if constexpr (FMT == CF_BF16) {
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c) {
              uint32_t a[4];
              ldsm4t(a, vt + chunk_at<FMT, ROW>(16 * mt + (lane & 7) + ((lane >> 4) << 3), 2 * c + ((lane >> 3) & 1)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma2_bf16(acc[c][nt], a, pf[mt][nt]);
            }
          } else if constexpr (FMT == CF_MXFP4) {
            uint32_t f[2][C::NG];  // the groups' factors of the lane's tokens, two at a time as pf has them
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int g = 0; g < C::NG; g += 2) {
                const uint2 x = lds64(prep + 4 * C::NG * TW + 4 * C::NG * (8 * mt + 4 * e + (lane & 3)) + 4 * g);
                f[e][g] = x.x;
                f[e][g + 1] = x.y;
              }
#pragma unroll
            for (int g = 0; g < C::NG; g += 2) {
              // lane: four dims of group g (v[0], v[1]) and g + 1 of tokens 2 (lane % 4) and + 1, and + 8
              uint32_t v[4];
              ldsm4t(v, vt + chunk_at<FMT, ROW>(16 * mt + (lane & 15), g + (lane >> 4)));
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                // a byte of ev, od: a dim's codes of a token and the next one
                const uint32_t x = __byte_perm(v[2 * i], v[2 * i + 1], 0x5410), y = __byte_perm(v[2 * i], v[2 * i + 1], 0x7632);
                const uint32_t ev = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), od = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
                uint32_t a[4], b[4];
                e2m1x8_to_f16x8(ev, a);
                e2m1x8_to_f16x8(od, b);
                const uint32_t a0[4] = {a[0], b[0], a[2], b[2]}, a1[4] = {a[1], b[1], a[3], b[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint32_t w[2] = {hmul2(pf[mt][nt][0], f[0][g + i]), hmul2(pf[mt][nt][1], f[1][g + i])};
                  mma2_f16(acc[2 * (g + i)][nt], a0, w);
                  mma2_f16(acc[2 * (g + i) + 1][nt], a1, w);
                }
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < KSTEPS; c += 2) {
              uint32_t v[4];
              ldsm4t(v, vt + chunk_at<FMT, ROW>(16 * mt + (lane & 15), c + (lane >> 4)));
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // bytes (t, d) (t, d + 1) (t + 1, d) (t + 1, d + 1) -> the two tokens of each dim
                uint32_t a[4];
                e4m3x4_f16x4(__byte_perm(v[2 * e], 0, 0x3120), a[0], a[1]);
                e4m3x4_f16x4(__byte_perm(v[2 * e + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma2_f16(acc[c + e][nt], a, pf[mt][nt]);
              }
            }
          }
        }
      }
      const int used = stage * C::STAGE;  // this tile's stage: read out, copied over in the next turn
      stage = stage == STAGES - 1 ? 0 : stage + 1;

      // ---- the end of a part: join the warps, then write the result or leave a record
      const DecAt now = at;
      at.next(p, ulog, end, start);
      if (!at.in(end, whole_units, start) || now.u == now.nu - 1) {
        const bool whole = part_u0 == 0 && now.u == now.nu - 1;
        cut |= !whole;
        const int64_t row0 = (int64_t)now.b * p.Hq + head0;
        float* const rec = p.parts + (2 * worker + part_slot) * C::REC;
        // the warps trade maxima and sums of weights, bring their sums to the team's maximum and
        // lay them out in the stage, where the team adds them up
        const int w0 = team << wlog;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            l[nt].x += __shfl_xor_sync(0xFFFFFFFFu, l[nt].x, o);
            l[nt].y += __shfl_xor_sync(0xFFFFFFFFu, l[nt].y, o);
          }
          if (lane < 4)
            *reinterpret_cast<float4*>(s_ml + 2 * (warp * HEADS + nt * 8 + 2 * lane)) =
                make_float4(m[nt].x, l[nt].x, m[nt].y, l[nt].y);
        }
        team_sync(team, tthreads);
        float2 f[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float4 ml[WARPS];
          float2 top = make_float2(-INFINITY, -INFINITY), sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            ml[w] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
            if (w < W) ml[w] = *reinterpret_cast<const float4*>(s_ml + 2 * ((w0 + w) * HEADS + nt * 8 + 2 * (lane & 3)));
            top = make_float2(fmaxf(top.x, ml[w].x), fmaxf(top.y, ml[w].z));
          }
          const float2 base = make_float2(top.x == -INFINITY ? 0.f : top.x, top.y == -INFINITY ? 0.f : top.y);
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            sum.x = fmaf(ml[w].y, ex2(ml[w].x - base.x), sum.x);
            sum.y = fmaf(ml[w].w, ex2(ml[w].z - base.y), sum.y);
          }
          if constexpr (FMT != CF_BF16)
            f[nt] = make_float2(ex2(vm[nt].x + (m[nt].x - base.x)), ex2(vm[nt].y + (m[nt].y - base.y)));
          else
            f[nt] = make_float2(ex2(m[nt].x - base.x), ex2(m[nt].y - base.y));
          if (whole) {  // (a sum of 0: nothing was attended to, the sums are 0 too)
            f[nt].x = sum.x == 0.f ? 0.f : f[nt].x / sum.x;
            f[nt].y = sum.y == 0.f ? 0.f : f[nt].y / sum.y;
          }
          const int h = nt * 8 + 2 * (lane & 3);
          if (tw == 0 && lane < 4 && h < heads) {
            if (!whole) {
              *reinterpret_cast<float2*>(rec + HEADS * DP + 2 * h) = make_float2(top.x, sum.x);
              *reinterpret_cast<float2*>(rec + HEADS * DP + 2 * h + 2) = make_float2(top.y, sum.y);
            } else if (p.lse) {
              p.lse[row0 + h] = lse_of(base.x, sum.x);
              if (h + 1 < heads) p.lse[row0 + h + 1] = lse_of(base.y, sum.y);
            }
          }
        }
        float* const mine_out = reinterpret_cast<float*>(smem + warp * STAGES * C::STAGE + used);
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += C::PN) {
          // dim d of head h at d ^ (h / 2 % 4 * 8): the heads of a fragment lie in different banks
#pragma unroll
          for (int n = 0; n < C::PN; ++n)
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c) {
              const float2 a = mul2(acc[c][n0 + n][0], f[n0 + n]), b = mul2(acc[c][n0 + n][1], f[n0 + n]);
              float* const x = mine_out + (8 * n + 2 * (lane & 3)) * DP;
              if constexpr (FMT == CF_BF16) {
                const int d0 = (16 * c + lane / 4) ^ ((lane & 3) << 3), d1 = (16 * c + lane / 4 + 8) ^ ((lane & 3) << 3);
                x[d0] = a.x;
                x[d1] = b.x;
                x[DP + d0] = a.y;
                x[DP + d1] = b.y;
              } else {
                const int d0 = (FMT == CF_MXFP4 ? 32 * (c / 2) + 4 * (lane / 4) + 2 * (c & 1) : 16 * c + 2 * (lane / 4)) ^
                               ((lane & 3) << 3);
                *reinterpret_cast<float2*>(x + d0) = make_float2(a.x, b.x);
                *reinterpret_cast<float2*>(x + DP + d0) = make_float2(a.y, b.y);
              }
            }
          if (EARLY && n0 + C::PN >= NT && at.in(end, whole_units, start)) load_queries(at);
          team_sync(team, tthreads);
          const int hs = min(heads - 8 * n0, 8 * C::PN);
#pragma unroll 2
          for (int i = tthread; i < hs * (DP / 4); i += tthreads) {
            const int hp = i / (DP / 4), h = 8 * n0 + hp, d = 4 * (i % (DP / 4));
            const uint8_t* const x = smem + w0 * STAGES * C::STAGE + used + 4 * (hp * DP + (d ^ ((hp >> 1 & 3) << 3)));
            float4 o = *reinterpret_cast<const float4*>(x);
#pragma unroll
            for (int w = 1; w < WARPS; ++w) {
              if (w >= W) continue;
              const float4 v = *reinterpret_cast<const float4*>(x + w * STAGES * C::STAGE);
              o.x += v.x;
              o.y += v.y;
              o.z += v.z;
              o.w += v.w;
            }
            if (!whole)
              *reinterpret_cast<float4*>(rec + h * DP + d) = o;
            else if (d < p.D)
              *reinterpret_cast<uint2*>(p.out + (row0 + h) * p.D + d) = bf16x4(o.x, o.y, o.z, o.w);
          }
          team_sync(team, tthreads);
        }
        if (p.D < DP) {  // the dims past D of the stage are zero again
          const int pad = CPR - cpr;
          for (int i = lane; i < 2 * TW * pad; i += 32) {
            const int r = i / pad, ch = cpr + i % pad;
            *reinterpret_cast<uint4*>(smem + warp * STAGES * C::STAGE + used + (r < TW ? 0 : TW * ROW) +
                                      chunk_at<FMT, ROW>(r & (TW - 1), ch)) = make_uint4(0, 0, 0, 0);
          }
        }
        if (!whole && tthread == 0) {
          // the teams of this (sequence, head group), whose first unit is i0 of all
          const int64_t i0 = unit0 + now.x - now.u;
          const int32_t c0 = (int32_t)div64(i0, chunk), c1 = (int32_t)div64(i0 + now.nu - 1, chunk);
          s_part[2 * team + part_slot] = DecPart{i0, row0, c0, c1 - c0 + 1, heads, 1};
          (part_slot ? got[1] : got[0]) = arrive(p.arrived + c0);
        }
      }
    }
    cp_async_wait<0>();

    // ---- parts: the team that arrived last joins a sequence's records
#pragma unroll
    for (int slot = 0; slot < 2 && cut; ++slot) {
      __syncwarp();
      if (tthread == 0)
        s_last[team] = s_part[2 * team + slot].there && got[slot] == (uint32_t)(s_part[2 * team + slot].parts - 1);
      team_sync(team, tthreads);
      if (s_last[team]) {
        const DecPart x = s_part[2 * team + slot];
        if (tthread == 0) p.arrived[x.c0] = 0;
        // SIDE quads of dims a thread and some records at a time, whose loads are in flight
        // together: 8 / SIDE of few records, 32 / SIDE of more than 16 (1 x 64000 tokens, 8 heads,
        // D 128, bf16 18.7 us, 21.9 at 8; E4M3 18.5, 19.8; but 8 x 1000 tokens 11.2, 10.6 at 8).
        // 16 heads keep to 8: the registers cost them more (201 windowed sequences 64.8 us, 63.5)
        constexpr int QUADS = HEADS * DP / 4 / THREADS, SIDE = QUADS >= 4 ? 4 : QUADS >= 2 ? 2 : 1;
        for (int i0 = tthread; i0 < x.heads * (DP / 4); i0 += SIDE * tthreads) {
          float top[SIDE], sum[SIDE], o[SIDE][4];
          int h[SIDE], d[SIDE];
#pragma unroll
          for (int s = 0; s < SIDE; ++s) {
            const int i = i0 + s * tthreads;
            h[s] = i / (DP / 4);
            d[s] = 4 * (i % (DP / 4));
            top[s] = -INFINITY;
            sum[s] = o[s][0] = o[s][1] = o[s][2] = o[s][3] = 0.f;
          }
          auto take = [&](int j0, auto at_once) {
            constexpr int BATCH = decltype(at_once)::value;
            float2 ml[SIDE][BATCH];
            float4 v[SIDE][BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
              // team c0's part is in its slot 0 where it begins at the team's first place
              const int at_second = j0 + j == 0 && x.i0 - x.c0 * chunk > start;
              const float* y = p.parts + (2 * (int64_t)(x.c0 + j0 + j) + at_second) * C::REC;
#pragma unroll
              for (int s = 0; s < SIDE; ++s) {
                ml[s][j] = make_float2(-INFINITY, 0.f);
                v[s][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j0 + j < x.parts && h[s] < x.heads) {
                  ml[s][j] = __ldcg(reinterpret_cast<const float2*>(y + HEADS * DP + 2 * h[s]));
                  v[s][j] = __ldcg(reinterpret_cast<const float4*>(y + h[s] * DP + d[s]));
                }
              }
            }
#pragma unroll
            for (int s = 0; s < SIDE; ++s) {
              float m1 = top[s];
#pragma unroll
              for (int j = 0; j < BATCH; ++j) m1 = fmaxf(m1, ml[s][j].x);
              const float base = m1 == -INFINITY ? 0.f : m1, fall = ex2(top[s] - base);
              top[s] = m1;
              sum[s] *= fall;
#pragma unroll
              for (int e = 0; e < 4; ++e) o[s][e] *= fall;
#pragma unroll
              for (int j = 0; j < BATCH; ++j) {
                const float f = ex2(ml[s][j].x - base);
                sum[s] = fmaf(ml[s][j].y, f, sum[s]);
                o[s][0] = fmaf(v[s][j].x, f, o[s][0]);
                o[s][1] = fmaf(v[s][j].y, f, o[s][1]);
                o[s][2] = fmaf(v[s][j].z, f, o[s][2]);
                o[s][3] = fmaf(v[s][j].w, f, o[s][3]);
              }
            }
          };
          if (NT == 1 && x.parts > 16)
            for (int j0 = 0; j0 < x.parts; j0 += 32 / SIDE) take(j0, std::integral_constant<int, 32 / SIDE>());
          else
            for (int j0 = 0; j0 < x.parts; j0 += 8 / SIDE) take(j0, std::integral_constant<int, 8 / SIDE>());
#pragma unroll
          for (int s = 0; s < SIDE; ++s) {
            if (h[s] >= x.heads) continue;
            const float r = sum[s] == 0.f ? 0.f : 1.f / sum[s];
            if (d[s] < p.D)
              *reinterpret_cast<uint2*>(p.out + (x.row + h[s]) * p.D + d[s]) =
                  bf16x4(o[s][0] * r, o[s][1] * r, o[s][2] * r, o[s][3] * r);
            if (d[s] == 0 && p.lse) p.lse[x.row + h[s]] = lse_of(top[s], sum[s]);
          }
        }
      }
      team_sync(team, tthreads);
    }
  }

  // ---- sequences with no tokens
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    bool bad;
    if (seq_len(p, b, bad) != 0) continue;
    for (int i = threadIdx.x; i < p.Hq * p.D / 8; i += THREADS)
      *reinterpret_cast<uint4*>(p.out + (int64_t)b * p.Hq * p.D + 8 * i) = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = threadIdx.x; i < p.Hq; i += THREADS) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
  }
}

}  // namespace k3
