// k3_qkv.cuh -- norms of queries and keys per head with the position rotation, and the rows of
// the paged cache: written (bf16, or E4M3 codes with a row scale) and read back.
//
// All of it moves each byte once; HBM is the floor (GB300, copy rate 6789 GB/s).  Measured: read
// of 100003 tokens of 8 E4M3 heads of 128 at 98% of the copy rate, import of 65536 at 83%
// (issue slots: the quantisation), norms of 16381 tokens of 72 heads at 79% and the append of
// 8192 tokens at 68% (warps waiting at the barrier for their token's angles, the largest stall; then
// issue slots, 66 and 61% used; fp64 units 9 and 8%).  Few heads a token are bound by the fp64 units
// that form the angles, twice a token in an append: 65536 tokens of 4 query heads and 1 key head of
// 128 take 118 us into an E4M3 cache (23%; fp64 units 68% busy), norms alone 63 us (39%).
//
// A row (a head of a token) is taken by 8, 16 or 32 lanes, eight elements a lane, and a thread
// has the loads of up to QKV_ROWS rows in flight before it waits for any.
#pragma once

#include <cuda_fp8.h>

#include "../k3_common.cuh"
#include "../../../include/k3attn.h"

namespace k3 {

enum { CF_NONE = -1, CF_BF16 = K3ATTN_BF16, CF_E4M3 = K3ATTN_E4M3 };

// two fp32 at once
K3_DEVI float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&r);
}
K3_DEVI float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return *reinterpret_cast<const float2*>(&r);
}

// n / d for n < 2^31 as the high half of a product: with 2^shift >= d and mul = floor(2^32
// (2^shift - d) / d) + 1 it is (umulhi(n, mul) + n) >> shift
struct Divisor {
  uint32_t mul, shift;
  static Divisor of(uint32_t d) {
    Divisor x{0, 0};
    while ((1u << x.shift) < d) ++x.shift;
    x.mul = (uint32_t)(((((uint64_t)1 << x.shift) - d) << 32) / d + 1);
    return x;
  }
  K3_DEVI uint32_t operator()(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// the cache as the kernels address it: strides of the rows in bytes, of the scales in elements
struct CacheView {
  uint8_t *k, *v;
  float *ks, *vs;
  int64_t page, head, tok;
  int64_t spage, shead, stok;
  int32_t n_pages, page_size;
  Divisor by_page;
};

struct QkvParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int32_t T, Hq, Hkv, D, R, inter;
  float eps;
  const int32_t *pos, *slots;
  const double* inv_freq;
  const float *q_w, *k_w;
  uint16_t *q_out, *k_out, *v_out;
  CacheView c;
  uint32_t* status;
  int32_t tokens, rows, parts;             // norms: a block's tokens, rows of each, blocks for them all
  int32_t kv_blocks, kv_tokens, kv_warps;  // the keys' and values' blocks, their tokens, warps of each
  Divisor by_heads;                        // rows: by Hkv
};

constexpr int QKV_THREADS = 512;  // most threads of a block
constexpr int QKV_ROWS = 4;       // rows of a thread in flight
constexpr int QKV_TOKENS = 8;     // most tokens of a block of the norms
// Registers of the norm kernel: warps in flight count for more than the few spilled words
// (16381 tokens of 72 heads of 128: 112 us at 56 registers, 121 at 64, 114 at 52; the append of
// 8192 tokens to an E4M3 cache: 69 us at 64, 75 at 56, 78 at 72).  One row a thread: all it asks.
constexpr int qkv_registers(int fmt, int rows) { return rows == 1 ? 128 : (fmt == CF_NONE ? 56 : 64); }
constexpr float E4M3_MAX = 448.0f;
constexpr float KV_MIN_SCALE = 0x1p-100f;  // its reciprocal and 448 times it are normal numbers

// cos and sin of pos * f: the product in turns in fp64, its whole turns taken off there (a far
// position's angle has no digits left in fp32), the rest in [-1/2, 1/2] turns rounded to fp32
K3_DEVI void rotation(int32_t pos, double f, float& c, float& s) {
  const double turns = (double)pos * (f * 0.15915494309189535);
  sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
}

// eight bf16 as four pairs of fp32, and back
K3_DEVI void unpack8(uint4 v, float2 (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
K3_DEVI uint4 pack8(const float2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __float22bfloat162_rn(x[i]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// eight values to E4M3 (round to nearest even, saturated)
K3_DEVI uint2 e4m3x8(const float2 (&x)[4]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __nv_cvt_float2_to_fp8x2(x[i], __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
// eight E4M3 codes times s, rounded to bf16
K3_DEVI uint4 e4m3x8_bf16(uint2 c, float s) {
  float2 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2_raw hr =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((k < 2 ? c.x : c.y) >> (16 * (k & 1))), __NV_E4M3);
    x[k] = mul2(__half22float2(__half2(hr)), make_float2(s, s));
  }
  return pack8(x);
}

// The place of a slot in the cache.
struct Place {
  int64_t page;
  int32_t at;
  bool ok;
};
K3_DEVI Place place_of(const QkvParams& p, int32_t slot, bool report) {
  Place x{0, 0, false};
  if (slot >= 0) {
    const int32_t pg = (int32_t)p.c.by_page(slot);
    x.ok = pg < p.c.n_pages;
    x.page = x.ok ? pg : 0;
    x.at = x.ok ? slot - pg * p.c.page_size : 0;
  }
  if (!x.ok && slot != -1 && report) flag_status(p.status, K3ATTN_DEV_BAD_SLOT);
  return x;
}

// byte offset of a head's row at a place, and the place of its scale
K3_DEVI int64_t row_at(const QkvParams& p, const Place& pl, int h) {
  return pl.page * p.c.page + (h * p.c.head + pl.at * p.c.tok);
}
K3_DEVI int64_t scale_at(const QkvParams& p, const Place& pl, int h) {
  return pl.page * p.c.spage + (h * p.c.shead + pl.at * p.c.stok);
}

// The largest magnitude of a row by its bits, where infinities and NaN order above every number
// (all lanes of a row get it): of fp32 values, of bf16 values (as an fp32's bits).
template <int LPR>
K3_DEVI uint32_t row_max(const float2 (&y)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = max(m, max(__float_as_uint(y[i].x) & 0x7FFFFFFFu, __float_as_uint(y[i].y) & 0x7FFFFFFFu));
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m;
}
template <int LPR>
K3_DEVI uint32_t row_max(uint4 raw) {
  constexpr uint32_t ABS = 0x7FFF7FFFu;
  uint32_t m = __vmaxu2(__vmaxu2(raw.x & ABS, raw.y & ABS), __vmaxu2(raw.z & ABS, raw.w & ABS));
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return max(m & 0xFFFF0000u, m << 16);
}
// a row's scale from its largest magnitude
K3_DEVI float scale_of(uint32_t m) {
  return m < 0x7F800000u ? fmaxf(__uint_as_float(m) / E4M3_MAX, KV_MIN_SCALE) : __uint_as_float(0x7FC00000u);
}
// The scales of a key's and a value's row, and their inverses: even lanes form the key's, odd
// ones the value's (s: the lane's own), and trade the inverses.
K3_DEVI void scales_of(uint32_t mk, uint32_t mv, int li, float& s, float& ik, float& iv) {
  const bool odd = li & 1;
  s = scale_of(odd ? mv : mk);
  const float own = 1.0f / s, other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
  ik = odd ? other : own;
  iv = odd ? own : other;
}
// a lane's eight codes of a row, given the inverse of its scale
K3_DEVI uint2 codes_of(const float2 (&y)[4], float inv) {
  float2 z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = mul2(y[i], make_float2(inv, inv));
  return e4m3x8(z);
}

// What a lane multiplies its pieces of normed rows of one kind (queries or keys) of one token by:
// y = x * co + z * si, z the other element of x's pair; without rotation co is the weight alone.
struct Turn {
  float2 co[4], si[4];
  // the pieces of four elements at ea and eb; c, s: cos and sin from this lane's first angle
  K3_DEVI void form(const QkvParams& p, const float* w, int ea, int eb, bool rotated, const float* cp,
                    const float* sp) {
    const float4 wa = __ldg(reinterpret_cast<const float4*>(w + ea));
    const float4 wb = __ldg(reinterpret_cast<const float4*>(w + eb));
    co[0] = make_float2(wa.x, wa.y);
    co[1] = make_float2(wa.z, wa.w);
    co[2] = make_float2(wb.x, wb.y);
    co[3] = make_float2(wb.z, wb.w);
    if (!rotated) return;
    const float4 c = *reinterpret_cast<const float4*>(cp), s = *reinterpret_cast<const float4*>(sp);
    if (p.inter) {  // pairs are (x, y) of each of the four
      const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        si[k] = make_float2(-co[k].y * sn[k], co[k].x * sn[k]);
        co[k] = mul2(co[k], make_float2(cc[k], cc[k]));
      }
    } else {  // 0 with 2, 1 with 3
      si[0] = make_float2(-co[2].x * s.x, -co[2].y * s.y);
      si[1] = make_float2(-co[3].x * s.z, -co[3].y * s.w);
      si[2] = mul2(co[0], make_float2(s.x, s.y));
      si[3] = mul2(co[1], make_float2(s.z, s.w));
      const float2 c0 = make_float2(c.x, c.y), c1 = make_float2(c.z, c.w);
      co[0] = mul2(co[0], c0);
      co[1] = mul2(co[1], c1);
      co[2] = mul2(co[2], c0);
      co[3] = mul2(co[3], c1);
    }
  }
  K3_DEVI void with(const QkvParams& p, bool rotated, float2 (&x)[4], float2 z0, float2 z1, float2 z2,
                    float2 z3) const {
    const float2 z[4] = {z0, z1, z2, z3};
    float2 y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = mul2(x[k], co[k]);
    if (p.R == p.D || rotated)
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = fma2(z[k], si[k], y[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = y[k];
  }
  // x: a row's pieces -> normed and rotated (all lanes of a warp call it: the sum over the row)
  template <int LPR>
  K3_DEVI void apply(const QkvParams& p, float over_d, bool rotated, float2 (&x)[4]) const {
    float2 s2 = mul2(x[0], x[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) s2 = fma2(x[k], x[k], s2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const float rs = rsqrtf(ss * over_d + p.eps);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = mul2(x[k], make_float2(rs, rs));
    if (p.inter)
      with(p, rotated, x, make_float2(x[0].y, x[0].x), make_float2(x[1].y, x[1].x), make_float2(x[2].y, x[2].x),
           make_float2(x[3].y, x[3].x));
    else
      with(p, rotated, x, x[2], x[3], x[0], x[1]);
  }
};

// A lane's pieces of a row of queries or keys, four elements from ea and four from eb, and its
// first angle: the two halves of four rotated pairs (pairs (i, i + R/2)), or eight neighbours,
// so that pairs never cross lanes.
struct Pieces {
  int ea, eb, angle;
  bool on, rotated;
  K3_DEVI Pieces(const QkvParams& p, int li) {
    on = 8 * li < p.D;
    rotated = 8 * li < p.R;
    ea = 8 * li;
    eb = ea + 4;
    angle = ea / 2;
    if (!p.inter && rotated) {
      ea = angle = 4 * li;
      eb = ea + p.R / 2;
    }
  }
};

// Norms and rotation of dense rows (queries and, FMT none, keys), and with FMT bf16 or E4M3 the
// keys and values of the same tokens into the cache in the same launch: the first p.kv_blocks
// blocks take those, a head's key and value together.
//
// A block of the dense rows has p.rows rows of each of p.tokens tokens, LPR lanes a row and up
// to ROWS rows a thread, whose loads it issues before it forms the token's angles (fp64 products
// and one sine and cosine per token and pair, shared by the block).  A thread's pieces are the
// same in all its rows, so that it keeps the products of weights and angles in registers and a
// row takes 12 packed operations for its norm and rotation.
template <int LPR, int FMT, int ROWS>
__global__ void __maxnreg__(qkv_registers(FMT, ROWS)) k3_norm_kernel(const QkvParams p) {
  __shared__ __align__(16) float s_cos[QKV_TOKENS][128], s_sin[QKV_TOKENS][128];
  const int half = p.R / 2;
  const float over_d = 1.0f / (float)p.D;
  grid_dep_wait();
  grid_dep_launch();

  if (FMT != CF_NONE && (int)blockIdx.x < p.kv_blocks) {
    constexpr int ITEMS = ROWS > 1 ? 2 : 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, group = warp / p.kv_warps;
    const int li = lane % LPR, sub = (warp - group * p.kv_warps) * (32 / LPR) + lane / LPR;
    const int subs = p.kv_warps * (32 / LPR);
    const int t0 = blockIdx.x * p.kv_tokens, nt = min(p.kv_tokens, p.T - t0);
    const bool mine = group < nt;
    const int64_t t = t0 + (mine ? group : 0);
    const Pieces pc(p, li);
    const int32_t slot = mine ? p.slots[t] : -1;
    const uint16_t *kp = p.k + t * p.k_stride, *vp = p.v + t * p.v_stride;
    uint2 ra[ITEMS], rb[ITEMS];
    uint4 rv[ITEMS];
    auto load = [&](int first) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int h = first + i * subs;
        ra[i] = rb[i] = make_uint2(0, 0);
        rv[i] = make_uint4(0, 0, 0, 0);
        if (mine && h < p.Hkv && pc.on) {
          ra[i] = *reinterpret_cast<const uint2*>(kp + h * p.D + pc.ea);
          rb[i] = *reinterpret_cast<const uint2*>(kp + h * p.D + pc.eb);
          rv[i] = *reinterpret_cast<const uint4*>(vp + h * p.D + 8 * li);
        }
      }
    };
    load(sub);
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
      const int g = i / half, j = i - g * half;
      rotation(p.pos[t0 + g], p.inv_freq[j], s_cos[g][j], s_sin[g][j]);
    }
    const Place pl = place_of(p, slot, sub == 0 && li == 0);
    const int64_t row0 = row_at(p, pl, 0), scale0 = FMT == CF_E4M3 ? scale_at(p, pl, 0) : 0;
    __syncthreads();
    if (!mine) return;  // the whole warp
    Turn turn{};
    if (pc.on)
      turn.form(p, p.k_w, pc.ea, pc.eb, pc.rotated, &s_cos[group][pc.angle], &s_sin[group][pc.angle]);
    for (int first = 0; first < p.Hkv; first += ITEMS * subs) {  // (of the whole warp)
      if (first > 0) load(first + sub);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int h = first + sub + i * subs;
        if (first + i * subs >= p.Hkv) break;
        const bool keep = h < p.Hkv && pc.on;
        float2 x[4];
        unpack8(make_uint4(ra[i].x, ra[i].y, rb[i].x, rb[i].y), x);
        turn.template apply<LPR>(p, over_d, pc.rotated, x);
        const uint4 kb = pack8(x);
        if (keep && p.k_out) {
          uint16_t* dst = p.k_out + (t * p.Hkv + h) * p.D;
          *reinterpret_cast<uint2*>(dst + pc.ea) = make_uint2(kb.x, kb.y);
          *reinterpret_cast<uint2*>(dst + pc.eb) = make_uint2(kb.z, kb.w);
        }
        const int64_t row = row0 + h * p.c.head;
        if constexpr (FMT == CF_BF16) {
          if (keep && pl.ok) {
            *reinterpret_cast<uint2*>(p.c.k + row + 2 * pc.ea) = make_uint2(kb.x, kb.y);
            *reinterpret_cast<uint2*>(p.c.k + row + 2 * pc.eb) = make_uint2(kb.z, kb.w);
            *reinterpret_cast<uint4*>(p.c.v + row + 16 * li) = rv[i];
          }
        } else {
          float s, ik, iv;
          scales_of(row_max<LPR>(x), row_max<LPR>(rv[i]), li, s, ik, iv);
          const uint2 kc = codes_of(x, ik);
          unpack8(rv[i], x);
          const uint2 vc = codes_of(x, iv);
          if (keep && pl.ok) {
            *reinterpret_cast<uint32_t*>(p.c.k + row + pc.ea) = kc.x;
            *reinterpret_cast<uint32_t*>(p.c.k + row + pc.eb) = kc.y;
            *reinterpret_cast<uint2*>(p.c.v + row + 8 * li) = vc;
            if (li < 2) (li ? p.c.vs : p.c.ks)[scale0 + h * p.c.shead] = s;
          }
        }
      }
    }
    return;
  }

  const int block = FMT == CF_NONE ? blockIdx.x : blockIdx.x - p.kv_blocks;
  const int tb = block / p.parts, part = block - tb * p.parts;
  const int warps = blockDim.x / 32 / p.tokens, warp = threadIdx.x / 32, group = warp / warps;
  const int lane = threadIdx.x % 32, li = lane % LPR;
  const int sub = (warp - group * warps) * (32 / LPR) + lane / LPR, subs = warps * (32 / LPR);
  const int t0 = tb * p.tokens, r0 = part * p.rows, nt = min(p.tokens, p.T - t0);
  const bool mine = group < nt;  // this warp's token: there is one
  const int64_t t = t0 + (mine ? group : 0);
  const int r1 = mine ? min(r0 + p.rows, p.Hq + (FMT == CF_NONE ? p.Hkv : 0)) : 0;
  const Pieces pc(p, li);
  // where row 0 would be, were all rows of its kind
  const uint16_t* const qs = p.q + t * p.q_stride;
  const uint16_t* const ks = p.k + t * p.k_stride - p.Hq * p.D;
  uint2 ra[ROWS], rb[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + sub + i * subs;
    ra[i] = rb[i] = make_uint2(0, 0);
    if (r < r1 && pc.on) {
      const uint16_t* src = (FMT != CF_NONE || r < p.Hq ? qs : ks) + r * p.D;
      ra[i] = *reinterpret_cast<const uint2*>(src + pc.ea);
      rb[i] = *reinterpret_cast<const uint2*>(src + pc.eb);
    }
  }
  if (mine)
    for (int i = threadIdx.x - 32 * group * warps; i < half; i += 32 * warps)
      rotation(p.pos[t], p.inv_freq[i], s_cos[group][i], s_sin[group][i]);
  __syncthreads();
  uint16_t* const qd = p.q_out + t * p.Hq * p.D;
  uint16_t* const kd = p.k_out + (t * p.Hkv - p.Hq) * p.D;
  Turn turn{};
  int have = -1;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + sub + i * subs;
    const bool there = r < r1 && pc.on, is_q = FMT != CF_NONE || r < p.Hq;
    if (!__any_sync(0xFFFFFFFFu, there)) break;
    if (there && have != (int)is_q) {
      have = is_q;
      turn.form(p, is_q ? p.q_w : p.k_w, pc.ea, pc.eb, pc.rotated, &s_cos[group][pc.angle], &s_sin[group][pc.angle]);
    }
    float2 x[4];
    unpack8(make_uint4(ra[i].x, ra[i].y, rb[i].x, rb[i].y), x);
    turn.template apply<LPR>(p, over_d, pc.rotated, x);
    if (there) {
      const uint4 raw = pack8(x);
      uint16_t* dst = (is_q ? qd : kd) + r * p.D;
      *reinterpret_cast<uint2*>(dst + pc.ea) = make_uint2(raw.x, raw.y);
      *reinterpret_cast<uint2*>(dst + pc.eb) = make_uint2(raw.z, raw.w);
    }
  }
}

// Rows of the cache written from dense k, v (WRITE) or read back: an item is a head of a token,
// its key and its value, LPR lanes an item and ITEMS items a thread.  32 registers, so that an
// SM holds all its warps: the read of 100003 tokens of 8 E4M3 heads of 128 takes 93 us (98% of
// the copy rate; 100 us without the bound), the import of 65536 tokens 72 us (83%, against 85;
// by then bound by the instructions of the quantisation).
template <int LPR, int FMT, bool WRITE, int ITEMS>
__global__ void __launch_bounds__(256, ITEMS > 1 ? 8 : 1) k3_rows_kernel(const QkvParams p) {
  constexpr int SUBS = 256 / LPR;
  const int li = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const bool on = 8 * li < p.D;
  const int64_t first = (int64_t)blockIdx.x * (SUBS * ITEMS);
  const int32_t t0 = (int32_t)(first / p.Hkv), rest = (int32_t)(first - (int64_t)t0 * p.Hkv);
  grid_dep_wait();
  grid_dep_launch();
  int32_t tok[ITEMS], head[ITEMS], slot[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int32_t it = rest + sub + i * SUBS, dt = (int32_t)p.by_heads(it);
    head[i] = it - dt * p.Hkv;
    tok[i] = dt < p.T - t0 ? t0 + dt : -1;
    slot[i] = tok[i] >= 0 ? p.slots[tok[i]] : -1;
  }
  uint4 k[ITEMS], v[ITEMS];
  float ks[ITEMS], vs[ITEMS];
  Place pl[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    pl[i] = place_of(p, slot[i], li == 0);
    k[i] = v[i] = make_uint4(0, 0, 0, 0);
    ks[i] = vs[i] = 0.f;
    if (!on || !pl[i].ok) continue;
    if constexpr (WRITE) {
      const int32_t o = head[i] * p.D + 8 * li;
      k[i] = *reinterpret_cast<const uint4*>(p.k + tok[i] * p.k_stride + o);
      v[i] = *reinterpret_cast<const uint4*>(p.v + tok[i] * p.v_stride + o);
    } else {
      const int64_t o = row_at(p, pl[i], head[i]);
      if constexpr (FMT == CF_BF16) {
        k[i] = *reinterpret_cast<const uint4*>(p.c.k + o + 16 * li);
        v[i] = *reinterpret_cast<const uint4*>(p.c.v + o + 16 * li);
      } else {
        const uint2 kc = *reinterpret_cast<const uint2*>(p.c.k + o + 8 * li);
        const uint2 vc = *reinterpret_cast<const uint2*>(p.c.v + o + 8 * li);
        k[i].x = kc.x; k[i].y = kc.y;
        v[i].x = vc.x; v[i].y = vc.y;
        const int64_t so = scale_at(p, pl[i], head[i]);
        ks[i] = p.c.ks[so];
        vs[i] = p.c.vs[so];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if constexpr (WRITE) {
      const int64_t o = row_at(p, pl[i], head[i]);
      if constexpr (FMT == CF_BF16) {
        if (on && pl[i].ok) {
          *reinterpret_cast<uint4*>(p.c.k + o + 16 * li) = k[i];
          *reinterpret_cast<uint4*>(p.c.v + o + 16 * li) = v[i];
        }
      } else {
        float s, ik, iv;
        scales_of(row_max<LPR>(k[i]), row_max<LPR>(v[i]), li, s, ik, iv);
        float2 x[4];
        unpack8(k[i], x);
        const uint2 kc = codes_of(x, ik);
        unpack8(v[i], x);
        const uint2 vc = codes_of(x, iv);
        if (on && pl[i].ok) {
          *reinterpret_cast<uint2*>(p.c.k + o + 8 * li) = kc;
          *reinterpret_cast<uint2*>(p.c.v + o + 8 * li) = vc;
          if (li < 2) (li ? p.c.vs : p.c.ks)[scale_at(p, pl[i], head[i])] = s;
        }
      }
    } else if (on && tok[i] >= 0) {
      if constexpr (FMT == CF_E4M3) {
        k[i] = e4m3x8_bf16(make_uint2(k[i].x, k[i].y), ks[i]);
        v[i] = e4m3x8_bf16(make_uint2(v[i].x, v[i].y), vs[i]);
      }
      const int64_t o = ((int64_t)tok[i] * p.Hkv + head[i]) * p.D + 8 * li;
      *reinterpret_cast<uint4*>(p.k_out + o) = k[i];
      *reinterpret_cast<uint4*>(p.v_out + o) = v[i];
    }
  }
}

}  // namespace k3
