// k3_qkv.cuh -- norms of queries and keys per head with the position rotation, and the rows of
// the paged cache: written (bf16, or E4M3 codes with a row scale) and read back.
//
// All of it is bound by HBM: a row (a head of a token) is taken by 8, 16 or 32 lanes, eight
// elements a lane (16-byte accesses), and a thread has the loads of up to QKV_ROWS rows in
// flight before it waits for any.
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
  int32_t tokens, rows, warps;  // norms: a block's tokens, rows of each and warps for each
  Divisor by_heads;             // rows: by Hkv
};

constexpr int QKV_THREADS = 512;  // most threads of a block
constexpr int QKV_ROWS = 4;       // rows of a thread in flight
constexpr int QKV_TOKENS = 8;     // most tokens of a block of the norms
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
// a lane's eight codes of a row, given the inverse of its scale
K3_DEVI uint2 codes_of(const float2 (&y)[4], float inv) {
  float2 z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = mul2(y[i], make_float2(inv, inv));
  return e4m3x8(z);
}

// Norms and rotation (FMT none), with the cache's rows in the same pass (FMT bf16, E4M3): a
// block has p.rows rows of each of p.tokens tokens, p.warps warps a token, LPR lanes a row and
// up to ROWS rows a thread.  A lane holds two pieces of four elements of a row: the two halves
// of four rotated pairs (pairs (i, i + R/2)), or eight neighbours, so that pairs never cross
// lanes.  Its pieces are the same in all its rows: the products of weights and angles stay in
// registers, formed anew where queries give way to keys, and a row takes 12 packed operations
// for its norm and rotation.  The angles (fp64 products and one sine and cosine per token and
// pair) are shared by the block.
template <int LPR, int FMT, int ROWS>
__global__ void __launch_bounds__(QKV_THREADS, 2) k3_norm_kernel(const QkvParams p) {
  __shared__ __align__(16) float s_cos[QKV_TOKENS][128], s_sin[QKV_TOKENS][128];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, group = warp / p.warps;
  const int li = lane % LPR, sub = (warp - group * p.warps) * (32 / LPR) + lane / LPR, subs = p.warps * (32 / LPR);
  const int t0 = blockIdx.x * p.tokens, r0 = blockIdx.y * p.rows;
  const int nt = min(p.tokens, p.T - t0);
  const bool mine = group < nt;  // this warp's token: there is one
  const int64_t t = t0 + (mine ? group : 0);
  const int r1 = mine ? min(r0 + p.rows, p.Hq + p.Hkv * (FMT == CF_NONE ? 1 : 2)) : 0;
  const bool on = 8 * li < p.D, rotated = 8 * li < p.R;
  const int half = p.R / 2, k0 = p.Hq, v0 = p.Hq + p.Hkv;
  // this lane's pieces and their first angle
  int ea = 8 * li, eb = ea + 4, angle = ea / 2;
  if (!p.inter && rotated) {
    ea = angle = 4 * li;
    eb = ea + half;
  }
  // where row 0 would be, were all rows of its kind
  const uint16_t* const qs = p.q + t * p.q_stride;
  const uint16_t* const ks = p.k + t * p.k_stride - k0 * p.D;
  const uint16_t* const vs = p.v + t * p.v_stride - v0 * p.D;
  grid_dep_wait();
  grid_dep_launch();
  uint2 ra[ROWS], rb[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + sub + i * subs;
    ra[i] = rb[i] = make_uint2(0, 0);
    if (r < r1 && on) {
      const uint16_t* src = (r < k0 ? qs : (FMT == CF_NONE || r < v0 ? ks : vs)) + r * p.D;
      ra[i] = *reinterpret_cast<const uint2*>(src + ea);
      rb[i] = *reinterpret_cast<const uint2*>(src + eb);
    }
  }
  for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
    const int g = i / half, j = i - g * half;
    rotation(p.pos[t0 + g], p.inv_freq[j], s_cos[g][j], s_sin[g][j]);
  }
  Place pl{0, 0, false};
  if constexpr (FMT != CF_NONE) {
    if (r1 > v0 - p.Hkv) pl = place_of(p, p.slots[t], lane == 0);
  }
  __syncthreads();
  const float over_d = 1.0f / (float)p.D;
  uint16_t* const qd = p.q_out + t * p.Hq * p.D;
  uint16_t* const kd = p.k_out + (t * p.Hkv - k0) * p.D;
  // y = x * co + z * si, z the other element of x's pair; without rotation co is the weight alone
  float2 co[4] = {}, si[4] = {};
  int have = -1;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + sub + i * subs;
    const bool there = r < r1;
    if (!__any_sync(0xFFFFFFFFu, there)) break;
    const bool is_q = r < k0, is_v = FMT != CF_NONE && r >= v0;
    uint4 raw = make_uint4(ra[i].x, ra[i].y, rb[i].x, rb[i].y);
    float2 x[4];
    unpack8(raw, x);
    float2 s2 = mul2(x[0], x[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) s2 = fma2(x[k], x[k], s2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (!is_v) {
      if (on && there && have != (int)is_q) {
        have = is_q;
        const float* w = is_q ? p.q_w : p.k_w;
        const float4 wa = __ldg(reinterpret_cast<const float4*>(w + ea));
        const float4 wb = __ldg(reinterpret_cast<const float4*>(w + eb));
        co[0] = make_float2(wa.x, wa.y);
        co[1] = make_float2(wa.z, wa.w);
        co[2] = make_float2(wb.x, wb.y);
        co[3] = make_float2(wb.z, wb.w);
        if (rotated) {
          const float4 c = *reinterpret_cast<const float4*>(&s_cos[group][angle]);
          const float4 s = *reinterpret_cast<const float4*>(&s_sin[group][angle]);
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
      }
      const float rs = rsqrtf(ss * over_d + p.eps);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = mul2(x[k], make_float2(rs, rs));
      float2 z[4] = {x[2], x[3], x[0], x[1]};
      if (p.inter)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = make_float2(x[k].y, x[k].x);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] = mul2(x[k], co[k]);
        if (rotated) x[k] = fma2(z[k], si[k], x[k]);
      }
      raw = pack8(x);
    }
    if (there && on && !is_v && (is_q || p.k_out)) {
      uint16_t* dst = (is_q ? qd : kd) + r * p.D;
      *reinterpret_cast<uint2*>(dst + ea) = make_uint2(raw.x, raw.y);
      *reinterpret_cast<uint2*>(dst + eb) = make_uint2(raw.z, raw.w);
    }
    if constexpr (FMT != CF_NONE) {
      if (__any_sync(0xFFFFFFFFu, there && !is_q)) {
        const int h = r - (is_v ? v0 : k0);
        const bool keep = there && !is_q && pl.ok;
        uint8_t* to = (is_v ? p.c.v : p.c.k) + row_at(p, pl, h);
        if constexpr (FMT == CF_BF16) {
          if (keep && on) {
            *reinterpret_cast<uint2*>(to + 2 * ea) = make_uint2(raw.x, raw.y);
            *reinterpret_cast<uint2*>(to + 2 * eb) = make_uint2(raw.z, raw.w);
          }
        } else {
          const float s = scale_of(row_max<LPR>(x));
          const uint2 codes = codes_of(x, 1.0f / s);
          if (keep && on) {
            *reinterpret_cast<uint32_t*>(to + ea) = codes.x;
            *reinterpret_cast<uint32_t*>(to + eb) = codes.y;
          }
          if (keep && li == 0) (is_v ? p.c.vs : p.c.ks)[scale_at(p, pl, h)] = s;
        }
      }
    }
  }
}

// Rows of the cache written from dense k, v (WRITE) or read back: an item is a head of a token,
// its key and its value, LPR lanes an item and ITEMS items a thread.
template <int LPR, int FMT, bool WRITE, int ITEMS>
__global__ void __launch_bounds__(256) k3_rows_kernel(const QkvParams p) {
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
        // even lanes form the key's scale and inverse, odd ones the value's, and trade them
        const uint32_t mk = row_max<LPR>(k[i]), mv = row_max<LPR>(v[i]);
        const bool odd = li & 1;
        const float s = scale_of(odd ? mv : mk), inv = 1.0f / s;
        const float inv1 = __shfl_xor_sync(0xFFFFFFFFu, inv, 1);
        float2 x[4];
        unpack8(k[i], x);
        const uint2 kc = codes_of(x, odd ? inv1 : inv);
        unpack8(v[i], x);
        const uint2 vc = codes_of(x, odd ? inv : inv1);
        if (on && pl[i].ok) {
          *reinterpret_cast<uint2*>(p.c.k + o + 8 * li) = kc;
          *reinterpret_cast<uint2*>(p.c.v + o + 8 * li) = vc;
          if (li < 2) (odd ? p.c.vs : p.c.ks)[scale_at(p, pl[i], head[i])] = s;
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
