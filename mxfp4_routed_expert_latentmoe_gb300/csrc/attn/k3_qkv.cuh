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
  int32_t tokens, rows;  // a block's tokens (norms), and rows of each
  Divisor by_rows;       // by `rows`; rows_kernel: by 2 Hkv
};

constexpr int QKV_THREADS = 256;
constexpr int QKV_ROWS = 4;    // rows of a thread
constexpr int QKV_TOKENS = 8;  // most tokens of a block of the norms
constexpr float E4M3_MAX = 448.0f;
constexpr float KV_MIN_SCALE = 0x1p-100f;  // its reciprocal and 448 times it are normal numbers

// cos and sin of pos * f: the product in turns in fp64, its whole turns taken off there (a far
// position's angle has no digits left in fp32), the rest in [-1/2, 1/2] turns rounded to fp32
K3_DEVI void rotation(int32_t pos, double f, float& c, float& s) {
  const double turns = (double)pos * (f * 0.15915494309189535);
  sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
}

K3_DEVI void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
K3_DEVI uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// eight values to E4M3 (round to nearest even, saturated)
K3_DEVI uint2 e4m3x8(const float (&x)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
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

// One row of the cache from its LPR lanes (lane li holds the four elements from ea and the four
// from eb, `on` where they lie below D): `raw` is the row in bf16 (a row that came as bf16
// keeps its bits), y in fp32.  All lanes of a warp call it; `keep`: whether the row is written.
template <int FMT, int LPR>
K3_DEVI void store_row(const QkvParams& p, bool is_v, int h, const Place& pl, bool keep, uint4 raw,
                       const float (&y)[8], int li, int ea, int eb, bool on) {
  uint8_t* row = (is_v ? p.c.v : p.c.k) + pl.page * p.c.page + h * p.c.head + pl.at * p.c.tok;
  if constexpr (FMT == CF_BF16) {
    if (on && keep) {
      *reinterpret_cast<uint2*>(row + 2 * ea) = make_uint2(raw.x, raw.y);
      *reinterpret_cast<uint2*>(row + 2 * eb) = make_uint2(raw.z, raw.w);
    }
  } else {
    // the largest magnitude by its bits, where infinities and NaN order above every number
    uint32_t m = 0;
    if (on)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float s = m < 0x7F800000u ? fmaxf(__uint_as_float(m) / E4M3_MAX, KV_MIN_SCALE) : __uint_as_float(0x7FC00000u);
    const float inv = 1.0f / s;
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = y[i] * inv;
    if (on && keep) {
      const uint2 codes = e4m3x8(z);
      *reinterpret_cast<uint32_t*>(row + ea) = codes.x;
      *reinterpret_cast<uint32_t*>(row + eb) = codes.y;
    }
    if (li == 0 && keep) (is_v ? p.c.vs : p.c.ks)[pl.page * p.c.spage + h * p.c.shead + pl.at * p.c.stok] = s;
  }
}

// Norms and rotation (FMT none), with the cache's rows in the same pass (FMT bf16, E4M3): a
// block has p.rows rows of each of p.tokens tokens, LPR lanes a row and up to ROWS rows a
// thread.  A lane holds two pieces of four elements of a row: the two halves of four rotated
// pairs (pairs (i, i + R/2)), or eight neighbours, so that pairs never cross lanes.  Its pieces
// are the same in all its rows: weights and angles stay in registers, reloaded where the kind
// of row or the token changes.  The angles (fp64 products and one sine and cosine per token and
// pair) are shared by the block.
template <int LPR, int FMT, int ROWS>
__global__ void __launch_bounds__(QKV_THREADS, 4) k3_norm_kernel(const QkvParams p) {
  __shared__ __align__(16) float s_cos[QKV_TOKENS][128], s_sin[QKV_TOKENS][128];
  constexpr int SUBS = QKV_THREADS / LPR;
  const int li = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int t0 = blockIdx.x * p.tokens, r0 = blockIdx.y * p.rows;
  const int nt = min(p.tokens, p.T - t0), nr = min(p.rows, p.Hq + p.Hkv * (FMT == CF_NONE ? 1 : 2) - r0);
  const bool on = 8 * li < p.D, rotated = 8 * li < p.R;
  const int half = p.R / 2;
  // this lane's pieces and their first angle
  int ea = 8 * li, eb = ea + 4, angle = ea / 2;
  if (!p.inter && rotated) {
    ea = angle = 4 * li;
    eb = ea + half;
  }
  grid_dep_wait();
  grid_dep_launch();
  uint2 ra[ROWS], rb[ROWS];
  int tok[ROWS], row[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int it = sub + i * SUBS;
    tok[i] = p.tokens == 1 ? (it < nr ? 0 : 1) : (int)p.by_rows(it);
    row[i] = r0 + it - tok[i] * p.rows;
    ra[i] = rb[i] = make_uint2(0, 0);
    if (tok[i] < nt && on) {
      const int64_t t = t0 + tok[i];
      const int r = row[i];
      const uint16_t* src = r < p.Hq ? p.q + t * p.q_stride + r * p.D
                            : r < p.Hq + p.Hkv ? p.k + t * p.k_stride + (r - p.Hq) * p.D
                                               : p.v + t * p.v_stride + (r - p.Hq - p.Hkv) * p.D;
      ra[i] = *reinterpret_cast<const uint2*>(src + ea);
      rb[i] = *reinterpret_cast<const uint2*>(src + eb);
    }
  }
  for (int i = threadIdx.x; i < nt * half; i += QKV_THREADS) {
    const int t = i / half, j = i - t * half;
    rotation(p.pos[t0 + t], p.inv_freq[j], s_cos[t][j], s_sin[t][j]);
  }
  __syncthreads();
  const float over_d = 1.0f / (float)p.D;
  float4 wa = {}, wb = {}, c = {}, s = {};
  int have_tok = -1, have_w = -1;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (i * SUBS >= nt * nr) break;  // the whole block
    const bool there = tok[i] < nt;
    const int r = row[i];
    const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
    const int h = is_q ? r : (is_v ? r - p.Hq - p.Hkv : r - p.Hq);
    float x[8];
    unpack8(make_uint4(ra[i].x, ra[i].y, rb[i].x, rb[i].y), x);
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    uint4 raw = make_uint4(ra[i].x, ra[i].y, rb[i].x, rb[i].y);
    if (!is_v) {
      const float rs = rsqrtf(ss * over_d + p.eps);
      if (on && have_w != (int)is_q) {
        have_w = is_q;
        const float* w = is_q ? p.q_w : p.k_w;
        wa = __ldg(reinterpret_cast<const float4*>(w + ea));
        wb = __ldg(reinterpret_cast<const float4*>(w + eb));
      }
      x[0] *= rs * wa.x; x[1] *= rs * wa.y; x[2] *= rs * wa.z; x[3] *= rs * wa.w;
      x[4] *= rs * wb.x; x[5] *= rs * wb.y; x[6] *= rs * wb.z; x[7] *= rs * wb.w;
      if (rotated) {
        if (there && tok[i] != have_tok) {
          have_tok = tok[i];
          c = *reinterpret_cast<const float4*>(&s_cos[have_tok][angle]);
          s = *reinterpret_cast<const float4*>(&s_sin[have_tok][angle]);
        }
        const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
        if (p.inter) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = x[2 * k], b = x[2 * k + 1];
            x[2 * k] = a * cc[k] - b * sn[k];
            x[2 * k + 1] = b * cc[k] + a * sn[k];
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = x[k], b = x[4 + k];
            x[k] = a * cc[k] - b * sn[k];
            x[4 + k] = b * cc[k] + a * sn[k];
          }
        }
      }
      raw = pack8(x);
    }
    const int64_t t = t0 + tok[i];
    if (there && on && !is_v) {
      uint16_t* dst = is_q ? p.q_out + (t * p.Hq + h) * p.D : (p.k_out ? p.k_out + (t * p.Hkv + h) * p.D : nullptr);
      if (dst) {
        *reinterpret_cast<uint2*>(dst + ea) = make_uint2(raw.x, raw.y);
        *reinterpret_cast<uint2*>(dst + eb) = make_uint2(raw.z, raw.w);
      }
    }
    if constexpr (FMT != CF_NONE) {
      const bool cached = there && !is_q;
      if (__any_sync(0xFFFFFFFFu, cached)) {
        const Place pl = place_of(p, cached ? p.slots[t] : -1, li == 0);
        store_row<FMT, LPR>(p, is_v, h, pl, cached && pl.ok, raw, x, li, ea, eb, on);
      }
    }
  }
}

// Rows of the cache written from dense k, v (WRITE) or read back: row r of 2 Hkv a token, keys
// first; a block takes ROWS times its row groups in a line.
template <int LPR, int FMT, bool WRITE, int ROWS>
__global__ void __launch_bounds__(QKV_THREADS) k3_rows_kernel(const QkvParams p) {
  constexpr int SUBS = QKV_THREADS / LPR;
  const int li = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const bool on = 8 * li < p.D;
  const int nr = 2 * p.Hkv;
  const int64_t first = (int64_t)blockIdx.x * (SUBS * ROWS);
  const int32_t t0 = (int32_t)(first / nr), rest = (int32_t)(first - (int64_t)t0 * nr);
  grid_dep_wait();
  grid_dep_launch();
  int32_t slot[ROWS], tok[ROWS], row[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int32_t it = rest + sub + i * SUBS, dt = (int32_t)p.by_rows(it);
    row[i] = it - dt * nr;
    tok[i] = dt < p.T - t0 ? t0 + dt : -1;
    slot[i] = tok[i] >= 0 ? p.slots[tok[i]] : -1;
  }
  uint4 raw[ROWS];
  float sc[ROWS];
  Place pl[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    pl[i] = place_of(p, slot[i], li == 0);
    const bool is_v = row[i] >= p.Hkv;
    const int h = is_v ? row[i] - p.Hkv : row[i];
    raw[i] = make_uint4(0, 0, 0, 0);
    sc[i] = 0.f;
    if (WRITE) {
      if (on && pl[i].ok)
        raw[i] = *reinterpret_cast<const uint4*>((is_v ? p.v + tok[i] * p.v_stride : p.k + tok[i] * p.k_stride) +
                                                 h * p.D + 8 * li);
    } else if (on && pl[i].ok) {
      const uint8_t* src = (is_v ? p.c.v : p.c.k) + pl[i].page * p.c.page + h * p.c.head + pl[i].at * p.c.tok;
      if constexpr (FMT == CF_BF16) {
        raw[i] = *reinterpret_cast<const uint4*>(src + 16 * li);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(src + 8 * li);
        raw[i].x = w.x;
        raw[i].y = w.y;
        sc[i] = (is_v ? p.c.vs : p.c.ks)[pl[i].page * p.c.spage + h * p.c.shead + pl[i].at * p.c.stok];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const bool is_v = row[i] >= p.Hkv;
    const int h = is_v ? row[i] - p.Hkv : row[i];
    float x[8];
    if constexpr (WRITE) {
      unpack8(raw[i], x);
      store_row<FMT, LPR>(p, is_v, h, pl[i], pl[i].ok, raw[i], x, li, 8 * li, 8 * li + 4, on);
    } else {
      if constexpr (FMT == CF_E4M3) {
        const uint32_t w[2] = {raw[i].x, raw[i].y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2_raw hr =
              __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k / 2] >> (16 * (k & 1))), __NV_E4M3);
          const float2 f = __half22float2(__half2(hr));
          x[2 * k] = f.x * sc[i];
          x[2 * k + 1] = f.y * sc[i];
        }
        raw[i] = pack8(x);
      }
      if (on && tok[i] >= 0)
        *reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + ((int64_t)tok[i] * p.Hkv + h) * p.D + 8 * li) = raw[i];
    }
  }
}

}  // namespace k3
