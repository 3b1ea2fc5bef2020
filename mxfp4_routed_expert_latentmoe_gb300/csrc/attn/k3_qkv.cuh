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

// the cache as the kernels address it: strides of the rows in bytes, of the scales in elements
struct CacheView {
  uint8_t *k, *v;
  float *ks, *vs;
  int64_t page, head, tok;
  int64_t spage, shead, stok;
  int32_t n_pages, page_size;
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
  int32_t tokens;  // tokens of a block (norms), rows of a token in a block
  int32_t rows;
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
K3_DEVI void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
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
    const int32_t pg = slot / p.c.page_size;
    x.ok = pg < p.c.n_pages;
    x.page = x.ok ? pg : 0;
    x.at = x.ok ? slot - pg * p.c.page_size : 0;
  }
  if (!x.ok && slot != -1 && report) flag_status(p.status, K3ATTN_DEV_BAD_SLOT);
  return x;
}

// One row of the cache from its LPR lanes (lane li holds elements 8 li .. 8 li + 7, `on` where
// they lie below D): `raw` is the row in bf16 (a row that came as bf16 keeps its bits), y in
// fp32.  All lanes of a warp call it; `keep`: whether the row is written.
template <int FMT, int LPR>
K3_DEVI void store_row(const QkvParams& p, bool is_v, int h, const Place& pl, bool keep, uint4 raw,
                       const float (&y)[8], int li, bool on) {
  uint8_t* row = (is_v ? p.c.v : p.c.k) + pl.page * p.c.page + h * p.c.head + pl.at * p.c.tok;
  if constexpr (FMT == CF_BF16) {
    if (on && keep) *reinterpret_cast<uint4*>(row + 16 * li) = raw;
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
    if (on && keep) *reinterpret_cast<uint2*>(row + 8 * li) = e4m3x8(z);
    if (li == 0 && keep) (is_v ? p.c.vs : p.c.ks)[pl.page * p.c.spage + h * p.c.shead + pl.at * p.c.stok] = s;
  }
}

// Norms and rotation (FMT none), with the cache's rows in the same pass (FMT bf16, E4M3): a
// block has p.rows rows of p.tokens tokens, LPR lanes a row.  A thread's place in its rows is
// always the same, so it keeps the weights and, for a token's rows, the angles in registers;
// the angles (fp64 products and one sine and cosine per token and pair) are shared by the block.
template <int LPR, int FMT>
__global__ void __launch_bounds__(QKV_THREADS) k3_norm_kernel(const QkvParams p) {
  // (four more: the last pairs' load8 reaches past them)
  __shared__ __align__(16) float s_cos[QKV_TOKENS][132], s_sin[QKV_TOKENS][132];
  constexpr int SUBS = QKV_THREADS / LPR;
  const int li = threadIdx.x % LPR, sub = threadIdx.x / LPR, e = 8 * li;
  const int t0 = blockIdx.x * p.tokens, r0 = blockIdx.y * p.rows;
  const int nt = min(p.tokens, p.T - t0), nr = min(p.rows, p.Hq + p.Hkv * (FMT == CF_NONE ? 1 : 2) - r0);
  const bool on = e < p.D;
  grid_dep_wait();
  grid_dep_launch();
  uint4 raw[QKV_ROWS];
  int tok[QKV_ROWS], row[QKV_ROWS];
#pragma unroll
  for (int i = 0; i < QKV_ROWS; ++i) {
    const int it = sub + i * SUBS;
    tok[i] = it / nr;
    row[i] = r0 + it - tok[i] * nr;
    const int64_t t = t0 + tok[i];
    const int r = row[i];
    raw[i] = make_uint4(0, 0, 0, 0);
    if (tok[i] < nt && on) {
      const uint16_t* src = r < p.Hq ? p.q + t * p.q_stride + r * p.D
                            : r < p.Hq + p.Hkv ? p.k + t * p.k_stride + (r - p.Hq) * p.D
                                               : p.v + t * p.v_stride + (r - p.Hq - p.Hkv) * p.D;
      raw[i] = *reinterpret_cast<const uint4*>(src + e);
    }
  }
  float wq[8] = {}, wk[8] = {};
  if (on) {
    load8(p.q_w + e, wq);
    load8(p.k_w + e, wk);
  }
  const int half = p.R / 2;
  for (int i = threadIdx.x; i < nt * half; i += QKV_THREADS) {
    const int t = i / half, j = i - t * half;
    rotation(p.pos[t0 + t], p.inv_freq[j], s_cos[t][j], s_sin[t][j]);
  }
  __syncthreads();
  // the lanes of the other half of the rotated dims, this lane's angles
  const bool first = e < half, rotated = e < p.R;
  const int partner = (threadIdx.x & 31) + (rotated ? (first ? half / 8 : -(half / 8)) : 0);
  const int a0 = p.inter ? e / 2 : (first ? e : e - half);
  float c[8] = {}, s[8] = {};
  int have = -1;
#pragma unroll
  for (int i = 0; i < QKV_ROWS; ++i) {
    if (i * SUBS >= nt * nr) break;  // the whole block
    const bool there = tok[i] < nt;
    const int r = row[i];
    const int64_t t = t0 + tok[i];
    const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
    const int h = is_q ? r : (is_v ? r - p.Hq - p.Hkv : r - p.Hq);
    float x[8];
    unpack8(raw[i], x);
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const float rs = 1.0f / sqrtf(ss / (float)p.D + p.eps);
    if (!is_v)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] *= rs * (is_q ? wq[k] : wk[k]);
    if (half) {
      if (there && tok[i] != have && rotated) {
        have = tok[i];
        load8(&s_cos[have][a0], c);  // (interleaved pairs use the first four)
        load8(&s_sin[have][a0], s);
      }
      if (p.inter) {
        if (rotated && !is_v)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = x[2 * k], b = x[2 * k + 1];
            x[2 * k] = a * c[k] - b * s[k];
            x[2 * k + 1] = b * c[k] + a * s[k];
          }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float o = __shfl_sync(0xFFFFFFFFu, x[k], partner);
          if (rotated && !is_v) x[k] = first ? x[k] * c[k] - o * s[k] : x[k] * c[k] + o * s[k];
        }
      }
    }
    if (!is_v) raw[i] = pack8(x);
    if (there && on) {
      if (is_q) *reinterpret_cast<uint4*>(p.q_out + (t * p.Hq + h) * p.D + e) = raw[i];
      if (!is_q && !is_v && p.k_out) *reinterpret_cast<uint4*>(p.k_out + (t * p.Hkv + h) * p.D + e) = raw[i];
    }
    if constexpr (FMT != CF_NONE) {
      const bool cached = there && !is_q;
      if (__any_sync(0xFFFFFFFFu, cached)) {
        const Place pl = place_of(p, cached ? p.slots[t] : -1, li == 0);
        store_row<FMT, LPR>(p, is_v, h, pl, cached && pl.ok, raw[i], x, li, on);
      }
    }
  }
}

// Rows of the cache written from dense k, v (WRITE) or read back: row r of 2 Hkv a token, keys
// first; a block takes QKV_ROWS times its row groups in a line.
template <int LPR, int FMT, bool WRITE>
__global__ void __launch_bounds__(QKV_THREADS) k3_rows_kernel(const QkvParams p) {
  constexpr int SUBS = QKV_THREADS / LPR;
  const int li = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const bool on = 8 * li < p.D;
  const int nr = 2 * p.Hkv;
  const int64_t first = (int64_t)blockIdx.x * (SUBS * QKV_ROWS);
  const int32_t t0 = (int32_t)(first / nr), rest = (int32_t)(first - (int64_t)t0 * nr);
  grid_dep_wait();
  grid_dep_launch();
  int32_t slot[QKV_ROWS], tok[QKV_ROWS], row[QKV_ROWS];
#pragma unroll
  for (int i = 0; i < QKV_ROWS; ++i) {
    const int32_t it = rest + sub + i * SUBS, dt = it / nr;
    row[i] = it - dt * nr;
    tok[i] = dt < p.T - t0 ? t0 + dt : -1;
    slot[i] = tok[i] >= 0 ? p.slots[tok[i]] : -1;
  }
  uint4 raw[QKV_ROWS];
  float sc[QKV_ROWS];
  Place pl[QKV_ROWS];
#pragma unroll
  for (int i = 0; i < QKV_ROWS; ++i) {
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
  for (int i = 0; i < QKV_ROWS; ++i) {
    const bool is_v = row[i] >= p.Hkv;
    const int h = is_v ? row[i] - p.Hkv : row[i];
    float x[8];
    if constexpr (WRITE) {
      unpack8(raw[i], x);
      store_row<FMT, LPR>(p, is_v, h, pl[i], pl[i].ok, raw[i], x, li, on);
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
