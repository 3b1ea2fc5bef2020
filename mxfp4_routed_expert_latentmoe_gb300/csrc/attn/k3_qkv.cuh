// k3_qkv.cuh -- norms of queries and keys per head with the position rotation, and the rows of
// the paged cache: written (bf16, or E4M3 codes with a row scale) and read back.
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
};

constexpr int QKV_WARPS = 8;
constexpr float E4M3_MAX = 448.0f;
constexpr float KV_MIN_SCALE = 0x1p-100f;  // its reciprocal and 448 times it are normal numbers

// cos and sin of pos * f: the product in turns in fp64, its whole turns taken off there (a far
// position's angle has no digits left in fp32), the rest in [-1/2, 1/2] turns rounded to fp32
K3_DEVI float2 rotation(int32_t pos, double f) {
  const double turns = (double)pos * (f * 0.15915494309189535);
  float s, c;
  sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
  return make_float2(c, s);
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

// One row of the cache from a warp's lanes (lane l < D / 8 holds elements 8l .. 8l + 7): `raw`
// is the row in bf16 (a row that came as bf16 keeps its bits), y in fp32.
template <int FMT>
K3_DEVI void store_row(uint8_t* row, float* scale, uint4 raw, const float (&y)[8], int lane, bool on) {
  if constexpr (FMT == CF_BF16) {
    if (on) *reinterpret_cast<uint4*>(row + 16 * lane) = raw;
  } else {
    // the largest magnitude by its bits, where infinities and NaN order above every number
    uint32_t m = 0;
    if (on)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    const float s = m < 0x7F800000u ? fmaxf(__uint_as_float(m) / E4M3_MAX, KV_MIN_SCALE) : __uint_as_float(0x7FC00000u);
    const float inv = 1.0f / s;
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = y[i] * inv;
    if (on) *reinterpret_cast<uint2*>(row + 8 * lane) = e4m3x8(z);
    if (lane == 0) *scale = s;
  }
}

// One warp per row (a head of a token); a block has one token's rows.
template <bool NORM, int FMT>
__global__ void __launch_bounds__(QKV_WARPS * 32) k3_qkv_kernel(const QkvParams p) {
  __shared__ float2 rot[128];
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  if (NORM) {
    for (int i = threadIdx.x; i < p.R / 2; i += blockDim.x) rot[i] = rotation(p.pos[t], p.inv_freq[i]);
    __syncthreads();
  }
  int64_t page = 0, in_page = 0;
  bool keep = false;
  if constexpr (FMT != CF_NONE) {
    const int32_t slot = p.slots[t];
    keep = slot >= 0 && slot / p.c.page_size < p.c.n_pages;
    if (keep) {
      page = slot / p.c.page_size;
      in_page = slot % p.c.page_size;
    } else if (slot != -1 && threadIdx.x == 0) {
      flag_status(p.status, K3ATTN_DEV_BAD_SLOT);
    }
  }
  const int nq = NORM ? p.Hq : 0, rows = nq + p.Hkv + (FMT != CF_NONE ? p.Hkv : 0);
  const bool on = lane < p.D / 8;
  for (int r = warp; r < rows; r += QKV_WARPS) {
    const bool is_q = r < nq, is_v = r >= nq + p.Hkv;
    const int h = is_q ? r : (is_v ? r - nq - p.Hkv : r - nq);
    const uint16_t* src = (is_q ? p.q + t * p.q_stride : (is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride)) +
                          (int64_t)h * p.D + 8 * lane;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (on) raw = *reinterpret_cast<const uint4*>(src);
    float x[8];
    unpack8(raw, x);
    if (NORM && !is_v) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const float rs = 1.0f / sqrtf(ss / (float)p.D + p.eps);
      const float* w = is_q ? p.q_w : p.k_w;
      if (on)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= rs * w[8 * lane + i];
      const int e = 8 * lane;
      if (p.inter) {
        if (e < p.R)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 cs = rot[e / 2 + i];
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * cs.x - b * cs.y;
            x[2 * i + 1] = b * cs.x + a * cs.y;
          }
      } else {
        const int half = p.R / 2, hl = half / 8;  // lanes of half the rotated dims
        const bool first = e < half, rotated = e < p.R;
        const int partner = rotated ? (first ? lane + hl : lane - hl) : lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(0xFFFFFFFFu, x[i], partner);
          if (rotated) {
            const float2 cs = rot[(first ? e : e - half) + i];
            x[i] = first ? x[i] * cs.x - o * cs.y : x[i] * cs.x + o * cs.y;
          }
        }
      }
      uint16_t* dst = is_q ? p.q_out + ((int64_t)t * p.Hq + h) * p.D
                           : (p.k_out ? p.k_out + ((int64_t)t * p.Hkv + h) * p.D : nullptr);
      raw = pack8(x);
      if (on && dst) *reinterpret_cast<uint4*>(dst + 8 * lane) = raw;
    }
    if constexpr (FMT != CF_NONE) {
      if (!is_q && keep) {
        uint8_t* row = (is_v ? p.c.v : p.c.k) + page * p.c.page + h * p.c.head + in_page * p.c.tok;
        float* sc = FMT == CF_E4M3
                        ? (is_v ? p.c.vs : p.c.ks) + page * p.c.spage + h * p.c.shead + in_page * p.c.stok
                        : nullptr;
        store_row<FMT>(row, sc, raw, x, lane, on);
      }
    }
  }
}

// The rows of T slots back as dense bf16; a block has one token's rows, one warp per row.
template <int FMT>
__global__ void __launch_bounds__(QKV_WARPS * 32) k3_kv_read_kernel(const QkvParams p) {
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  const int32_t slot = p.slots[t];
  const bool there = slot >= 0 && slot / p.c.page_size < p.c.n_pages;
  if (!there && slot != -1 && threadIdx.x == 0) flag_status(p.status, K3ATTN_DEV_BAD_SLOT);
  const int64_t page = there ? slot / p.c.page_size : 0, in_page = there ? slot % p.c.page_size : 0;
  if (lane >= p.D / 8) return;
  for (int r = warp; r < 2 * p.Hkv; r += QKV_WARPS) {
    const bool is_v = r >= p.Hkv;
    const int h = is_v ? r - p.Hkv : r;
    const uint8_t* row = (is_v ? p.c.v : p.c.k) + page * p.c.page + h * p.c.head + in_page * p.c.tok;
    uint4 o = make_uint4(0, 0, 0, 0);
    if (there) {
      if constexpr (FMT == CF_BF16) {
        o = *reinterpret_cast<const uint4*>(row + 16 * lane);
      } else {
        const float s = *((is_v ? p.c.vs : p.c.ks) + page * p.c.spage + h * p.c.shead + in_page * p.c.stok);
        const uint2 c = *reinterpret_cast<const uint2*>(row + 8 * lane);
        const uint32_t w[2] = {c.x, c.y};
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2_raw hr =
              __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
          const float2 f = __half22float2(__half2(hr));
          x[2 * i] = f.x * s;
          x[2 * i + 1] = f.y * s;
        }
        o = pack8(x);
      }
    }
    *reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + ((int64_t)t * p.Hkv + h) * p.D + 8 * lane) = o;
  }
}

}  // namespace k3
