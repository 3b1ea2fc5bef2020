// k3_decode.cuh -- attention of one new token over a paged key-value cache.
#pragma once

#include "k3_qkv.cuh"

namespace k3 {

struct DecodeParams {
  const uint16_t* q;
  int64_t q_stride;
  int32_t B, Hq, Hkv, D, window;
  float scale;
  CacheView c;
  const int32_t *table, *lens;
  int32_t table_width;
  uint16_t* out;
  float* lse;
  uint32_t* status;
};

constexpr int DEC_WARPS = 8;

// length of sequence b within what its table can hold
K3_DEVI int32_t seq_len(const DecodeParams& p, int b, bool& bad) {
  const int32_t n = p.lens[b];
  const int64_t most = (int64_t)p.table_width * p.c.page_size;
  bad = n < 0 || n > most;
  return n < 0 ? 0 : (n > most ? (int32_t)most : n);
}

// One block per (query head, sequence); its warps take every DEC_WARPS-th token, lane l < D / 8
// elements 8l .. 8l + 7, each warp with a running maximum and sum, joined at the end.
template <int FMT>
__global__ void __launch_bounds__(DEC_WARPS * 32) k3_decode_kernel(const DecodeParams p) {
  __shared__ float sm[DEC_WARPS], sl[DEC_WARPS], so[DEC_WARPS][256];
  const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  bool bad;
  const int32_t n = seq_len(p, b, bad);
  if (bad && threadIdx.x == 0) flag_status(p.status, K3ATTN_DEV_BAD_LENGTH);
  const int32_t f = p.window > 0 && n > p.window ? n - p.window : 0;
  const int64_t j = h / (p.Hq / p.Hkv);
  const bool on = lane < p.D / 8;
  const float c = p.scale * 1.4426950408889634f;  // logits in powers of two
  float q[8] = {}, o[8] = {}, m = -INFINITY, l = 0.f;
  if (on) unpack8(*reinterpret_cast<const uint4*>(p.q + b * p.q_stride + (int64_t)h * p.D + 8 * lane), q);
  auto row = [&](const uint8_t* base, const float* scales, int64_t page, int64_t at, float (&x)[8]) {
    if (!on) return;
    const uint8_t* r = base + page * p.c.page + j * p.c.head + at * p.c.tok;
    if constexpr (FMT == CF_BF16) {
      unpack8(*reinterpret_cast<const uint4*>(r + 16 * lane), x);
    } else {
      const float s = scales[page * p.c.spage + j * p.c.shead + at * p.c.stok];
      const uint2 w = *reinterpret_cast<const uint2*>(r + 8 * lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2_raw hr =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1))), __NV_E4M3);
        const float2 v = __half22float2(__half2(hr));
        x[2 * i] = v.x * s;
        x[2 * i + 1] = v.y * s;
      }
    }
  };
  for (int32_t t = f + warp; t < n; t += DEC_WARPS) {
    const int32_t page = p.table[(int64_t)b * p.table_width + t / p.c.page_size];
    if (page < 0 || page >= p.c.n_pages) {
      if (lane == 0) flag_status(p.status, K3ATTN_DEV_BAD_PAGE);
      continue;
    }
    float x[8] = {};
    row(p.c.k, p.c.ks, page, t % p.c.page_size, x);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
    s *= c;
    const float m1 = fmaxf(m, s), base = m1 == -INFINITY ? 0.f : m1;
    const float a = exp2f(m - base), e = exp2f(s - base);
    m = m1;
    l = l * a + e;
    row(p.c.v, p.c.vs, page, t % p.c.page_size, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * a + e * x[i];
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  if (on)
#pragma unroll
    for (int i = 0; i < 8; ++i) so[warp][8 * lane + i] = o[i];
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < DEC_WARPS; ++w) top = fmaxf(top, sm[w]);
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int w = 0; w < DEC_WARPS; ++w) sum += sl[w] * exp2f(sm[w] - base);
  for (int i = threadIdx.x; i < p.D; i += blockDim.x) {
    float v = 0.f;
    for (int w = 0; w < DEC_WARPS; ++w) v += so[w][i] * exp2f(sm[w] - base);
    p.out[((int64_t)b * p.Hq + h) * p.D + i] = f32_to_bf16_bits(sum == 0.f ? 0.f : v / sum);
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[(int64_t)b * p.Hq + h] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace k3
