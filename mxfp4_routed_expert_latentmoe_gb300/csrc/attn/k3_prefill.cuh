// k3_prefill.cuh -- attention of many new tokens per sequence over the paged key-value cache.
//
// A warp takes one (token, query head): 32 keys at a time, a lane computes a key's logit, then the
// lanes hold dims of the value sum.
#pragma once

#include "k3_decode.cuh"

namespace k3 {

struct PrefillParams {
  const uint16_t* q;
  int64_t q_stride;
  int32_t B, T, Hq, Hkv, G, D, window, sinks;
  float scale;  // softmax_scale * log2(e): logits in powers of two
  CacheView c;
  const int32_t *starts, *table, *lens;
  int32_t table_width;
  uint16_t* out;
  float* lse;
  uint32_t* status;
};

// eight values of a cached row
template <int FMT>
K3_DEVI void row8(const uint8_t* row, int chunk, float scale, const uint8_t* exps, float (&x)[8]) {
  uint4 v;
  if constexpr (FMT == CF_BF16) {
    v = ldg128(row + 16 * chunk);
  } else if constexpr (FMT == CF_E4M3) {
    const uint2 c = ldg64(row + 8 * chunk);
    uint32_t h[4];
    e4m3x4_f16x4(c.x, h[0], h[1]);
    e4m3x4_f16x4(c.y, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      x[2 * i] = f.x * scale;
      x[2 * i + 1] = f.y * scale;
    }
    return;
  } else {
    v = e2m1x8_bf16(__ldg(reinterpret_cast<const uint32_t*>(row + 4 * chunk)), exps[chunk / 4]);
  }
  float2 y[4];
  unpack8(v, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = y[i].x;
    x[2 * i + 1] = y[i].y;
  }
}

template <int FMT>
__global__ void __launch_bounds__(256) k3_prefill_simple_kernel(const PrefillParams p) {
  __shared__ float s_q[8][256];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t item = (int64_t)blockIdx.x * 8 + warp;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += 256) {
      const int64_t most = (int64_t)p.table_width * p.c.page_size;
      const int32_t s0 = p.starts[b], s1 = p.starts[b + 1], n = p.lens[b];
      if (s0 < 0 || s1 < s0 || s1 > p.T || n < 0 || n > most || n < s1 - s0) flag_status(p.status, K3ATTN_DEV_BAD_LENGTH);
    }
  if (item >= (int64_t)p.T * p.Hq) return;
  const int t = (int)(item / p.Hq), h = (int)(item % p.Hq), kvh = h / p.G;
  int lo = 0, hi = p.B;  // the last sequence that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    (p.starts[mid] <= t ? lo : hi) = mid;
  }
  const int32_t s0 = max(p.starts[lo], 0), s1 = min(p.starts[lo + 1], p.T);
  if (t < s0 || t >= s1) return;  // no sequence's
  const int64_t most = min((int64_t)p.table_width * p.c.page_size, (int64_t)INT32_MAX);
  const int32_t n = (int32_t)min(most, (int64_t)max(p.lens[lo], 0)), pos = n - s1 + t;
  for (int d = lane; d < p.D; d += 32) s_q[warp][d] = bf16_bits_to_f32(p.q[t * p.q_stride + (int64_t)h * p.D + d]);
  __syncwarp();
  const int32_t f = p.window > 0 && pos >= p.window ? pos + 1 - p.window : 0, ns = min(p.sinks, f);
  const int32_t count = pos < 0 ? 0 : ns + (pos + 1 - f);
  float m = -INFINITY, l = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int32_t i0 = 0; i0 < count; i0 += 32) {
    const int32_t i = i0 + lane;
    int64_t row = -1, so = 0;
    float s = -INFINITY;
    if (i < count) {
      const int32_t tok = i < ns ? i : f + (i - ns), pg = (int32_t)p.c.by_page(tok), at = tok - pg * p.c.page_size;
      const int32_t entry = p.table[(int64_t)lo * p.table_width + pg];
      if (entry >= 0 && entry < p.c.n_pages) {
        row = entry * p.c.page + kvh * p.c.head + at * p.c.tok;
        so = entry * p.c.spage + kvh * p.c.shead + at * p.c.stok;
        s = 0.f;
        const float ks = FMT == CF_E4M3 ? p.c.ks[so] : 1.f;
        for (int c = 0; c < p.D / 8; ++c) {
          float x[8];
          row8<FMT>(p.c.k + row, c, 1.f, p.c.k_exps() + so, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(x[e], s_q[warp][8 * c + e], s);
        }
        s *= ks * p.scale;
      } else {
        flag_status(p.status, K3ATTN_DEV_BAD_PAGE);
      }
    }
    float top = s;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float m1 = fmaxf(m, top), base = m1 == -INFINITY ? 0.f : m1, fall = exp2f(m - base), w = exp2f(s - base);
    m = m1;
    l = l * fall + w;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= fall;
    for (int j = 0; j < 32; ++j) {
      const int64_t r = __shfl_sync(0xFFFFFFFFu, row, j), o = __shfl_sync(0xFFFFFFFFu, so, j);
      const float wj = __shfl_sync(0xFFFFFFFFu, w, j);
      if (r < 0 || 8 * lane >= p.D) continue;
      float x[8];
      row8<FMT>(p.c.v + r, lane, FMT == CF_E4M3 ? p.c.vs[o] : 1.f, p.c.v_exps() + o, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(wj, x[e], acc[e]);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  const float r = l == 0.f ? 0.f : 1.f / l;
  const int64_t row = (int64_t)t * p.Hq + h;
  if (8 * lane < p.D) {
    const uint2 a = bf16x4(acc[0] * r, acc[1] * r, acc[2] * r, acc[3] * r), b = bf16x4(acc[4] * r, acc[5] * r, acc[6] * r, acc[7] * r);
    *reinterpret_cast<uint4*>(p.out + row * p.D + 8 * lane) = make_uint4(a.x, a.y, b.x, b.y);
  }
  if (lane == 0 && p.lse) p.lse[row] = lse_of(m == -INFINITY ? 0.f : m, l);
}

}  // namespace k3
