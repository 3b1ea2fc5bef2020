// k3_decode.cuh -- attention of one new token over a paged key-value cache.
//
// One pass over the cached rows with a running maximum and sum.  The query heads of one key
// head (8 or 16 of them at a time) are the N side of the matrix instructions and the tokens
// the M side, so that a key head with few query heads wastes no rows:
//   S^T [16 tokens x 8 heads]  = K  [16 tokens x D]  Q^T
//   O^T [16 dims x 8 heads]   += V^T [16 dims x 16 tokens]  P^T
// (mma.sync: the products are 2 G flops a cached byte, far below what they reach; the cache's
// bytes bound the kernel.)  Each warp streams its own tiles of 16 or 32 tokens through a ring
// in shared memory with cp.async, row by row through the page table (any page size, any
// strides), and joins its block's other warps only at the end of a sequence's part.
//
// E4M3 rows become fp16 operands exactly; a key's scale multiplies its logit, a value's scale
// goes into its weight's exponent, with a maximum of its own, so that weights of values of any
// size keep fp16's full precision.  bf16 rows are multiplied as they are.
//
// The work is cut into units (a block's tokens of one (sequence, key head, head group)), which
// are dealt out evenly: block c takes units c * chunk .. (c + 1) * chunk - 1 of all of them,
// whatever the lengths.  A part that is not a whole sequence leaves an unnormalised record in
// the workspace; the block that arrives last joins a sequence's records, in block order.
#pragma once

#include "k3_qkv.cuh"

namespace k3 {

struct DecodeParams {
  const uint16_t* q;
  int64_t q_stride;
  int32_t B, Hq, Hkv, G, D, window;
  int32_t groups;  // head groups of a key head: ceil(G / (8 NT))
  float scale;     // softmax_scale * log2(e): logits in powers of two
  CacheView c;
  const int32_t *table, *lens;
  int32_t table_width;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  uint32_t* arrived;  // one counter a block, zero between calls
  float* parts;       // two records a block
};

// most blocks of a launch (the workspace holds their counters and records)
constexpr int DEC_MAX_BLOCKS = 192;

// Shapes of one instance: the warps of a block, the tokens of a warp's tile, the ring's depth,
// and the dims that one pass of the block's join takes (its buffer gets what the ring leaves).
template <int FMT, int DP, int NT>
struct DecCfg {
  static constexpr int ES = FMT == CF_E4M3 ? 1 : 2;
  static constexpr int ROW = DP * ES;  // bytes of a row in shared memory
  static constexpr int MT = 2 * ROW * 32 <= 8192 ? 2 : 1;
  static constexpr int TW = 16 * MT;
  static constexpr int KV = 2 * TW * ROW;
  static constexpr int WARPS = KV <= 8192 ? 8 : 4;
  static constexpr int STAGES = 196608 / (WARPS * KV);
  static constexpr int STAGE = KV + (FMT == CF_E4M3 ? 8 * TW : 0) + 16;  // rows, scales, mask
  static constexpr int HEADS = 8 * NT;
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int ML = WARPS * HEADS * 3 * 4;
  static constexpr int room() { return 227 * 1024 - 256 - RING - ML; }
  static constexpr int join_bytes(int pd) { return WARPS * HEADS * (pd + 4) * 4; }
  static constexpr int fit(int pd) { return join_bytes(pd) <= room() ? pd : fit(pd / 2); }
  static constexpr int PD = fit(DP);
  static constexpr int SMEM = RING + ML + join_bytes(PD) + 256;
  static constexpr int REC = HEADS * (DP + 2);  // floats of a record
  static_assert(STAGES >= 2 && SMEM <= 227 * 1024 && PD % 16 == 0, "does not fit");
  static_assert(DEC_MAX_BLOCKS * HEADS * 4 <= join_bytes(PD), "the records' weights use the join buffer");
};
constexpr int DEC_MAX_REC = 16 * (256 + 2);

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
// two E4M3 codes (the low 16 bits) -> two fp16
K3_DEVI uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t y;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(y) : "r"(w));
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
  if constexpr (ROW % 128 == 0) {
    if constexpr (FMT == CF_E4M3) {
      const int f = ((r & 1) << 2) | ((r >> 1) & 3);
      return r * ROW + ((c ^ f) << 4);
    }
    return r * ROW + ((c ^ (r & 7)) << 4);
  } else {  // an odd number of 64-byte pieces a row
    return r * ROW + ((c ^ ((r >> 1) & 3)) << 4);
  }
}

// length of sequence b within what its table can hold
K3_DEVI int32_t seq_len(const DecodeParams& p, int b, bool& bad) {
  const int32_t n = __ldg(p.lens + b);
  const int64_t most = (int64_t)p.table_width * p.c.page_size;
  bad = n < 0 || n > most;
  return n < 0 ? 0 : (n > most ? (int32_t)most : n);
}

// A place in the order of the units: sequence b, head group hr of its Hkv * groups, unit u of nu.
template <int UNIT>
struct DecAt {
  int32_t b, hr, u, nu, first, n;
  K3_DEVI bool open(const DecodeParams& p) {  // sequence b's tokens and units; false: a bad length
    bool bad;
    n = seq_len(p, b, bad);
    first = p.window > 0 && n > p.window ? n - p.window : 0;
    nu = (n - first) / UNIT + ((n - first) % UNIT != 0);
    return !bad;
  }
  K3_DEVI void next(const DecodeParams& p) {
    if (++u < nu) return;
    u = 0;
    if (++hr < p.Hkv * p.groups) return;
    hr = 0;
    do {
      if (++b >= p.B) return;
      open(p);
    } while (nu == 0);
  }
};

template <int FMT, int DP, int NT>
__global__ void __launch_bounds__(DecCfg<FMT, DP, NT>::WARPS * 32, 1) k3_decode_kernel(const DecodeParams p) {
  using C = DecCfg<FMT, DP, NT>;
  constexpr int WARPS = C::WARPS, THREADS = WARPS * 32, TW = C::TW, MT = C::MT, STAGES = C::STAGES, ROW = C::ROW;
  constexpr int UNIT = WARPS * TW, HEADS = C::HEADS, KSTEPS = DP / 16, PD = C::PD;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ring = smem_u32(smem) + warp * STAGES * C::STAGE;
  float* s_ml = reinterpret_cast<float*>(smem + C::RING);  // [WARPS][HEADS] maxima, sums, value maxima
  float* s_join = reinterpret_cast<float*>(smem + C::RING + C::ML);
  int64_t* s_misc = reinterpret_cast<int64_t*>(smem + C::SMEM - 256);

  // dims past D: zero in every stage, never written again
  if (p.D < DP)
    for (int i = threadIdx.x; i < C::RING / 16; i += THREADS)
      *reinterpret_cast<uint4*>(smem + 16 * i) = make_uint4(0, 0, 0, 0);

  grid_dep_wait();
  grid_dep_launch();

  // ---- this block's units: all units counted, and the sequence that holds the first one found
  const int32_t HR = p.Hkv * p.groups;
  const int per = (p.B + THREADS - 1) / THREADS;
  DecAt<UNIT> at;
  int64_t mine = 0;
  const int b_lo = min(p.B, (int)threadIdx.x * per), b_hi = min(p.B, b_lo + per);
  bool any_bad = false;
  for (at.b = b_lo; at.b < b_hi; ++at.b) {
    any_bad |= !at.open(p);
    mine += at.nu;
  }
  if (any_bad && blockIdx.x == 0) flag_status(p.status, K3ATTN_DEV_BAD_LENGTH);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) s_misc[warp] = upto;
  __syncthreads();
  int64_t all = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w == warp) upto += all;
    all += s_misc[w];
  }
  const int64_t total = all * HR;
  const int64_t chunk = max((int64_t)1, (total + gridDim.x - 1) / gridDim.x);
  const int64_t unit0 = blockIdx.x * chunk;
  const int64_t left64 = min(total, unit0 + chunk) - unit0;
  if (left64 > 0 && mine > 0 && unit0 >= (upto - mine) * HR && unit0 < upto * HR) {
    int64_t before = (upto - mine) * HR;
    for (at.b = b_lo;; ++at.b) {
      at.open(p);
      if (unit0 < before + (int64_t)at.nu * HR) break;
      before += (int64_t)at.nu * HR;
    }
    s_misc[8] = at.b;
    s_misc[9] = unit0 - before;
  }
  __syncthreads();

  if (left64 > 0) {
    const int32_t units = (int32_t)min(left64, (int64_t)INT32_MAX);
    at.b = (int32_t)s_misc[8];
    at.open(p);
    at.hr = (int32_t)(s_misc[9] / at.nu);
    at.u = (int32_t)(s_misc[9] % at.nu);
    DecAt<UNIT> ahead = at;  // the tile whose page entries are in `entry`
    int32_t entry = 0, issued = 0;

    // row `lane` (of TW) of the tile at `ahead`
    auto row_token = [&]() { return ahead.first + (ahead.u * WARPS + warp) * TW + (lane & (TW - 1)); };
    auto fetch = [&]() {  // the tile's page entries
      const int32_t t = row_token();
      entry = 0;
      if (t < ahead.n) {
        const uint32_t pg = p.c.by_page(t);
        entry = __ldg(p.table + (int64_t)ahead.b * p.table_width + pg);
      }
    };
    auto issue = [&](int stage) {  // the copies of the tile at `ahead`
      const uint32_t st = ring + stage * C::STAGE;
      const int32_t t = row_token();
      const bool in = t < ahead.n;
      const bool ok = in && entry >= 0 && entry < p.c.n_pages;
      if (in && !ok) flag_status(p.status, K3ATTN_DEV_BAD_PAGE);
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
      if (lane == 0) *reinterpret_cast<uint32_t*>(__cvta_shared_to_generic(st + C::STAGE - 16)) = mask;
      if (mask == 0) return;
      const int32_t kvh = ahead.hr / p.groups;
      const uint32_t pg = p.c.by_page(t);
      const int64_t in_page = t - (int32_t)(pg * (uint32_t)p.c.page_size);
      const int64_t off = ok ? entry * p.c.page + kvh * p.c.head + in_page * p.c.tok : 0;
      if constexpr (FMT == CF_E4M3) {
        const int64_t so = ok ? entry * p.c.spage + kvh * p.c.shead + in_page * p.c.stok : 0;
        const uint32_t dst = st + C::KV + 4 * (lane & (TW - 1));
        if (TW == 32 || lane < 16) cp_async4_or_zero(dst, p.c.ks + so, ok ? 4 : 0);
        if (TW == 32 || lane >= 16) cp_async4_or_zero(dst + 4 * TW, p.c.vs + so, ok ? 4 : 0);
      }
      constexpr int CPR = ROW / 16;
      const int cpr = p.D * C::ES / 16;
#pragma unroll
      for (int i = 0; i < TW * CPR / 32; ++i) {
        const int r = (i * 32 + lane) / CPR, ch = (i * 32 + lane) % CPR;
        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r) + 16 * ch;
        const uint32_t n = (mask >> r) & 1u ? 16u : 0u;
        if (ch < cpr) {
          const uint32_t dst = st + chunk_at<FMT, ROW>(r, ch);
          cp_async16_or_zero(dst, p.c.k + (n ? o : 0), n);
          cp_async16_or_zero(dst + TW * ROW, p.c.v + (n ? o : 0), n);
        }
      }
    };
    // copies tile `issued` (if there is one) and fetches the entries of the next
    auto advance = [&](int stage) {
      if (issued < units) {
        issue(stage);
        ++issued;
        if (issued < units) {
          ahead.next(p);
          fetch();
        }
      }
      cp_async_commit();
    };
    fetch();
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) advance(s);

    float acc[KSTEPS][NT][4], m[NT][2], l[NT][2], vm[NT][2], qs[NT][2];
    uint32_t qf[KSTEPS][NT][2];
    int32_t seg_u0 = 0;
    int stage = 0;
    for (int32_t k = 0; k < units; ++k) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      advance(stage == 0 ? STAGES - 1 : stage - 1);
      const int32_t kvh = at.hr / p.groups, grp = at.hr - kvh * p.groups;
      const int32_t heads = min(HEADS, p.G - grp * HEADS);  // of this group
      const int64_t head0 = (int64_t)kvh * p.G + grp * HEADS;

      if (k == 0 || at.u == 0) {  // a new part: its queries, empty sums
        seg_u0 = at.u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int h = nt * 8 + lane / 4;
          const uint16_t* q = p.q + at.b * p.q_stride + (head0 + h) * p.D;
          const bool on = h < heads;
          if constexpr (FMT == CF_BF16) {
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int d = 16 * c + 8 * e + 2 * (lane & 3);
                qf[c][nt][e] = on && d < p.D ? __ldg(reinterpret_cast<const uint32_t*>(q + d)) : 0u;
              }
            qs[nt][0] = qs[nt][1] = p.scale;
          } else {
            // fp16, scaled by the power of two that brings the row's largest into [2^14, 2^15);
            // step 4 j + i of the contraction holds dims 64 j + 16 (lane % 4) + 4 i .. + 3
            uint2 raw[KSTEPS];
            uint32_t mx = 0;
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c) {
              const int d = 64 * (c / 4) + 16 * (lane & 3) + 4 * (c & 3);
              raw[c] = on && d < p.D ? ldg64(q + d) : make_uint2(0, 0);
              mx = max(max(mx, raw[c].x & 0x7FFFu), max((raw[c].x >> 16) & 0x7FFFu, raw[c].y & 0x7FFFu));
              mx = max(mx, (raw[c].y >> 16) & 0x7FFFu);
            }
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            const int pw = act_exp_from_max(mx << 16);
            const float f1 = pow2f(pw >> 1), f2 = pow2f(pw - (pw >> 1));
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c) {
              const uint32_t w[2] = {raw[c].x, raw[c].y};
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const __half2 hh = __floats2half2_rn(__uint_as_float(w[e] << 16) * f1 * f2,
                                                     __uint_as_float(w[e] & 0xFFFF0000u) * f1 * f2);
                qf[c][nt][e] = *reinterpret_cast<const uint32_t*>(&hh);
              }
            }
            // the scale's inverse, for the two heads whose logits this lane holds
            const float inv = p.scale * pow2f(-(pw >> 1)) * pow2f((pw >> 1) - pw);
#pragma unroll
            for (int e = 0; e < 2; ++e) qs[nt][e] = __shfl_sync(0xFFFFFFFFu, inv, 4 * (2 * (lane & 3) + e));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            m[nt][e] = vm[nt][e] = -INFINITY;
            l[nt][e] = 0.f;
          }
#pragma unroll
          for (int c = 0; c < KSTEPS; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][nt][e] = 0.f;
        }
      }

      const uint32_t st = ring + stage * C::STAGE;
      const uint32_t mask = lds32(st + C::STAGE - 16);
      if (mask != 0) {
        // ---- logits: lane holds tokens lane / 4 and + 8 of each 16, heads 2 (lane % 4) and + 1
        float s[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
          if constexpr (FMT == CF_BF16) {
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c) {
              uint32_t a[4];
              ldsm4(a, st + chunk_at<FMT, ROW>(16 * mt + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_bf16(s[mt][nt], a, qf[c][nt][0], qf[c][nt][1], s[mt][nt]);
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
                  mma_f16(s[mt][nt], a, qf[4 * j + i][nt][0], qf[4 * j + i][nt][1], s[mt][nt]);
              }
            }
          }
        }
        // ---- weights
        float lvs[MT][2];  // log2 of the values' scales
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 16 * mt + lane / 4 + 8 * e;
            const bool ok = (mask >> r) & 1u;
            float ks = 1.f;
            if constexpr (FMT == CF_E4M3) {
              ks = lds_f32(st + C::KV + 4 * r);
              lvs[mt][e] = lg2(lds_f32(st + C::KV + 4 * (TW + r)));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float& x = s[mt][nt][2 * e + h];
                x = ok ? x * ks * qs[nt][h] : -INFINITY;
              }
          }
        uint32_t pf[MT][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float base[2], vbase[2], fall[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float t = -INFINITY, tv = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                t = fmaxf(t, s[mt][nt][2 * e + h]);
                if constexpr (FMT == CF_E4M3) tv = fmaxf(tv, s[mt][nt][2 * e + h] + lvs[mt][e]);
              }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
              if constexpr (FMT == CF_E4M3) tv = fmaxf(tv, __shfl_xor_sync(0xFFFFFFFFu, tv, o));
            }
            const float m1 = fmaxf(m[nt][h], t);
            base[h] = m1 == -INFINITY ? 0.f : m1;
            const float f = ex2(m[nt][h] - base[h]);
            m[nt][h] = m1;
            l[nt][h] *= f;
            fall[h] = f;
            if constexpr (FMT == CF_E4M3) {
              const float v1 = fmaxf(vm[nt][h], tv);
              vbase[h] = v1 == -INFINITY ? 0.f : v1;
              fall[h] = ex2(vm[nt][h] - vbase[h]);
              vm[nt][h] = v1;
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float w[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float x = s[mt][nt][2 * e + h], pr = ex2(x - base[h]);
                l[nt][h] += pr;
                w[h] = FMT == CF_E4M3 ? ex2(x + lvs[mt][e] - vbase[h]) : pr;
              }
              // a masked token's scale is not read (its logit is -infinity, the sum NaN if its
              // place held garbage): zero-filled, log2 -infinity, weight 0
              if constexpr (FMT == CF_E4M3) {
                const __half2 hh = __floats2half2_rn(w[0], w[1]);
                pf[mt][nt][e] = movm(*reinterpret_cast<const uint32_t*>(&hh));
              } else {
                const __nv_bfloat162 hh = __floats2bfloat162_rn(w[0], w[1]);
                pf[mt][nt][e] = movm(*reinterpret_cast<const uint32_t*>(&hh));
              }
            }
          if (__any_sync(0xFFFFFFFFu, fall[0] != 1.f || fall[1] != 1.f))
#pragma unroll
            for (int c = 0; c < KSTEPS; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[c][nt][e] *= fall[e & 1];
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
              for (int nt = 0; nt < NT; ++nt) mma_bf16(acc[c][nt], a, pf[mt][nt][0], pf[mt][nt][1], acc[c][nt]);
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
                  mma_f16(acc[c + e][nt], a, pf[mt][nt][0], pf[mt][nt][1], acc[c + e][nt]);
              }
            }
          }
        }
      }
      stage = stage == STAGES - 1 ? 0 : stage + 1;

      // ---- the end of a part: join the warps, then write the result or leave a record
      if (k == units - 1 || at.u == at.nu - 1) {
        const bool whole = seg_u0 == 0 && at.u == at.nu - 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[nt][h] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][h], o);
            if (lane < 4) {
              float* x = s_ml + (warp * HEADS + nt * 8 + 2 * lane + h) * 3;
              x[0] = m[nt][h];
              x[1] = l[nt][h];
              x[2] = FMT == CF_E4M3 ? vm[nt][h] : m[nt][h];
            }
          }
        float* rec = p.parts + (2 * (int64_t)blockIdx.x + (seg_u0 == at.u - k ? 0 : 1)) * C::REC;
#pragma unroll
        for (int pass = 0; pass < DP / PD; ++pass) {
#pragma unroll
          for (int c = pass * (PD / 16); c < (pass + 1) * (PD / 16); ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float* x = s_join + (warp * HEADS + nt * 8 + 2 * (lane & 3) + h) * (PD + 4) + 16 * c - pass * PD;
                if constexpr (FMT == CF_BF16) {
                  x[lane / 4] = acc[c][nt][h];
                  x[lane / 4 + 8] = acc[c][nt][2 + h];
                } else {
                  *reinterpret_cast<float2*>(x + 2 * (lane / 4)) = make_float2(acc[c][nt][h], acc[c][nt][2 + h]);
                }
              }
          __syncthreads();
          for (int i = threadIdx.x; i < heads * (PD / 4); i += THREADS) {
            const int h = i / (PD / 4), d = 4 * (i % (PD / 4));
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_ml[(w * HEADS + h) * 3]);
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
              const float* x = s_ml + (w * HEADS + h) * 3;
              sum += x[1] * ex2(x[0] - base);
              const float f = ex2(x[2] - base);
              const float4 v = *reinterpret_cast<const float4*>(s_join + (w * HEADS + h) * (PD + 4) + d);
              o[0] = fmaf(v.x, f, o[0]);
              o[1] = fmaf(v.y, f, o[1]);
              o[2] = fmaf(v.z, f, o[2]);
              o[3] = fmaf(v.w, f, o[3]);
            }
            const int dim = pass * PD + d;
            if (whole) {
              const float r = sum == 0.f ? 0.f : 1.f / sum;
              const int64_t row = (int64_t)at.b * p.Hq + head0 + h;
              if (dim < p.D) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(sum == 0.f ? 0.f : o[0] * r, sum == 0.f ? 0.f : o[1] * r);
                const __nv_bfloat162 hi = __floats2bfloat162_rn(sum == 0.f ? 0.f : o[2] * r, sum == 0.f ? 0.f : o[3] * r);
                *reinterpret_cast<uint2*>(p.out + row * p.D + dim) = make_uint2(
                    *reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
              }
              if (dim == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
            } else {
              __stcg(reinterpret_cast<float4*>(rec + h * DP + dim), make_float4(o[0], o[1], o[2], o[3]));
              if (dim == 0) {
                __stcg(rec + HEADS * DP + h, top);
                __stcg(rec + HEADS * DP + HEADS + h, sum);
              }
            }
          }
          __syncthreads();
        }
        if (!whole) {
          // the blocks of this (sequence, head group): units i0 .. i1 - 1 of all
          const int64_t i0 = unit0 + k - at.u, i1 = i0 + at.nu;
          const int32_t c0 = (int32_t)(i0 / chunk), c1 = (int32_t)((i1 - 1) / chunk), parts = c1 - c0 + 1;
          int32_t* s_last = reinterpret_cast<int32_t*>(s_misc + 10);
          if (threadIdx.x == 0) {
            __threadfence();
            *s_last = atomicAdd(p.arrived + c0, 1u) == (uint32_t)(parts - 1);
          }
          __syncthreads();
          if (*s_last) {
            __threadfence();
            if (threadIdx.x == 0) p.arrived[c0] = 0;
            auto record = [&](int i) {  // block c0's part is its first only where it begins there
              return p.parts + (2 * (int64_t)(c0 + i) + (i == 0 && i0 != c0 * chunk ? 1 : 0)) * C::REC;
            };
            // the records' weights [parts][HEADS] into the join buffer
            for (int h = warp; h < heads; h += WARPS) {
              float top = -INFINITY, sum = 0.f;
              for (int i = lane; i < parts; i += 32) top = fmaxf(top, __ldcg(record(i) + HEADS * DP + h));
#pragma unroll
              for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
              const float base = top == -INFINITY ? 0.f : top;
              for (int i = lane; i < parts; i += 32) {
                const float f = ex2(__ldcg(record(i) + HEADS * DP + h) - base);
                s_join[i * HEADS + h] = f;
                sum += f * __ldcg(record(i) + HEADS * DP + HEADS + h);
              }
#pragma unroll
              for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
              if (lane == 0) {
                s_ml[h] = sum;
                if (p.lse)
                  p.lse[(int64_t)at.b * p.Hq + head0 + h] =
                      sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
              }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < heads * (DP / 4); i += THREADS) {
              const int h = i / (DP / 4), d = 4 * (i % (DP / 4));
              if (d >= p.D) continue;
              float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
              for (int j = 0; j < parts; ++j) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(record(j) + h * DP + d));
                const float f = s_join[j * HEADS + h];
                o[0] = fmaf(v.x, f, o[0]);
                o[1] = fmaf(v.y, f, o[1]);
                o[2] = fmaf(v.z, f, o[2]);
                o[3] = fmaf(v.w, f, o[3]);
              }
              const float sum = s_ml[h], r = 1.f / sum;
              const __nv_bfloat162 lo = __floats2bfloat162_rn(sum == 0.f ? 0.f : o[0] * r, sum == 0.f ? 0.f : o[1] * r);
              const __nv_bfloat162 hi = __floats2bfloat162_rn(sum == 0.f ? 0.f : o[2] * r, sum == 0.f ? 0.f : o[3] * r);
              *reinterpret_cast<uint2*>(p.out + ((int64_t)at.b * p.Hq + head0 + h) * p.D + d) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            }
            __syncthreads();
          }
        }
      }
      at.next(p);
    }
    cp_async_wait<0>();
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
