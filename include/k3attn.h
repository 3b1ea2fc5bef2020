/*
 * k3attn.h -- C ABI of the attention operators that stand before the routed-expert block
 * of a decoder layer when it serves tokens: norms of queries and keys for each head with
 * the position rotation, a paged key-value cache (16 bits, or quantised to 8 as it is
 * written), and the attention of one new token over its pages.
 *
 * With D = head_dim, R = rot_dim, per token at position p and per head row x in R^D:
 *
 *   n   = w * x / sqrt(mean(x^2) + eps)           w: one weight vector for all query heads,
 *                                                 one for all key heads
 *   y   = n, but for the R / 2 pairs (n0, n1) of its first R elements:
 *         (n0 cos a_i - n1 sin a_i, n1 cos a_i + n0 sin a_i),  a_i = p * inv_freq[i]
 *         pair i: elements i and i + R/2, or with rot_interleaved 2i and 2i + 1
 *
 * The cache holds, for each token and each of the Hkv key heads, a row of D values for K
 * and one for V, in one of two formats:
 *   K3ATTN_BF16  the row rounded to bf16
 *   K3ATTN_E4M3  D codes and one f32 scale:  s = max(amax / 448, 2^-100), amax = max |row|;
 *                code = e4m3(value * (1 / s)), rounded to nearest even and saturated at 448;
 *                the value read back is code * s.  A row with an infinity or a NaN gets a
 *                NaN scale and NaN codes: all of it reads back as NaN.
 * A token's place is its slot: page * page_size + place in the page.
 *
 * Attention of one new token per sequence b over the cached tokens f .. len_b - 1,
 * f = max(0, len_b - window) with a window, else 0 (the new token's own key and value are in
 * the cache, len_b counts it); query head h reads key head j = h / (Hq / Hkv):
 *
 *   l_t = softmax_scale * q_h . k_t,j     out_h = sum_t e^(l_t) v_t,j / sum_t e^(l_t)
 *   lse_h = log sum_t e^(l_t)
 * A sequence with nothing to attend to (len_b = 0, or every l_t = -infinity) gives out 0 and
 * lse -infinity.  Nothing outside f .. len_b - 1 is read: what pages hold there (stale rows,
 * NaN) has no part in the result.
 *
 * Conventions: those of k3moe.h (device pointers, 16-byte aligned; bf16 as uint16_t; host
 * validation before any launch; the caller owns all memory; nothing is allocated or
 * synchronised; calls can be captured into graphs), but index arrays (positions, slots,
 * page_table, lens), scales and lse need 4-byte alignment only, inv_freq 8.  The workspace
 * differs in one point:
 *   - Set it up ONCE with k3attn_workspace_init.  Calls leave its counters ready for the
 *     next call, and OR device-detected conditions (K3ATTN_DEV_*) into its first word, where
 *     they stay until the next k3attn_workspace_init; read them with k3moe_device_status.
 *   - One workspace serves any head shape that it is large enough for, and calls that run
 *     one after the other.  Calls that may overlap need workspaces of their own.
 */
#ifndef K3ATTN_H
#define K3ATTN_H

#include "k3moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define K3ATTN_BF16 0
#define K3ATTN_E4M3 1

typedef struct {
  int32_t n_heads;         /* Hq: query heads, 1..1024 */
  int32_t n_kv_heads;      /* Hkv: key and value heads; divides n_heads */
  int32_t head_dim;        /* D: multiple of 16, 16..256 */
  int32_t rot_dim;         /* R: multiple of 16, 0..D (0: no rotation) */
  int32_t rot_interleaved; /* 0: pairs (i, i + R/2); 1: pairs (2i, 2i + 1) */
  float rms_eps;           /* epsilon of the norms, 0..1 */
  float softmax_scale;     /* > 0, e.g. 1 / sqrt(D) */
  int32_t window;          /* attend to the last `window` tokens; 0: to all */
} k3attn_dims;

/* A paged cache.  k and v have the same strides (in elements), k_scale and v_scale theirs;
 * the D values of a row are dense.  Dense pages [n_pages, Hkv, page_size, D] have
 * token_stride D, head_stride page_size * D, page_stride Hkv * page_size * D; any other
 * order of pages, heads and tokens is described by its strides (rows must not overlap).
 * A row must start at a multiple of 16 bytes: strides are multiples of 16 elements
 * (K3ATTN_E4M3) or 8 (K3ATTN_BF16).  n_pages * page_size is below 2^31 (slots are int32);
 * offsets in the cache may pass 32 bits. */
typedef struct {
  void* k;
  void* v;
  float* k_scale; /* K3ATTN_E4M3 only; else NULL */
  float* v_scale;
  int32_t format; /* K3ATTN_BF16, K3ATTN_E4M3 */
  int32_t n_pages;
  int32_t page_size; /* tokens in a page, any positive number */
  int32_t reserved;  /* 0 */
  int64_t page_stride, head_stride, token_stride;
  int64_t scale_page_stride, scale_head_stride, scale_token_stride;
} k3attn_cache;

/* Bits of the status word at the start of the workspace. */
#define K3ATTN_DEV_BAD_SLOT 0x1u   /* a slot outside the cache (and not -1): a write was skipped, a
                                      read gave zeros */
#define K3ATTN_DEV_BAD_PAGE 0x2u   /* a page of a sequence's attended tokens is not in the cache:
                                      its tokens were left out */
#define K3ATTN_DEV_BAD_LENGTH 0x4u /* a length outside 0 .. table_width * page_size: taken as the
                                      nearest of these */

/* Bytes of workspace for k3attn_decode with these dims; the other calls need the first
 * K3ATTN_MIN_WORKSPACE of them.  0 for invalid dims. */
#define K3ATTN_MIN_WORKSPACE 256u
size_t k3attn_workspace_bytes(const k3attn_dims* dims);

/* Readies a workspace, once before its first use (clears the status word and the counters
 * on `stream`). */
k3moe_status k3attn_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* Norms of queries and keys for each head, with the rotation, for T tokens.
 *   q [T] rows of Hq * D bf16, q_stride elements apart;  k likewise with Hkv * D
 *     (slices of one projection's output: strides are multiples of 8, at least a row)
 *   positions [T] int32;  inv_freq [R / 2] f64 (NULL when R = 0)
 *   q_w, k_w [D] f32 norm weights
 *   q_out [T, Hq, D], k_out [T, Hkv, D] bf16; either may be its input where that is dense
 * Everything is held in fp32 (angles in fp64, reduced to a turn) and rounded once.  A row whose
 * sum of squares passes fp32's range (elements of about 1e18 and more) therefore comes out as
 * zeros, and with rms_eps = 0 one whose sum vanishes there as infinities or NaN.  T = 0 is a
 * no-op. */
k3moe_status k3attn_qk_norm_rope(const k3attn_dims* dims, int32_t T, const uint16_t* q, int64_t q_stride,
                                 const uint16_t* k, int64_t k_stride, const int32_t* positions,
                                 const double* inv_freq, const float* q_w, const float* k_w, uint16_t* q_out,
                                 uint16_t* k_out, void* stream);

/* Keys and values of T tokens into the cache as they are (quantised by its format).
 *   k, v [T] rows of Hkv * D bf16, k_stride and v_stride elements apart
 *   slots [T] int32: distinct places, -1 for a token that is not written
 * dims: the head counts and head_dim. */
k3moe_status k3attn_kv_write(const k3attn_dims* dims, int32_t T, const uint16_t* k, int64_t k_stride,
                             const uint16_t* v, int64_t v_stride, const int32_t* slots, const k3attn_cache* cache,
                             void* ws, size_t ws_bytes, void* stream);

/* One pass over the new tokens' q, k and v: k3attn_qk_norm_rope for q (into q_out) and k, and
 * k3attn_kv_write of the keys (before any rounding to 16 bits) and the values.  k_out
 * [T, Hkv, D] bf16 also receives the keys unless it is NULL. */
k3moe_status k3attn_kv_append(const k3attn_dims* dims, int32_t T, const uint16_t* q, int64_t q_stride,
                              const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                              const int32_t* positions, const int32_t* slots, const double* inv_freq,
                              const float* q_w, const float* k_w, const k3attn_cache* cache, uint16_t* q_out,
                              uint16_t* k_out, void* ws, size_t ws_bytes, void* stream);

/* The rows of T slots back as bf16: k_out, v_out [T, Hkv, D] (zeros for slot -1). */
k3moe_status k3attn_kv_read(const k3attn_dims* dims, int32_t T, const int32_t* slots, const k3attn_cache* cache,
                            uint16_t* k_out, uint16_t* v_out, void* ws, size_t ws_bytes, void* stream);

/* Attention of one new token for each of B sequences.
 *   q [B] rows of Hq * D bf16, q_stride elements apart;  B at most 65535
 *   page_table [B, table_width] int32: the pages of each sequence in order; entries past its
 *     last attended token, and before its first one, are not read
 *   lens [B] int32: cached tokens of each sequence, the new one included; table_width *
 *     page_size is below 2^31.  They must not change while the call runs
 *   out [B, Hq, D] bf16;  lse [B, Hq] f32 or NULL
 * The work is split evenly over the SMs whatever the lengths, which are read on the device
 * (a captured call replays with new ones).  With more than 8 query heads a key head the longest
 * length that table_width and window allow decides between two ways to group the heads: a table
 * much wider than the sequences is right, and slower for few short ones.  The result does not
 * depend on the order in which the parts finish.
 * Logits, softmax statistics and sums are held in fp32, powers of two to 2^-22.  A token's weight
 * enters the sum of values rounded to the type of its product, bf16 for a K3ATTN_BF16 cache (off
 * by 2^-8 of itself at most), fp16 for K3ATTN_E4M3 (2^-11, or 2^-40 of the largest); the sum of
 * weights is of the unrounded ones.  The result is rounded to bf16 once. */
k3moe_status k3attn_decode(const k3attn_dims* dims, int32_t B, const uint16_t* q, int64_t q_stride,
                           const k3attn_cache* cache, const int32_t* page_table, int32_t table_width,
                           const int32_t* lens, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* K3ATTN_H */
