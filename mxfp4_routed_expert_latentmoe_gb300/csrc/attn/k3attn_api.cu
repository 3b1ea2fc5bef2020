// k3attn_api.cu -- C ABI of the attention operators (see include/k3attn.h): host-side
// validation and launches.  No allocation, no synchronisation.
#include <atomic>
#include <cmath>
#include <utility>

#include "k3_decode.cuh"
#include "k3_qkv.cuh"

namespace {

using namespace k3;

constexpr int kMaxDevices = 64;

#define K3A_TRY(x)                                       \
  do {                                                   \
    if ((x) != cudaSuccess) {                            \
      (void)cudaGetLastError();                          \
      return K3MOE_ERR_CUDA;                             \
    }                                                    \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

k3moe_status check_dims(const k3attn_dims* d) {
  if (!d) return K3MOE_ERR_ARG;
  if (d->n_heads <= 0 || d->n_heads > 1024 || d->n_kv_heads <= 0 || d->n_heads % d->n_kv_heads) return K3MOE_ERR_SHAPE;
  if (d->head_dim < 16 || d->head_dim > 256 || d->head_dim % 16) return K3MOE_ERR_SHAPE;
  if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % 16) return K3MOE_ERR_SHAPE;
  if (d->rot_interleaved != 0 && d->rot_interleaved != 1) return K3MOE_ERR_ARG;
  if (!(d->rms_eps >= 0.0f) || d->rms_eps > 1.0f) return K3MOE_ERR_ARG;
  if (!(d->softmax_scale > 0.0f) || std::isinf(d->softmax_scale)) return K3MOE_ERR_ARG;
  if (d->window < 0) return K3MOE_ERR_ARG;
  return K3MOE_OK;
}

k3moe_status check_cache(const k3attn_cache* c, const k3attn_dims& d) {
  if (!c || !c->k || !c->v) return K3MOE_ERR_ARG;
  if (c->format != K3ATTN_BF16 && c->format != K3ATTN_E4M3) return K3MOE_ERR_ARG;
  const bool e4m3 = c->format == K3ATTN_E4M3;
  if (e4m3 && (!c->k_scale || !c->v_scale)) return K3MOE_ERR_ARG;
  if (c->n_pages <= 0 || c->page_size <= 0 || c->reserved != 0) return K3MOE_ERR_ARG;
  if ((int64_t)c->n_pages * c->page_size > INT32_MAX) return K3MOE_ERR_SHAPE;  // slots are int32
  if (c->page_stride < d.head_dim || c->head_stride < d.head_dim || c->token_stride < d.head_dim)
    return K3MOE_ERR_SHAPE;
  const int64_t unit = e4m3 ? 16 : 8;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % unit || c->head_stride % unit ||
      c->token_stride % unit)
    return K3MOE_ERR_ALIGN;
  if (e4m3) {
    if (c->scale_page_stride < 1 || c->scale_head_stride < 1 || c->scale_token_stride < 1) return K3MOE_ERR_SHAPE;
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return K3MOE_ERR_ALIGN;
  }
  return K3MOE_OK;
}

CacheView view_of(const k3attn_cache& c) {
  const int64_t b = c.format == K3ATTN_E4M3 ? 1 : 2;
  CacheView v{};
  v.k = static_cast<uint8_t*>(c.k);
  v.v = static_cast<uint8_t*>(c.v);
  v.ks = c.k_scale;
  v.vs = c.v_scale;
  v.page = c.page_stride * b;
  v.head = c.head_stride * b;
  v.tok = c.token_stride * b;
  v.spage = c.scale_page_stride;
  v.shead = c.scale_head_stride;
  v.stok = c.scale_token_stride;
  v.n_pages = c.n_pages;
  v.page_size = c.page_size;
  v.by_page = Divisor::of((uint32_t)c.page_size);
  return v;
}

// rows of `width` bf16 values, `stride` apart
k3moe_status check_rows(int64_t stride, int64_t width) {
  if (stride < width) return K3MOE_ERR_SHAPE;
  return stride % 8 ? K3MOE_ERR_ALIGN : K3MOE_OK;
}

struct DevInfo {
  int sms = 0;
  bool ok = false;
};
DevInfo g_dev[kMaxDevices];
std::atomic<bool> g_dev_init[kMaxDevices];

k3moe_status check_device(int* dev_out, int* sms_out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)cudaGetLastError();
    return K3MOE_ERR_DEVICE;
  }
  if (!g_dev_init[dev].load(std::memory_order_acquire)) {
    int major = 0, minor = 0, sms = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    g_dev[dev].sms = sms;
    g_dev[dev].ok = (major == 10 && minor == 3);
    g_dev_init[dev].store(true, std::memory_order_release);
  }
  if (!g_dev[dev].ok) return K3MOE_ERR_DEVICE;
  *dev_out = dev;
  *sms_out = g_dev[dev].sms;
  return K3MOE_OK;
}

// Launch with programmatic stream serialization: the kernel may start while its predecessor
// finishes; it waits (griddepcontrol.wait) before it touches memory.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, dim3 block, int smem, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

QkvParams qkv_params(const k3attn_dims& d, int32_t T) {
  QkvParams p{};
  p.T = T;
  p.Hq = d.n_heads;
  p.Hkv = d.n_kv_heads;
  p.D = d.head_dim;
  p.R = d.rot_dim;
  p.inter = d.rot_interleaved;
  p.eps = d.rms_eps;
  return p;
}

// lanes of a row: eight elements each
int lanes_of(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }

// ITEMS items a thread where that leaves every SM a block (a smaller call waits for latency:
// its items are spread out, one a thread)
template <int FMT, bool WRITE, int ITEMS>
cudaError_t launch_rows_t(const QkvParams& p, int lpr, int64_t grid, cudaStream_t s) {
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch(lpr == 8 ? k3_rows_kernel<8, FMT, WRITE, ITEMS>
                         : (lpr == 16 ? k3_rows_kernel<16, FMT, WRITE, ITEMS> : k3_rows_kernel<32, FMT, WRITE, ITEMS>),
                dim3((unsigned)grid), dim3(256), 0, s, p);
}
template <int FMT, bool WRITE>
cudaError_t launch_rows(QkvParams p, int sms, cudaStream_t s) {
  constexpr int ITEMS = 2;
  const int lpr = lanes_of(p.D);
  const int64_t items = (int64_t)p.T * p.Hkv, per = 256 / lpr;
  p.by_heads = Divisor::of(p.Hkv);
  const int64_t grid = (items + per * ITEMS - 1) / (per * ITEMS);
  if (grid >= sms) return launch_rows_t<FMT, WRITE, ITEMS>(p, lpr, grid, s);
  return launch_rows_t<FMT, WRITE, 1>(p, lpr, (items + per - 1) / per, s);
}

// The norms' blocks: ROWS rows a thread and just the warps that a token's rows take so; a token
// that takes more than a block has is cut into balanced parts, tokens of few rows share a block
// of up to 8 warps.  Keys and values for the cache have blocks of the same size.
template <int FMT, int ROWS>
cudaError_t launch_norm_t(QkvParams p, int sms, cudaStream_t s) {
  const int lpr = lanes_of(p.D), rows = p.Hq + (FMT == CF_NONE ? p.Hkv : 0);
  const int a_warp = 32 / lpr * ROWS, most = QKV_THREADS / 32 * a_warp;
  p.parts = (rows + most - 1) / most;
  p.rows = (rows + p.parts - 1) / p.parts;
  p.parts = (rows + p.rows - 1) / p.rows;
  const int token_warps = (p.rows + a_warp - 1) / a_warp;
  p.tokens = token_warps > 4 ? 1 : 8 / token_warps;
  if (p.tokens > p.T) p.tokens = p.T;
  const int warps = token_warps * p.tokens;
  p.kv_blocks = 0;
  if constexpr (FMT != CF_NONE) {
    const int kv_warp = 32 / lpr * (ROWS > 1 ? 2 : 1);
    p.kv_warps = (p.Hkv + kv_warp - 1) / kv_warp;
    if (p.kv_warps > warps) p.kv_warps = warps;
    p.kv_tokens = warps / p.kv_warps < QKV_TOKENS ? warps / p.kv_warps : QKV_TOKENS;
    p.kv_blocks = (int32_t)(((int64_t)p.T + p.kv_tokens - 1) / p.kv_tokens);
  }
  const int64_t grid = p.kv_blocks + ((int64_t)p.T + p.tokens - 1) / p.tokens * p.parts;
  if constexpr (ROWS > 1)
    if (grid < sms) return launch_norm_t<FMT, 1>(p, sms, s);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch(lpr == 8 ? k3_norm_kernel<8, FMT, ROWS>
                         : (lpr == 16 ? k3_norm_kernel<16, FMT, ROWS> : k3_norm_kernel<32, FMT, ROWS>),
                dim3((unsigned)grid), dim3(32 * warps), 0, s, p);
}
template <int FMT>
cudaError_t launch_norm(const QkvParams& p, int sms, cudaStream_t s) {
  return launch_norm_t<FMT, QKV_ROWS>(p, sms, s);
}

// per (kernel, device): raise the kernel's dynamic shared memory limit once
template <auto Kern>
bool set_smem(int dev, int bytes) {
  static std::atomic<bool> granted[kMaxDevices];
  if (granted[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  granted[dev].store(true, std::memory_order_release);
  return true;
}

// The decode workspace: the status word, the teams' counters (cleared once by
// k3attn_workspace_init), the teams' records.
constexpr size_t kCounters = K3ATTN_MIN_WORKSPACE, kRecords = kCounters + DEC_MAX_TEAMS * 4;
static_assert(kRecords % 16 == 0, "the records are written 16 bytes at a time");

// padded head dim and head group (8 NT query heads of a key head) of the decode instance
int dec_dp(const k3attn_dims& d) { return (d.head_dim + 63) / 64 * 64; }
int dec_nt(const k3attn_dims& d) { return d.n_heads / d.n_kv_heads <= 8 ? 1 : 2; }
// E4M3 heads past 192 dims: 8 query heads at a time, as 16 do not fit the registers (16 x 20000
// tokens of 2 key heads with 16 queries each, D 256: 65 us, 84 at 16 a time; the second pass
// over the rows finds most of them in L2.  bf16, which fits but for a few words: 114, 95 us)
int dec_nt_of(const k3attn_dims& d, int format) {
  return format == K3ATTN_E4M3 && d.head_dim > 192 ? 1 : dec_nt(d);
}

// Whether calls for more than 8 query heads a key head take them 8 at a time all the same: twice
// the tiles, but each instance's start and joins cost less than half, and a sequence has twice the
// teams.  Lengths are on the device, so the rule takes the longest that table and window allow:
// - a unit a block at most: 7 sequences up to 200 tokens, 16 heads a key head, D 128: bf16 8.1 us,
//   9.5 at 16 a time, E4M3 6.4, 7.9; 100 up to 200, above it: 12.4, 10.8, E4M3 12.1, 9.2
// - parts for a fifth of the blocks at most, cut between many teams, up to 16 units a block: 4 up
//   to 16000, D 128, bf16: 13.6 us, 20.0; 8 up to 8000, E4M3: 12.0, 15.3; but 18 up to 2000, 2 key
//   heads, bf16: 17.2, 15.8
// - E4M3, with no more parts than blocks, up to 4 units a block: 30 up to 800, 2 key heads, D 192:
//   15.4 us, 16.6, D 128: 12.4, 12.7; 30 up to 1600: 21.1, 20.3, D 128: 16.2, 15.4 (bf16 30 up to 800:
//   13.2, 12.5)
// - bf16 heads past 192 dims, whose 16 spill and are joined in two passes, up to 32 units a block: 1
//   up to 3000: 13.1 us, 33.3; 64 up to 1000: 32.7, 38.7; 200 up to 1000 (42): 45.8, 46.3
template <int FMT, int DP>
bool dec_narrow(const DecodeParams& p, int grid) {
  using C = DecCfg<FMT, DP, 1>;
  constexpr int UNIT = C::TW * C::WARPS;
  int64_t longest = (int64_t)p.table_width * p.c.page_size;
  if (p.window > 0 && p.window < longest) longest = p.window;
  const int64_t parts = (int64_t)p.B * p.Hkv * ((p.G + 7) / 8), units = parts * ((longest + UNIT - 1) / UNIT);
  const int most = FMT == CF_BF16 && DP > 192 ? 32
                   : 5 * parts <= grid        ? 16
                   : FMT == CF_E4M3 && parts <= grid ? 4 : 1;
  return units <= (int64_t)most * grid;
}

template <int FMT, int DP, int NT>
cudaError_t launch_decode_t(DecodeParams p, int dev, int sms, cudaStream_t s) {
  using C = DecCfg<FMT, DP, NT>;
  const int grid = sms < DEC_MAX_BLOCKS ? sms : DEC_MAX_BLOCKS;
  if constexpr (NT > 1)
    if (dec_narrow<FMT, DP>(p, grid)) return launch_decode_t<FMT, DP, 1>(p, dev, sms, s);
  if (!set_smem<k3_decode_kernel<FMT, DP, NT>>(dev, C::SMEM)) return cudaErrorInvalidValue;
  p.groups = (p.G + C::HEADS - 1) / C::HEADS;
  return launch(k3_decode_kernel<FMT, DP, NT>, dim3(grid), dim3(C::WARPS * 32), C::SMEM, s, p);
}
template <int FMT>
cudaError_t launch_decode(const DecodeParams& p, int dp, int nt, int dev, int sms, cudaStream_t s) {
  switch (dp * 2 + nt - 1) {
    case 128: return launch_decode_t<FMT, 64, 1>(p, dev, sms, s);
    case 129: return launch_decode_t<FMT, 64, 2>(p, dev, sms, s);
    case 256: return launch_decode_t<FMT, 128, 1>(p, dev, sms, s);
    case 257: return launch_decode_t<FMT, 128, 2>(p, dev, sms, s);
    case 384: return launch_decode_t<FMT, 192, 1>(p, dev, sms, s);
    case 385: return launch_decode_t<FMT, 192, 2>(p, dev, sms, s);
    case 512: return launch_decode_t<FMT, 256, 1>(p, dev, sms, s);
    case 513:
      if constexpr (FMT != CF_E4M3) return launch_decode_t<FMT, 256, 2>(p, dev, sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

extern "C" {

size_t k3attn_workspace_bytes(const k3attn_dims* dims) {
  if (check_dims(dims) != K3MOE_OK) return 0;
  return kRecords + (size_t)2 * DEC_MAX_TEAMS * 8 * dec_nt(*dims) * (dec_dp(*dims) + 2) * 4;
}

k3moe_status k3attn_workspace_init(void* ws, size_t ws_bytes, void* stream) {
  if (!ws) return K3MOE_ERR_ARG;
  if (!aligned(ws, 16)) return K3MOE_ERR_ALIGN;
  if (ws_bytes < K3ATTN_MIN_WORKSPACE) return K3MOE_ERR_WORKSPACE;
  int dev, sms;
  const k3moe_status st = check_device(&dev, &sms);
  if (st != K3MOE_OK) return st;
  K3A_TRY(cudaMemsetAsync(ws, 0, ws_bytes < kRecords ? ws_bytes : kRecords, static_cast<cudaStream_t>(stream)));
  return K3MOE_OK;
}

k3moe_status k3attn_qk_norm_rope(const k3attn_dims* dims, int32_t T, const uint16_t* q, int64_t q_stride,
                                 const uint16_t* k, int64_t k_stride, const int32_t* positions,
                                 const double* inv_freq, const float* q_w, const float* k_w, uint16_t* q_out,
                                 uint16_t* k_out, void* stream) {
  k3moe_status st = check_dims(dims);
  if (st != K3MOE_OK) return st;
  const k3attn_dims& d = *dims;
  if (T < 0) return K3MOE_ERR_ARG;
  if (T == 0) return K3MOE_OK;
  if (!q || !k || !positions || (d.rot_dim > 0 && !inv_freq) || !q_w || !k_w || !q_out || !k_out) return K3MOE_ERR_ARG;
  if ((st = check_rows(q_stride, (int64_t)d.n_heads * d.head_dim)) != K3MOE_OK) return st;
  if ((st = check_rows(k_stride, (int64_t)d.n_kv_heads * d.head_dim)) != K3MOE_OK) return st;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(positions, 4) || !aligned(inv_freq, 8) || !aligned(q_w, 16) ||
      !aligned(k_w, 16) || !aligned(q_out, 16) || !aligned(k_out, 16))
    return K3MOE_ERR_ALIGN;
  int dev, sms;
  if ((st = check_device(&dev, &sms)) != K3MOE_OK) return st;
  QkvParams p = qkv_params(d, T);
  p.q = q; p.q_stride = q_stride; p.k = k; p.k_stride = k_stride;
  p.pos = positions; p.inv_freq = inv_freq; p.q_w = q_w; p.k_w = k_w; p.q_out = q_out; p.k_out = k_out;
  K3A_TRY(launch_norm<CF_NONE>(p, sms, static_cast<cudaStream_t>(stream)));
  return K3MOE_OK;
}

k3moe_status k3attn_kv_write(const k3attn_dims* dims, int32_t T, const uint16_t* k, int64_t k_stride,
                             const uint16_t* v, int64_t v_stride, const int32_t* slots, const k3attn_cache* cache,
                             void* ws, size_t ws_bytes, void* stream) {
  k3moe_status st = check_dims(dims);
  if (st != K3MOE_OK) return st;
  const k3attn_dims& d = *dims;
  if ((st = check_cache(cache, d)) != K3MOE_OK) return st;
  if (T < 0) return K3MOE_ERR_ARG;
  if (T == 0) return K3MOE_OK;
  if (!k || !v || !slots || !ws) return K3MOE_ERR_ARG;
  if ((st = check_rows(k_stride, (int64_t)d.n_kv_heads * d.head_dim)) != K3MOE_OK) return st;
  if ((st = check_rows(v_stride, (int64_t)d.n_kv_heads * d.head_dim)) != K3MOE_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(ws, 16)) return K3MOE_ERR_ALIGN;
  if (ws_bytes < K3ATTN_MIN_WORKSPACE) return K3MOE_ERR_WORKSPACE;
  int dev, sms;
  if ((st = check_device(&dev, &sms)) != K3MOE_OK) return st;
  QkvParams p = qkv_params(d, T);
  p.k = k; p.k_stride = k_stride; p.v = v; p.v_stride = v_stride; p.slots = slots;
  p.c = view_of(*cache);
  p.status = static_cast<uint32_t*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  K3A_TRY((cache->format == K3ATTN_E4M3 ? launch_rows<CF_E4M3, true>(p, sms, s) : launch_rows<CF_BF16, true>(p, sms, s)));
  return K3MOE_OK;
}

k3moe_status k3attn_kv_append(const k3attn_dims* dims, int32_t T, const uint16_t* q, int64_t q_stride,
                              const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                              const int32_t* positions, const int32_t* slots, const double* inv_freq,
                              const float* q_w, const float* k_w, const k3attn_cache* cache, uint16_t* q_out,
                              uint16_t* k_out, void* ws, size_t ws_bytes, void* stream) {
  k3moe_status st = check_dims(dims);
  if (st != K3MOE_OK) return st;
  const k3attn_dims& d = *dims;
  if ((st = check_cache(cache, d)) != K3MOE_OK) return st;
  if (T < 0) return K3MOE_ERR_ARG;
  if (T == 0) return K3MOE_OK;
  if (!q || !k || !v || !positions || !slots || (d.rot_dim > 0 && !inv_freq) || !q_w || !k_w || !q_out || !ws)
    return K3MOE_ERR_ARG;
  if ((st = check_rows(q_stride, (int64_t)d.n_heads * d.head_dim)) != K3MOE_OK) return st;
  if ((st = check_rows(k_stride, (int64_t)d.n_kv_heads * d.head_dim)) != K3MOE_OK) return st;
  if ((st = check_rows(v_stride, (int64_t)d.n_kv_heads * d.head_dim)) != K3MOE_OK) return st;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(positions, 4) || !aligned(slots, 4) ||
      !aligned(inv_freq, 8) || !aligned(q_w, 16) || !aligned(k_w, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
      !aligned(ws, 16))
    return K3MOE_ERR_ALIGN;
  if (ws_bytes < K3ATTN_MIN_WORKSPACE) return K3MOE_ERR_WORKSPACE;
  int dev, sms;
  if ((st = check_device(&dev, &sms)) != K3MOE_OK) return st;
  QkvParams p = qkv_params(d, T);
  p.q = q; p.q_stride = q_stride; p.k = k; p.k_stride = k_stride; p.v = v; p.v_stride = v_stride;
  p.pos = positions; p.slots = slots; p.inv_freq = inv_freq; p.q_w = q_w; p.k_w = k_w;
  p.q_out = q_out; p.k_out = k_out;
  p.c = view_of(*cache);
  p.status = static_cast<uint32_t*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  K3A_TRY(cache->format == K3ATTN_E4M3 ? launch_norm<CF_E4M3>(p, sms, s) : launch_norm<CF_BF16>(p, sms, s));
  return K3MOE_OK;
}

k3moe_status k3attn_kv_read(const k3attn_dims* dims, int32_t T, const int32_t* slots, const k3attn_cache* cache,
                            uint16_t* k_out, uint16_t* v_out, void* ws, size_t ws_bytes, void* stream) {
  k3moe_status st = check_dims(dims);
  if (st != K3MOE_OK) return st;
  const k3attn_dims& d = *dims;
  if ((st = check_cache(cache, d)) != K3MOE_OK) return st;
  if (T < 0) return K3MOE_ERR_ARG;
  if (T == 0) return K3MOE_OK;
  if (!slots || !k_out || !v_out || !ws) return K3MOE_ERR_ARG;
  if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(ws, 16)) return K3MOE_ERR_ALIGN;
  if (ws_bytes < K3ATTN_MIN_WORKSPACE) return K3MOE_ERR_WORKSPACE;
  int dev, sms;
  if ((st = check_device(&dev, &sms)) != K3MOE_OK) return st;
  QkvParams p = qkv_params(d, T);
  p.slots = slots; p.k_out = k_out; p.v_out = v_out;
  p.c = view_of(*cache);
  p.status = static_cast<uint32_t*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  K3A_TRY((cache->format == K3ATTN_E4M3 ? launch_rows<CF_E4M3, false>(p, sms, s) : launch_rows<CF_BF16, false>(p, sms, s)));
  return K3MOE_OK;
}

k3moe_status k3attn_decode(const k3attn_dims* dims, int32_t B, const uint16_t* q, int64_t q_stride,
                           const k3attn_cache* cache, const int32_t* page_table, int32_t table_width,
                           const int32_t* lens, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                           void* stream) {
  k3moe_status st = check_dims(dims);
  if (st != K3MOE_OK) return st;
  const k3attn_dims& d = *dims;
  if ((st = check_cache(cache, d)) != K3MOE_OK) return st;
  if (B < 0 || table_width < 0) return K3MOE_ERR_ARG;
  if (B == 0) return K3MOE_OK;
  if (!q || (table_width > 0 && !page_table) || !lens || !out || !ws) return K3MOE_ERR_ARG;
  if (B > 65535 || (int64_t)table_width * cache->page_size > INT32_MAX) return K3MOE_ERR_SHAPE;
  if ((st = check_rows(q_stride, (int64_t)d.n_heads * d.head_dim)) != K3MOE_OK) return st;
  if (!aligned(q, 16) || !aligned(page_table, 4) || !aligned(lens, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(ws, 16))
    return K3MOE_ERR_ALIGN;
  if (ws_bytes < k3attn_workspace_bytes(dims)) return K3MOE_ERR_WORKSPACE;
  int dev, sms;
  if ((st = check_device(&dev, &sms)) != K3MOE_OK) return st;
  DecodeParams p{};
  p.q = q; p.q_stride = q_stride;
  p.B = B; p.Hq = d.n_heads; p.Hkv = d.n_kv_heads; p.G = d.n_heads / d.n_kv_heads; p.D = d.head_dim;
  p.window = d.window;
  p.scale = d.softmax_scale * 1.4426950408889634f;
  p.c = view_of(*cache);
  p.table = page_table; p.table_width = table_width; p.lens = lens;
  p.out = out; p.lse = lse;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.status = reinterpret_cast<uint32_t*>(w);
  p.arrived = reinterpret_cast<uint32_t*>(w + kCounters);
  p.parts = reinterpret_cast<float*>(w + kRecords);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int dp = dec_dp(d), nt = dec_nt_of(d, cache->format);
  K3A_TRY((cache->format == K3ATTN_E4M3 ? launch_decode<CF_E4M3>(p, dp, nt, dev, sms, s)
                                        : launch_decode<CF_BF16>(p, dp, nt, dev, sms, s)));
  return K3MOE_OK;
}

}  // extern "C"
