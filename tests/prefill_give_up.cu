// Launches of the prefill kernel in which one wait of one warp runs out at once, for a test of what
// the kernel does then.  Plain tensors: one table of pages, dense pages, window and sinks as given.
#include <cstdint>

__device__ unsigned give_block, give_warp, give_wait;  // which wait runs out: the warp's give_wait-th one (1, 2 ..)
__device__ unsigned given;                             // whether it came to that
__device__ unsigned waits[512];                        // of the block's threads, so far

// looks of the wait that a thread is about to begin
__device__ __forceinline__ uint32_t looks_of_wait() {
  if (blockIdx.x != give_block || threadIdx.x / 32 != give_warp) return 1u << 24;
  if (++waits[threadIdx.x] != give_wait) return 1u << 24;
  given = 1;
  return 0;
}
#define K3_MB_LOOKS looks_of_wait()

#include "../mxfp4_routed_expert_latentmoe_gb300/csrc/attn/k3_prefill.cuh"

namespace {
using namespace k3;
constexpr int D = 64;

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool map_rows(CUtensorMap* m, void* rows, int n_pages, int heads, int page) {
  void* f = nullptr;
  cudaDriverEntryPointQueryResult q{};
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess) return false;
  const cuuint64_t dims[4] = {D, (cuuint64_t)page, (cuuint64_t)heads, (cuuint64_t)n_pages};
  const cuuint64_t strides[3] = {2 * D, (cuuint64_t)page * 2 * D, (cuuint64_t)heads * page * 2 * D};
  const cuuint32_t box[4] = {64, 8, 1, 1}, each[4] = {1, 1, 1, 1};
  return reinterpret_cast<EncodeTiled>(f)(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, rows, dims, strides, box, each,
                                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT>
int run(const PrefillParams& p, const PrefillMaps& maps, int grid) {
  using C = PreCfg<FMT, D>;
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, k3_prefill_kernel<FMT, D>) != cudaSuccess || a.numRegs < PRE_REGS) return -1;  // (register split)
  if (cudaFuncSetAttribute(k3_prefill_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return -2;
  k3_prefill_kernel<FMT, D><<<grid, PRE_THREADS, C::SMEM>>>(maps, p);
  if (cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return -3;
  unsigned x = 0;
  return cudaMemcpyFromSymbol(&x, given, sizeof x) == cudaSuccess ? (int)x : -4;
}
}  // namespace

extern "C" {

// One call; 1: the wait ran out, 0: the warp has no such wait, below 0: an error.  bf16 (format 0) with boxes, or MXFP4 rows.
int give_up(int format, int block, int warp, int wait, int grid, int B, int T, int Hq, int Hkv, int window, int sinks, int n_pages,
            int page, int table_width, void* q, void* k, void* v, void* ks, void* vs, const int32_t* starts, const int32_t* table,
            const int32_t* lens, void* out, float* lse, uint32_t* status, uint32_t* arrived, float* parts) {
  const unsigned zero[512] = {}, which[3] = {(unsigned)block, (unsigned)warp, (unsigned)wait};
  if (cudaMemcpyToSymbol(waits, zero, sizeof zero) != cudaSuccess || cudaMemcpyToSymbol(given, zero, 4) != cudaSuccess ||
      cudaMemcpyToSymbol(give_block, which, 4) != cudaSuccess || cudaMemcpyToSymbol(give_warp, which + 1, 4) != cudaSuccess ||
      cudaMemcpyToSymbol(give_wait, which + 2, 4) != cudaSuccess)
    return -5;
  PrefillParams p{};
  PrefillMaps maps{};
  const int64_t row = format == CF_BF16 ? 2 * D : D / 2, scales = K3ATTN_MXFP4_SCALES(D);
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = Hq * D;
  p.B = B; p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.D = D; p.window = window; p.sinks = sinks;
  p.groups = 1;
  p.heads = p.G;
  p.tokens = 256 / p.G;
  p.scale = 0.125f * 1.4426950408889634f;
  p.c.k = static_cast<uint8_t*>(k);
  p.c.v = static_cast<uint8_t*>(v);
  p.c.ks = static_cast<float*>(ks);
  p.c.vs = static_cast<float*>(vs);
  p.c.tok = row; p.c.head = page * row; p.c.page = Hkv * page * row;
  p.c.stok = scales; p.c.shead = page * scales; p.c.spage = Hkv * page * scales;
  p.c.n_pages = n_pages;
  p.c.page_size = page;
  p.c.by_page = Divisor::of((uint32_t)page);
  p.starts = starts; p.table = table; p.table_width = table_width; p.lens = lens;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.status = status;
  p.arrived = arrived;
  p.parts = parts;
  if (format == CF_MXFP4) return run<CF_MXFP4>(p, maps, grid);
  if (!map_rows(&maps.k, k, n_pages, Hkv, page) || !map_rows(&maps.v, v, n_pages, Hkv, page)) return -6;
  p.boxes = 1;
  return run<CF_BF16>(p, maps, grid);
}

size_t parts_floats() { return (size_t)2 * PRE_MAX_BLOCKS * PreCfg<CF_BF16, D>::REC; }

}  // extern "C"
