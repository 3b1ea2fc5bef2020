// k3_tmem.cuh -- what the attention of many tokens uses of mbarriers, tensor memory and tcgen05.mma.
// (The expert GEMMs' wrappers stand beside their kernels, which belong to another translation unit.)
#pragma once

#include <cuda.h>

#include "../k3_common.cuh"

namespace k3 {

K3_DEVI void mb_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
K3_DEVI void mb_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory"); }
K3_DEVI void mb_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// bytes that boxes are going to bring to the phase
K3_DEVI void mb_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
// a box of a tensor of four dimensions
K3_DEVI void tma_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
K3_DEVI bool mb_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// whether the phase is through, without waiting
K3_DEVI bool mb_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase of the given parity; false if the block has given up, or after MB_LOOKS looks of
// some 7800 clocks each, about a minute (then it has).  The longest that a block's warps wait for one
// another is for rows that are formed again: 0.5 to 3 s for a tile over half a million tokens (64 to 256 dims).
constexpr uint32_t MB_LOOKS = 1u << 24;
#ifndef K3_MB_LOOKS  // (a test lets chosen waits run out at once)
#define K3_MB_LOOKS MB_LOOKS
#endif
K3_DEVI bool mb_wait(uint32_t bar, uint32_t parity, volatile int* gave_up, uint32_t looks = K3_MB_LOOKS) {
#pragma unroll 1
  for (uint32_t n = 1; n < looks; ++n) {
    if (mb_try(bar, parity)) return true;
    if ((n & 255) == 0 && *gave_up) return false;
  }
  *gave_up = 1;
  return false;
}

K3_DEVI void tm_alloc(uint32_t dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
K3_DEVI void tm_free(uint32_t tmem, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(columns) : "memory");
}
K3_DEVI void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
K3_DEVI void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
// shared-memory writes of the generic proxy before reads of the tensor core
K3_DEVI void fence_smem_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
// one lane of a warp whose lanes are all here
K3_DEVI bool elect_one() {
  uint32_t is;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(is));
  return is != 0;
}
K3_DEVI void tm_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
// D (+)= A B^T of 16 contraction steps: A in shared, and in tensor memory
K3_DEVI void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, uint32_t add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(kind), "r"(add)
      : "memory");
}
K3_DEVI void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, uint32_t add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(kind), "r"(add)
      : "memory");
}
// operands of bf16, sums of fp32, M x N; b_across: B's rows (of 64 elements) run along N
K3_HD constexpr uint32_t mma_kind(int M, int N, bool b_across) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_across ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Matrices in shared memory in blocks of 64 columns: rows of 128 bytes whose 16-byte pieces are
// permuted by the row's number modulo 8 (the 128-byte swizzle), 8 rows 1024 bytes.  Contraction along
// the columns: 16 of them are 32 bytes further.  Along the rows (b_across): 16 of them are 2048 bytes
// further, and the blocks of columns lie `block` bytes apart.
K3_DEVI uint64_t rows_desc(uint32_t addr, uint32_t block = 16) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(block >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
#define K3_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define K3_U4(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3])
#define K3_W4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
// a lane's 32 or 16 columns of its row
K3_DEVI void tm_ld32(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : K3_R4(r, 0), K3_R4(r, 4), K3_R4(r, 8), K3_R4(r, 12), K3_R4(r, 16), K3_R4(r, 20), K3_R4(r, 24), K3_R4(r, 28)
      : "r"(a)
      : "memory");
}
K3_DEVI void tm_ld16(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      : K3_R4(r, 0), K3_R4(r, 4), K3_R4(r, 8), K3_R4(r, 12)
      : "r"(a)
      : "memory");
}
// waits for the loads before it; N registers that they fill (nothing of theirs may be used in front of
// the wait, which the compiler sees by the registers alone)
template <int N>
K3_DEVI void tm_ld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i += 16)
    asm volatile("" : K3_U4(r, i), K3_U4(r, i + 4), K3_U4(r, i + 8), K3_U4(r, i + 12));
}
K3_DEVI void tm_st16(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};\n" ::"r"(a),
      K3_W4(r, 0), K3_W4(r, 4), K3_W4(r, 8), K3_W4(r, 12)
      : "memory");
}
K3_DEVI void tm_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// keeps a store's registers until its wait (the compiler does not know that it still reads them)
K3_DEVI void tm_keep16(const uint32_t* r) {
  asm volatile("" ::K3_W4(r, 0), K3_W4(r, 4), K3_W4(r, 8), K3_W4(r, 12));
}
#undef K3_R4
#undef K3_U4
#undef K3_W4

template <int N>
K3_DEVI void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
K3_DEVI void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

}  // namespace k3
