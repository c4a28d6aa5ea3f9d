// sdv_tcgen05.cuh -- the fifth-generation tensor cores of sm_103a in inline
// PTX: tensor memory, tcgen05.mma with 16-bit operands and fp32 sums, the
// descriptors it takes, and tiled TMA loads.
//
// Tensor memory is 128 lanes x 512 columns of 32 bits per SM; an address is
// lane << 16 | column.  Warp w of a warpgroup reads and writes lanes
// 32 (w % 4) .. + 31, one lane a thread, so a thread holds one row of an
// accumulator.
#pragma once

#include <cuda.h>

#include "sdv_tma.cuh"

namespace sdv {

// Allocate all 512 columns (one warp; blocks until they are free) and write
// their address to shared memory; give them back.
__device__ __forceinline__ void tmem_alloc_all(uint32_t *dst) {
  asm volatile(
      "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::
          "r"(smem_addr(dst))
      : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_all(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(
      addr));
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Order tcgen05 work of this thread before / after a synchronisation with
// other threads.
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

#define SDV_O8(r, i)                                                     \
  "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]),            \
      "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define SDV_I8(r, i)                                                     \
  "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
      "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this thread's lane, starting at `addr` (complete after
// tmem_wait_ld / tmem_wait_st).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, "
      "%7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
      "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SDV_O8(r, 0), SDV_O8(r, 8), SDV_O8(r, 16), SDV_O8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, "
      "%6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::
          "r"(addr),
      SDV_I8(r, 0), SDV_I8(r, 8), SDV_I8(r, 16), SDV_I8(r, 24)
      : "memory");
}

// Shared-memory matrix descriptor of a tile of 128-byte rows in the
// 128-byte swizzle (16-byte chunk c of row r lies at chunk c ^ (r & 7)).
// Low word: address, and lead_bytes, the distance between 64-element column
// blocks where the operand runs along its rows (MN-major; unused where it
// runs along the reduction, K-major).  High word: the distance between
// groups of eight rows, the version and the swizzle.  Moving along the tile
// adds bytes / 16 to the low word.
__device__ __forceinline__ uint32_t umma_desc_lo(const void *tile,
                                                 uint32_t lead_bytes) {
  return (smem_addr(tile) & 0x3ffff) >> 4 | (lead_bytes >> 4) << 16;
}
__host__ __device__ constexpr uint32_t umma_desc_hi(uint32_t group_bytes) {
  return group_bytes >> 4 | 1u << 14 | 2u << 29;
}

// One lane of the (converged) warp, always the same one.  The products are
// issued in a branch on this: 64 cycles apart at N = 128, the tensor cores'
// own rate; in a branch on the lane number they took 125, under a predicate
// 66 and more.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// Instruction descriptor: fp32 sums, both operands bf16 or fp16, A with the
// reduction contiguous, B as said; M x N.
__host__ __device__ constexpr uint32_t umma_idesc(bool bf16, bool b_mn_major,
                                                  int m, int n) {
  return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 |
         (b_mn_major ? 1u : 0u) << 16 | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(m >> 4) << 24;
}

// One step of 16 along the reduction: D (+)= A B, A in shared memory or in
// tensor memory (two elements a column).  One thread issues; products run in
// the order issued.
template <uint32_t HI>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo,
                                        uint32_t b_lo, uint32_t idesc,
                                        bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)add), "n"(HI)
      : "memory");
}
template <uint32_t HI>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo,
                                        uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(
          d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"((uint32_t)add), "n"(HI)
      : "memory");
}
// Arrive on `bar` when every tcgen05.mma this thread issued is complete.
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
      "[%0];" ::"r"(smem_addr(bar))
      : "memory");
}

// A box of a rank-4 tensor map, from coordinates x (elements; x times the
// element size is a multiple of 16 bytes), y, z, w, to shared memory.
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map,
                                            int x, int y, int z, int w,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

}  // namespace sdv
