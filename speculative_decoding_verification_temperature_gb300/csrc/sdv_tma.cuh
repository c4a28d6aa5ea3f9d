// sdv_tma.cuh -- bulk asynchronous copies (TMA, cp.async.bulk) from global
// to shared memory with mbarrier completion, written as inline PTX.
//
// Each wait is bounded: after kWaitLimit polls it gives up, reports
// SD_DEV_TIMEOUT through the status word and returns false, so a kernel
// never spins forever.  The caller keeps its barrier protocol intact (the
// data it then computes on is meaningless, and the host sees the bit).
#pragma once

#include <cstdint>

#include "sdv_device.cuh"

namespace sdv {

#ifndef SDV_SUSPEND
#define SDV_SUSPEND 0
#endif
constexpr unsigned kWaitLimit = 1u << 26;  // polls: seconds of waiting
constexpr unsigned kSuspendNs = 1000;      // suspend hint per poll

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint64_t *bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)),
               "r"(count)
               : "memory");
}

// Make the barrier initialisation visible to the async proxy.
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Order earlier generic-proxy accesses of shared memory before later
// async-proxy (TMA) writes to it.
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile(
      "mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
          smem_addr(bar)),
      "r"(bytes)
      : "memory");
}

// Bulk copy of `bytes` (multiple of 16, both addresses 16-byte aligned)
// from global to this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_g2s(void *dst, const void *src,
                                         uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// An L2 policy that marks the lines it loads first to be evicted: for data
// read once, so that it does not push out lines another phase re-reads.
__device__ __forceinline__ uint64_t l2_evict_first_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;"
               : "=l"(pol));
  return pol;
}

// bulk_g2s with an L2 cache policy for the lines it reads.
__device__ __forceinline__ void bulk_g2s_hint(void *dst, const void *src,
                                              uint32_t bytes, uint64_t *bar,
                                              uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(pol)
      : "memory");
}

// Hint: bring `bytes` (multiple of 16, 16-byte aligned) into L2.
__device__ __forceinline__ void prefetch_l2(const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src),
               "r"(bytes)
               : "memory");
}

// One poll; the thread may be suspended (up to kSuspendNs) until the
// phase completes, so a waiting warp issues almost nothing.
__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
#if SDV_SUSPEND
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(kSuspendNs)
      : "memory");
#else
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
#endif
  return ok != 0;
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// Wait for phase `parity` of the barrier to complete; bounded: after
// `limit` polls it sets SD_DEV_TIMEOUT and returns false.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity,
                                          int32_t *dev_status,
                                          unsigned limit = kWaitLimit) {
  for (unsigned it = 0; it < limit; ++it)
    if (mbar_try_wait(bar, parity)) return true;
  status_or(dev_status, SD_DEV_TIMEOUT);
  return false;
}

// The same with a limit for one CTA: after a failure anywhere in it every
// wait gives up at once (`abort` in its shared memory), so that all roles of
// a warp-specialised kernel leave their loops.
constexpr unsigned kRoleWaitLimit = 1u << 22;
__device__ __forceinline__ bool role_wait(uint64_t *bar, uint32_t parity,
                                          volatile int *abort,
                                          int32_t *dev_status) {
  for (unsigned it = 0; it < kRoleWaitLimit; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255) == 255 && *abort) return false;
  }
  *abort = 1;
  status_or(dev_status, SD_DEV_TIMEOUT);
  return false;
}

// A position in a ring of n slots: the slot, and the parity of its filling.
struct RingAt {
  int slot, n;
  uint32_t parity;
  __device__ RingAt(int n_) : slot(0), n(n_), parity(0) {}
  __device__ void next() {
    if (++slot == n) slot = 0, parity ^= 1;
  }
};

// Store two words to the same place in CTA `rank` of the cluster and count
// their eight bytes on its barrier there.
__device__ __forceinline__ void st_async_pair(void *here, uint64_t *bar,
                                              int rank, float a, float b) {
  uint32_t to, tb;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(to)
      : "r"(smem_addr(here)), "r"(rank));
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(tb)
      : "r"(smem_addr(bar)), "r"(rank));
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], "
      "{%1, %2}, [%3];" ::"r"(to),
      "f"(a), "f"(b), "r"(tb)
      : "memory");
}

}  // namespace sdv
