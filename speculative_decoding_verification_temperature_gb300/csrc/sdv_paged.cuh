// sdv_paged.cuh -- what the paged-cache kernels share: 16-bit element
// types, the sequence a packed row belongs to, and the host's checks of a
// cache description.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sdv_device.cuh"
#include "sdv_host.cuh"

namespace sdv {

// fp32 <-> the cache's 16-bit types (round to nearest even).
__device__ __forceinline__ float widen(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <class T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ __nv_bfloat16 narrow(float x) {
  return __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ __half narrow(float x) {
  return __float2half_rn(x);
}

// A sequence's chunk: n new tokens from packed row `start`, the last n of
// its kv keys.  usable: see sd_paged_kv; rows_ok: start and n are.
struct Chunk {
  int start, n, kv;
  bool rows_ok, usable;
};

__device__ __forceinline__ Chunk load_chunk(const int32_t *q_start,
                                            const int32_t *kv_len, int b,
                                            int total, long long max_kv) {
  Chunk c;
  c.start = __ldg(q_start + b);
  const int end = __ldg(q_start + b + 1);
  c.kv = __ldg(kv_len + b);
  c.rows_ok = c.start >= 0 && c.start <= end && end <= total;
  c.n = c.rows_ok ? end - c.start : 0;
  c.usable = c.rows_ok && c.n <= c.kv && c.kv <= max_kv;
  return c;
}

// The last sequence whose q_start is at most `row` (the row's own, where it
// has one: empty sequences before it share its q_start).  The whole warp
// looks, a 32nd of the range a lane.
__device__ __forceinline__ int warp_find_sequence(const int32_t *q_start,
                                                  int B, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const unsigned below =
        __ballot_sync(~0u, lane * step < n && __ldg(q_start + at) <= row);
    const int last = below ? 31 - __clz(below) : 0;
    n = min(step, n - last * step);
    lo += last * step;
  }
  return lo;
}

// Division of 0 <= x < 2^31 by a fixed d >= 1 as a multiplication (Granlund
// and Montgomery, "Division by invariant integers using multiplication",
// 1994): with l = ceil(log2 d) and mul = floor(2^32 (2^l - d) / d) + 1 the
// quotient is (hi(mul x) + x) >> l.
struct FastDiv {
  uint32_t mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f = {0, 0};
  while (f.shift < 31 && (1u << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
  return f;
}
__device__ __forceinline__ int div_by(int x, FastDiv f) {
  return (int)((__umulhi((uint32_t)x, f.mul) + (uint32_t)x) >> f.shift);
}

// Host checks of a cache description.
inline sd_status check_cache(const sd_paged_kv *c) {
  SDV_REQUIRE(c != nullptr, "cache is null");
  SDV_REQUIRE(c->dt == SD_BF16 || c->dt == SD_F16, "bad cache dtype %d",
              (int)c->dt);
  SDV_REQUIRE(c->num_pages >= 0, "num_pages < 0");
  SDV_REQUIRE(c->page_size >= 1, "page_size < 1");
  SDV_REQUIRE(c->max_pages >= 0, "max_pages < 0");
  SDV_REQUIRE((long long)c->max_pages * c->page_size < (1LL << 31) - 256,
              "max_pages page_size = %lld does not fit 31 bits",
              (long long)c->max_pages * c->page_size);
  SDV_REQUIRE(c->heads >= 1 && c->heads <= 65535, "heads=%d outside [1, 65535]",
              c->heads);
  SDV_REQUIRE(c->head_dim >= 1 && c->head_dim <= 1024,
              "head_dim=%d outside [1, 1024]", c->head_dim);
  SDV_REQUIRE(c->page_stride >= 0 && c->token_stride >= 0 &&
                  c->head_stride >= 0,
              "a cache stride is negative");
  if (c->page_size % 8 != 0)
    return fail(SD_ERR_UNSUPPORTED, "page_size=%d is not a multiple of 8",
                c->page_size);
  return SD_OK;
}

}  // namespace sdv
