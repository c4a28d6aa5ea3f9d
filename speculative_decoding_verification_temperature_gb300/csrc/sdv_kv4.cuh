// sdv_kv4.cuh -- the 4-bit cache: what its codes stand for, and the host's
// checks of a description.
//
// A group's pair (a, b) of fp16 numbers makes its code n the fp16 number
// nearest to b + (64 + n) a.  fp16 numbers from 64 on lie 2^-4 apart, so a
// code's four bits at bits 4 to 7 of 0x5400 are the number 64 + n: a pair of
// values is one logic operation and one fma of fp16 pairs, with a single
// rounding, on every path that reads the cache.  (With b + n a the 64 would
// cost a subtraction a pair: half as much again.)  b is coarser for it: fp16
// numbers at lo - 64 a lie up to a sixteenth of a step apart in groups about
// zero, and 2^-10 of the offset in those far from it; the codes are chosen by
// the b that is kept.  Values beyond kMost count as that, so that b, 64 steps
// below a group, stays inside fp16.
//
// A word of codes holds eight neighbours, elements 0, 2, 4, 6, 1, 3, 5, 7
// from its lowest nibble on: a mask then finds neighbours (2 j, 2 j + 1).
#pragma once

#include "sdv_paged.cuh"

namespace sdv {

constexpr float kKv4Most = 6144.f;

// Codes j and j + 4 of a word, which stand for elements 2 j and 2 j + 1, as
// the fp16 pair (64 + n, 64 + n').  Those at bits 0 to 3 of a half are made
// 1024 + n and 960 subtracted (exactly): a shift less for the pipe of integers
// and logic, which is the fuller one, and an addition more for the other.
__device__ __forceinline__ uint32_t kv4_codes(uint32_t w, int j) {
  const uint32_t x = j < 2 ? w : w >> 8;
  uint32_t y;  // x & mask | magic, one operation
  if (j & 1) {
    asm("lop3.b32 %0, %1, %2, %3, 0xea;"
        : "=r"(y)
        : "r"(x), "r"(0x00f000f0u), "r"(0x54005400u));
  } else {
    asm("lop3.b32 %0, %1, %2, %3, 0xea;"
        : "=r"(y)
        : "r"(x), "r"(0x000f000fu), "r"(0x64006400u));
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(y) : "r"(0xe380e380u));  // -960
  }
  return y;
}
__device__ __forceinline__ uint32_t kv4_fma(uint32_t x, uint32_t a,
                                            uint32_t b) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(a), "r"(b));
  return y;
}
// One number of a pair in both halves.
__device__ __forceinline__ uint32_t both_lo(uint32_t x) {
  return __byte_perm(x, x, 0x1010);
}
__device__ __forceinline__ uint32_t both_hi(uint32_t x) {
  return __byte_perm(x, x, 0x3232);
}

// 16 bytes from global to shared memory, asynchronously, if `there`.
__device__ __forceinline__ void cp16(uint32_t to, const void *from,
                                     bool there) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(to),
      "l"(from), "r"((int)there)
      : "memory");
}
// Arrive on `bar` when the copies that this thread has begun are complete.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}
__device__ __forceinline__ void cp_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared memory by its own addresses.
__device__ __forceinline__ uint32_t lds_word(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ void lds_pair(uint32_t at, uint32_t *x) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
               : "=r"(x[0]), "=r"(x[1])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void sts_v4(uint32_t at, uint4 x) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x),
               "r"(x.y), "r"(x.z), "r"(x.w)
               : "memory");
}
// A thread's share of a key's row: N words of shared memory.
template <int N>
__device__ __forceinline__ void lds_words(const char *p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

// Where the codes and the pairs of a cache lie: in bytes, pages `stride`
// apart, inside a page [heads][page_size] rows.
struct Kv4Cache {
  const char *k, *v, *k_scale, *v_scale;
  long long page_stride, scale_stride;
  int num_pages, scale_bytes;
  int shift;  // log2 of the group
};

inline sd_status check_kv4(const sd_paged_kv4 *c) {
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
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(SD_ERR_UNSUPPORTED, "head_dim=%d is neither 64 nor 128",
                c->head_dim);
  SDV_REQUIRE((c->group == 32 || c->group == 64 || c->group == 128) &&
                  c->group <= c->head_dim,
              "group=%d is not 32, 64 or 128, or above head_dim=%d", c->group,
              c->head_dim);
  if (c->page_size % 8 != 0)
    return fail(SD_ERR_UNSUPPORTED, "page_size=%d is not a multiple of 8",
                c->page_size);
  const long long rows = (long long)c->heads * c->page_size;
  SDV_REQUIRE(rows < (1LL << 31) - 256,
              "heads page_size = %lld does not fit 31 bits", rows);
  SDV_REQUIRE(c->num_pages <= 1 ||
                  (c->page_stride >= rows * (c->head_dim / 2) &&
                   c->scale_stride >= rows * (c->head_dim / c->group) * 4),
              "pages overlap: a stride is below a page's bytes");
  SDV_REQUIRE(c->page_stride >= 0 && c->scale_stride >= 0 &&
                  c->page_stride % 16 == 0 && c->scale_stride % 16 == 0,
              "page strides must be multiples of 16 bytes");
  SDV_REQUIRE(aligned16(c->k) && aligned16(c->v) && aligned16(c->k_scale) &&
                  aligned16(c->v_scale),
              "codes and scales must be 16-byte aligned");
  return SD_OK;
}

inline Kv4Cache kv4_cache(const sd_paged_kv4 *c) {
  Kv4Cache r;
  r.k = static_cast<const char *>(c->k);
  r.v = static_cast<const char *>(c->v);
  r.k_scale = static_cast<const char *>(c->k_scale);
  r.v_scale = static_cast<const char *>(c->v_scale);
  r.page_stride = c->page_stride;
  r.scale_stride = c->scale_stride;
  r.num_pages = c->num_pages;
  r.scale_bytes = c->head_dim / c->group * 4;
  r.shift = c->group == 32 ? 5 : c->group == 64 ? 6 : 7;
  return r;
}

}  // namespace sdv
