// sdv_attention.cu -- sd_paged_attention: a chunk of new tokens attends
// over the paged cache.
//
//   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j)
//
// in one pass over the keys with a running maximum m and sum l: a new
// maximum m' scales what is summed so far by exp(m - m').
#include "sdv_paged.cuh"

namespace sdv {
namespace {

struct AttnParams {
  const void *q, *k, *v;
  long long q_stride;
  const int32_t *q_start, *kv_len, *block_table, *mask;
  int mask_words;
  int B, total, Hq, Hkv;
  int num_pages, page_size, max_pages;
  long long page_stride, token_stride, head_stride;
  float scale_log2;  // scale x log2(e)
  void *out;
  float *lse;
  int32_t *dev_status;
};

// One warp per (token, query head); a lane holds D / 32 elements.
template <class T, int D>
__global__ void __launch_bounds__(kThreads)
attention_row_kernel(const __grid_constant__ AttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w =
      (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w >= (long long)p.total * p.Hq) return;
  const int row = (int)(w / p.Hq), h = (int)(w % p.Hq);
  const int b = find_sequence(p.q_start, p.B, row);
  Chunk c = load_chunk(p.q_start, p.kv_len, b, p.total,
                       (long long)p.max_pages * p.page_size);
  if (c.usable && p.mask && c.n > 32 * p.mask_words) c.usable = false;
  if (!c.usable && lane == 0) status_or(p.dev_status, SD_DEV_BAD_LENGTH);
  if (!c.rows_ok || row < c.start || row >= c.start + c.n) return;
  T *out = (T *)p.out + ((long long)row * p.Hq + h) * D;
  float *lse = p.lse ? p.lse + (long long)row * p.Hq + h : nullptr;
  const float nan = __int_as_float(0x7fc00000);
  const int i = row - c.start, ctx = c.kv - c.n;
  const T *q = (const T *)p.q + row * p.q_stride + (long long)h * D;
  const int kh = h / (p.Hq / p.Hkv);
  float qv[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = widen(q[lane + 32 * e]);
    o[e] = 0.f;
  }
  float m = -kInf, l = 0.f;
  bool bad = !c.usable;
  const int last = bad ? 0 : p.mask ? c.kv : ctx + i + 1;
  for (int j = 0; j < last; ++j) {
    const int page = __ldg(p.block_table + (long long)b * p.max_pages +
                           j / p.page_size);
    if (page < 0 || page >= p.num_pages) {
      bad = true;
      if (lane == 0) status_or(p.dev_status, SD_DEV_BAD_PAGE);
      break;
    }
    if (p.mask && j >= ctx) {
      const int x = j - ctx;
      const int32_t word =
          __ldg(p.mask + (long long)row * p.mask_words + (x >> 5));
      if (!((word >> (x & 31)) & 1)) continue;
    }
    const long long at = page * p.page_stride +
                         (j % p.page_size) * p.token_stride +
                         kh * p.head_stride;
    const T *k = (const T *)p.k + at, *v = (const T *)p.v + at;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qv[e], widen(k[lane + 32 * e]), s);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float f = m == -kInf ? 0.f : ex2(m - mn);
    const float wgt = ex2(s - mn);
    m = mn;
    l = l * f + wgt;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = fmaf(o[e], f, wgt * widen(v[lane + 32 * e]));
  }
  const float inv = bad ? nan : l > 0.f ? 1.f / l : l != l ? l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    out[lane + 32 * e] = narrow<T>(bad ? nan : o[e] * inv);
  if (lse && lane == 0)
    *lse = bad ? nan : l == 0.f ? -kInf : (m + log2f(l)) * 0.69314718f;
}

template <class T>
sd_status launch(const AttnParams &p, int D, cudaStream_t s) {
  const long long blocks = ((long long)p.total * p.Hq + kWarps - 1) / kWarps;
  SDV_REQUIRE(blocks < (1LL << 31), "too many rows");
  if (D == 64)
    attention_row_kernel<T, 64><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  else
    attention_row_kernel<T, 128><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  SDV_CUDA(cudaGetLastError());
  return SD_OK;
}

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_paged_attention_workspace(int q_heads, int heads,
                                               int head_dim, int max_q) {
  (void)q_heads;
  (void)heads;
  (void)head_dim;
  (void)max_q;
  return 0;
}

extern "C" sd_status sd_paged_attention(
    const void *q, long long q_stride, int q_heads, const sd_paged_kv *cache,
    const int32_t *q_start, const int32_t *kv_len, const int32_t *tree_mask,
    int mask_words, int B, int total, int max_q, float scale, void *out,
    float *lse, int32_t *dev_status, void *workspace, size_t ws_bytes,
    void *stream) {
  (void)workspace;
  (void)ws_bytes;
  sd_status st = check_cache(cache);
  if (st != SD_OK) return st;
  const int D = cache->head_dim;
  SDV_REQUIRE(B >= 0 && total >= 0, "B < 0 or total < 0");
  SDV_REQUIRE(max_q >= 0, "max_q < 0");
  SDV_REQUIRE(q_heads >= 1 && q_heads <= 65535 &&
                  q_heads % cache->heads == 0,
              "q_heads=%d is not a multiple of the cache's %d heads", q_heads,
              cache->heads);
  SDV_REQUIRE(scale > 0.f && std::isfinite(scale),
              "scale must be finite and > 0");
  SDV_REQUIRE(!tree_mask || mask_words >= 1, "mask_words < 1");
  if (D != 64 && D != 128)
    return fail(SD_ERR_UNSUPPORTED, "head_dim=%d is neither 64 nor 128", D);
  if (B == 0 || total == 0) return SD_OK;
  SDV_REQUIRE(q && cache->k && cache->v && q_start && kv_len && out,
              "null pointer");
  SDV_REQUIRE(cache->max_pages == 0 || cache->block_table,
              "block_table is null");
  SDV_REQUIRE(q_stride >= (long long)q_heads * D,
              "tokens overlap: q_stride is below q_heads x head_dim");
  SDV_REQUIRE(aligned16(q) && q_stride % 8 == 0 && aligned16(out),
              "q and out must be 16-byte aligned, q_stride a multiple of 8");
  SDV_REQUIRE(aligned16(cache->k) && aligned16(cache->v) &&
                  cache->page_stride % 8 == 0 &&
                  cache->token_stride % 8 == 0 && cache->head_stride % 8 == 0,
              "the cache must be 16-byte aligned, its strides multiples of 8");
  int sms = 0;
  st = check_device(&sms);
  if (st != SD_OK) return st;
  AttnParams p;
  p.q = q;
  p.k = cache->k;
  p.v = cache->v;
  p.q_stride = q_stride;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.block_table = cache->block_table;
  p.mask = tree_mask;
  p.mask_words = mask_words;
  p.B = B;
  p.total = total;
  p.Hq = q_heads;
  p.Hkv = cache->heads;
  p.num_pages = cache->num_pages;
  p.page_size = cache->page_size;
  p.max_pages = cache->max_pages;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.out = out;
  p.lse = lse;
  p.dev_status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->dt == SD_BF16 ? launch<__nv_bfloat16>(p, D, s)
                              : launch<__half>(p, D, s);
}
