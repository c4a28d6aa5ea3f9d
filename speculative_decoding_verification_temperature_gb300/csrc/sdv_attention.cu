// sdv_attention.cu -- sd_paged_attention: a chunk of new tokens attends
// over the paged cache.
#include "sdv_attention.cuh"

namespace sdv {
namespace {

// ------------------------------------------------------------------- host
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType,
                                 cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

sd_status encoder(EncodeTiled *out) {
  static std::atomic<EncodeTiled> known{nullptr};
  EncodeTiled f = known.load(std::memory_order_acquire);
  if (!f) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult res;
    SDV_CUDA(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn,
                                              12000, cudaEnableDefault, &res));
    if (!fn || res != cudaDriverEntryPointSuccess)
      return fail(SD_ERR_UNSUPPORTED, "the driver has no tensor maps");
    f = reinterpret_cast<EncodeTiled>(fn);
    known.store(f, std::memory_order_release);
  }
  *out = f;
  return SD_OK;
}

// The cache as (head_dim, token of a page, head, page), in boxes of 64
// columns (128 bytes) x `box` tokens, swizzled; what lies outside is zero.
sd_status cache_map(const sd_paged_kv *c, void *base, int box,
                    CUtensorMap *map) {
  EncodeTiled enc = nullptr;
  const sd_status st = encoder(&enc);
  if (st != SD_OK) return st;
  const cuuint64_t pages = c->num_pages > 0 ? c->num_pages : 1;
  const cuuint64_t dims[4] = {(cuuint64_t)c->head_dim,
                              (cuuint64_t)c->page_size,
                              (cuuint64_t)c->heads, pages};
  // a dimension of one element has no stride of its own
  const cuuint64_t any = (cuuint64_t)c->head_dim * 2;
  const cuuint64_t strides[3] = {
      (cuuint64_t)c->token_stride * 2,
      c->heads > 1 ? (cuuint64_t)c->head_stride * 2 : any,
      pages > 1 ? (cuuint64_t)c->page_stride * 2 : any};
  const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUresult r = enc(
      map,
      c->dt == SD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
      4, base, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(SD_ERR_INVALID_ARG,
                "no tensor map for the cache's strides (%lld, %lld, %lld)",
                c->page_stride, c->token_stride, c->head_stride);
  return SD_OK;
}

// With up to 128 rows a weight is two numbers.
template <class T>
sd_status dispatch(AttnParams &p, int D, bool pair, const CUtensorMap &km,
                   const CUtensorMap &vm, int sms, char *ws, cudaStream_t s) {
  if (D == 64)
    return pair ? launch<T, 64, true, false, false>(p, km, vm, sms, ws, s)
                : launch<T, 64, false, false, true>(p, km, vm, sms, ws, s);
  return pair ? launch<T, 128, true, false, false>(p, km, vm, sms, ws, s)
              : launch<T, 128, false, false, true>(p, km, vm, sms, ws, s);
}

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_paged_attention_workspace(int q_heads, int heads,
                                               int head_dim, int max_q) {
  if (heads < 1 || q_heads < heads || (head_dim != 64 && head_dim != 128))
    return 256;
  return ws_layout(kMaxGrid, pair_rows(max_q, q_heads / heads) ? 256 : 128,
                   head_dim)
      .bytes;
}

extern "C" sd_status sd_paged_attention(
    const void *q, long long q_stride, int q_heads, const sd_paged_kv *cache,
    const int32_t *q_start, const int32_t *kv_len, const int32_t *tree_mask,
    int mask_words, int B, int total, int max_q, float scale, void *out,
    float *lse, int32_t *dev_status, void *workspace, size_t ws_bytes,
    void *stream) {
  sd_status st = check_cache(cache);
  if (st != SD_OK) return st;
  const int D = cache->head_dim;
  SDV_REQUIRE(B >= 0 && total >= 0, "B < 0 or total < 0");
  SDV_REQUIRE(max_q >= 0, "max_q < 0");
  SDV_REQUIRE(q_heads >= 1 && q_heads <= 65535 &&
                  q_heads % cache->heads == 0,
              "q_heads=%d is not a multiple of the cache's %d heads", q_heads,
              cache->heads);
  SDV_REQUIRE(scale > 0.f && std::isfinite(scale * 1.5f),
              "scale must be > 0, and scale log2(e) finite");
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
  SDV_REQUIRE(aligned16(q) && q_stride % 8 == 0,
              "q must be 16-byte aligned, q_stride a multiple of 8");
  SDV_REQUIRE((reinterpret_cast<uintptr_t>(out) & 31) == 0,
              "out must be 32-byte aligned");
  SDV_REQUIRE(aligned16(cache->k) && aligned16(cache->v) &&
                  cache->page_stride % 8 == 0 &&
                  cache->token_stride % 8 == 0 && cache->head_stride % 8 == 0,
              "the cache must be 16-byte aligned, its strides multiples of 8");
  SDV_REQUIRE((long long)total * q_heads < (1LL << 31) - 256,
              "total x q_heads does not fit 31 bits");
  const size_t need = sd_paged_attention_workspace(q_heads, cache->heads, D,
                                                   max_q);
  SDV_REQUIRE(workspace && ws_bytes >= need &&
                  (reinterpret_cast<uintptr_t>(workspace) & 31) == 0,
              "a 32-byte aligned workspace of >= %zu bytes required", need);
  int sms = 0;
  st = check_device(&sms);
  if (st != SD_OK) return st;
  AttnParams p;
  p.q = q;
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
  p.G = q_heads / cache->heads;
  p.by_G = fast_div(p.G);
  p.by_page = fast_div(cache->page_size);
  for (p.box = 8; p.box < kTile && cache->page_size % (2 * p.box) == 0;)
    p.box *= 2;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.out = out;
  p.lse = lse;
  p.dev_status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CUtensorMap k_map, v_map;
  st = cache_map(cache, cache->k, p.box, &k_map);
  if (st == SD_OK) st = cache_map(cache, cache->v, p.box, &v_map);
  if (st != SD_OK) return st;
  const bool pair = pair_rows(max_q, p.G);
  char *ws = static_cast<char *>(workspace);
  return cache->dt == SD_BF16
             ? dispatch<__nv_bfloat16>(p, D, pair, k_map, v_map, sms, ws, s)
             : dispatch<__half>(p, D, pair, k_map, v_map, sms, ws, s);
}
