// sdv_append.cu -- sd_kv_append: new tokens' keys and values into the paged
// cache, keys and queries rotated by position on the way.
//
// Pair i of a head is a point of the plane turned by the angle of its
// position: (x c - y s, x s + y c).  Values, and elements past rot_dim, are
// copied.
#include "sdv_paged.cuh"

namespace sdv {
namespace {

struct AppendParams {
  const void *k, *v, *q;
  long long k_stride, v_stride, q_stride;
  const int32_t *q_start, *kv_len, *positions, *block_table;
  const float *cos_sin;
  int max_pos, rot, interleaved;
  int B, total, Hq, Hkv, D;
  int num_pages, page_size, max_pages;
  long long page_stride, token_stride, head_stride;
  void *k_cache, *v_cache, *q_out;
  int32_t *dev_status;
};

// Where one packed row goes: in the cache (page >= 0) and in the table of
// angles; st: the status bits it sets; owned: it belongs to a sequence.
struct Place {
  int page, token, pos, st;
  bool owned;
};

__device__ __forceinline__ Place place_row(const AppendParams &p, int row) {
  Place r{-1, 0, 0, 0, false};
  const int b = find_sequence(p.q_start, p.B, row);
  const Chunk c = load_chunk(p.q_start, p.kv_len, b, p.total,
                             (long long)p.max_pages * p.page_size);
  if (!c.rows_ok) {
    r.st = SD_DEV_BAD_LENGTH;
    return r;
  }
  if (row < c.start || row >= c.start + c.n) return r;
  r.owned = true;
  if (!c.usable) {
    r.st = SD_DEV_BAD_LENGTH;
    return r;
  }
  const int idx = c.kv - c.n + (row - c.start);
  r.pos = p.positions ? __ldg(p.positions + row) : idx;
  if (p.cos_sin && (r.pos < 0 || r.pos >= p.max_pos))
    r.st |= SD_DEV_BAD_POSITION;
  const int page =
      __ldg(p.block_table + (long long)b * p.max_pages + idx / p.page_size);
  if (page < 0 || page >= p.num_pages) r.st |= SD_DEV_BAD_PAGE;
  if (r.st == 0) {
    r.page = page;
    r.token = idx % p.page_size;
  }
  return r;
}

// One CTA per packed row, one thread per pair.
template <class T>
__global__ void __launch_bounds__(kThreads)
append_kernel(const __grid_constant__ AppendParams p) {
  const int row = blockIdx.x;
  const Place pl = place_row(p, row);
  if (threadIdx.x == 0) status_or(p.dev_status, pl.st);
  if (!pl.owned) return;
  const int half = p.D / 2 + (p.D & 1), pairs = p.rot / 2;
  const float *cs = p.cos_sin ? p.cos_sin + (long long)pl.pos * p.rot : nullptr;
  const int heads = p.Hq + 2 * p.Hkv;
  for (int it = threadIdx.x; it < heads * half; it += blockDim.x) {
    const int h = it / half, i = it % half;
    const T *src;
    T *dst;
    bool turn = cs != nullptr;
    if (h < p.Hq) {
      src = (const T *)p.q + row * p.q_stride + (long long)h * p.D;
      dst = (T *)p.q_out + ((long long)row * p.Hq + h) * p.D;
    } else {
      const bool is_k = h < p.Hq + p.Hkv;
      const int kh = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
      if (pl.page < 0) continue;
      turn = turn && is_k;
      src = is_k ? (const T *)p.k + row * p.k_stride + (long long)kh * p.D
                 : (const T *)p.v + row * p.v_stride + (long long)kh * p.D;
      dst = (T *)(is_k ? p.k_cache : p.v_cache) + pl.page * p.page_stride +
            pl.token * p.token_stride + kh * p.head_stride;
    }
    if (pl.page < 0) {
      for (int e = 2 * i; e < 2 * i + 2 && e < p.D; ++e)
        dst[e] = narrow<T>(0.f);
      continue;
    }
    if (turn && i < pairs) {
      const int a = p.interleaved ? 2 * i : i;
      const int b = p.interleaved ? 2 * i + 1 : i + pairs;
      const float x = widen(src[a]), y = widen(src[b]);
      const float c = cs[i], s = cs[pairs + i];
      dst[a] = narrow<T>(x * c - y * s);
      dst[b] = narrow<T>(x * s + y * c);
    } else {
      // the copied elements, two a thread: past rot_dim, or all of them
      for (int e = 2 * i; e < 2 * i + 2 && e < p.D; ++e) dst[e] = src[e];
    }
  }
}

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" sd_status sd_kv_append(
    const sd_paged_kv *cache, const void *k, long long k_stride,
    const void *v, long long v_stride, const void *q, long long q_stride,
    int q_heads, const int32_t *q_start, const int32_t *kv_len,
    const int32_t *positions, const float *cos_sin, int max_pos, int rot_dim,
    int interleaved, int B, int total, void *q_out, int32_t *dev_status,
    void *stream) {
  sd_status st = check_cache(cache);
  if (st != SD_OK) return st;
  SDV_REQUIRE(B >= 0 && total >= 0, "B < 0 or total < 0");
  SDV_REQUIRE(q_heads >= 0 && q_heads <= 65535,
              "q_heads=%d outside [0, 65535]", q_heads);
  SDV_REQUIRE((q == nullptr) == (q_out == nullptr),
              "q and q_out go together");
  const int Hq = q ? q_heads : 0;
  const int D = cache->head_dim;
  if (cos_sin) {
    SDV_REQUIRE(rot_dim >= 2 && rot_dim <= D && rot_dim % 2 == 0,
                "rot_dim=%d is not even and in [2, %d]", rot_dim, D);
    SDV_REQUIRE(max_pos >= 1, "max_pos < 1");
  }
  if (B == 0 || total == 0) return SD_OK;
  SDV_REQUIRE(k && v && cache->k && cache->v && q_start && kv_len,
              "null pointer");
  SDV_REQUIRE(cache->max_pages == 0 || cache->block_table,
              "block_table is null");
  SDV_REQUIRE(k_stride >= (long long)cache->heads * D &&
                  v_stride >= (long long)cache->heads * D &&
                  (!q || q_stride >= (long long)Hq * D),
              "tokens overlap: a stride is below heads x head_dim");
  int sms = 0;
  st = check_device(&sms);
  if (st != SD_OK) return st;
  AppendParams p;
  p.k = k;
  p.v = v;
  p.q = q;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.positions = positions;
  p.block_table = cache->block_table;
  p.cos_sin = cos_sin;
  p.max_pos = max_pos;
  p.rot = cos_sin ? rot_dim : 0;
  p.interleaved = interleaved;
  p.B = B;
  p.total = total;
  p.Hq = Hq;
  p.Hkv = cache->heads;
  p.D = D;
  p.num_pages = cache->num_pages;
  p.page_size = cache->page_size;
  p.max_pages = cache->max_pages;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  p.k_cache = cache->k;
  p.v_cache = cache->v;
  p.q_out = q_out;
  p.dev_status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->dt == SD_BF16)
    append_kernel<__nv_bfloat16><<<total, kThreads, 0, s>>>(p);
  else
    append_kernel<__half><<<total, kThreads, 0, s>>>(p);
  SDV_CUDA(cudaGetLastError());
  return SD_OK;
}
