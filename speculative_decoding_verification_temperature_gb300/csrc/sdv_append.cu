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
  FastDiv by_half;  // D / 2 rounded up, or the double chunks of a head
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
  const int b = warp_find_sequence(p.q_start, p.B, row);
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

// Any size and alignment: one CTA per packed row, one thread per pair.  For
// rotations and head sizes off the grid of 16 that models seldom have: loads
// and stores by the element, angles read for every head (25k tokens of 48
// heads of 96, rot_dim 20 or 24: 264 us, at HBM's rate 79).
template <class T>
__global__ void __launch_bounds__(kThreads)
append_any_kernel(const __grid_constant__ AppendParams p) {
  griddep_wait();
  const int row = blockIdx.x;
  const Place pl = place_row(p, row);
  if (threadIdx.x == 0) status_or(p.dev_status, pl.st);
  if (!pl.owned) return;
  const int half = p.D / 2 + (p.D & 1), pairs = p.rot / 2;
  const float *cs = p.cos_sin ? p.cos_sin + (long long)pl.pos * p.rot : nullptr;
  const int heads = p.Hq + 2 * p.Hkv;
  for (int it = threadIdx.x; it < heads * half; it += blockDim.x) {
    const int h = div_by(it, p.by_half), i = it - h * half;
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

// 16 elements, as two chunks of 16 bytes.
struct Double {
  uint4 a, b;
};

template <class T> __device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16),
                     __uint_as_float(u & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<__half2 *>(&u));
}
template <class T> __device__ __forceinline__ uint32_t pack2(float2 x);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 x) {
  const __nv_bfloat162 v = __float22bfloat162_rn(x);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float2 x) {
  const __half2 v = __float22half2_rn(x);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Turn the eight pairs of a double: (a_i, b_i), or neighbours of a then b.
template <class T, bool NEIGHBOURS>
__device__ __forceinline__ Double turn(Double x, const float (&c)[8],
                                       const float (&s)[8]) {
  uint32_t a[4] = {x.a.x, x.a.y, x.a.z, x.a.w};
  uint32_t b[4] = {x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<T>(a[i]), v = unpack2<T>(b[i]);
    if (NEIGHBOURS) {
      a[i] = pack2<T>(make_float2(u.x * c[i] - u.y * s[i],
                                  u.x * s[i] + u.y * c[i]));
      b[i] = pack2<T>(make_float2(v.x * c[i + 4] - v.y * s[i + 4],
                                  v.x * s[i + 4] + v.y * c[i + 4]));
    } else {
      a[i] = pack2<T>(make_float2(u.x * c[2 * i] - v.x * s[2 * i],
                                  u.y * c[2 * i + 1] - v.y * s[2 * i + 1]));
      b[i] = pack2<T>(make_float2(u.x * s[2 * i] + v.x * c[2 * i],
                                  u.y * s[2 * i + 1] + v.y * c[2 * i + 1]));
    }
  }
  return {make_uint4(a[0], a[1], a[2], a[3]),
          make_uint4(b[0], b[1], b[2], b[3])};
}

// Heads whose parts are whole double chunks (D and rot_dim multiples of 16,
// 16-byte aligned rows): a CTA per packed row, as many threads as its doubles
// need up to 256, a thread for one double of every (threads / doubles)-th
// head, so that it reads its eight cosines and sines once.  Bound by HBM
// where there are many rows (each byte is read and written once) and by the
// chain sequence -> page -> store where there are few; a thread's first
// kAhead heads are on their way before it starts on that chain.  25k tokens of
// 48 heads of 128, fp16: 700 MB in 120 us, 0.88 of the measured copy rate; one
// token 2.1 us, 288 tokens 3.7 us.
constexpr int kAhead = 3;
template <class T, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads)
append_kernel(const __grid_constant__ AppendParams p) {
  griddep_wait();
  const int row = blockIdx.x, per = p.D / 16;
  const int first = div_by(threadIdx.x, p.by_half);
  const int i = threadIdx.x - first * per;
  const int step = blockDim.x / per, heads = p.Hq + 2 * p.Hkv;
  const bool works = first < step;
  const bool turns = i * 16 < p.rot;
  // the double's chunks in a head: apart where pairs are, else neighbours
  const int a = turns && !NEIGHBOURS ? i * 8 : i * 16;
  const int b = turns && !NEIGHBOURS ? i * 8 + p.rot / 2 : i * 16 + 8;
  auto load = [&](int h) {
    const T *src;
    if (h < p.Hq)
      src = (const T *)p.q + row * p.q_stride + h * p.D;
    else if (h < p.Hq + p.Hkv)
      src = (const T *)p.k + row * p.k_stride + (h - p.Hq) * p.D;
    else
      src = (const T *)p.v + row * p.v_stride + (h - p.Hq - p.Hkv) * p.D;
    const bool pairs = turns && h < p.Hq + p.Hkv;
    return Double{ld_nc_v4(src + (pairs ? a : i * 16)),
                  ld_nc_v4(src + (pairs ? b : i * 16 + 8))};
  };
  Double x[kAhead];
#pragma unroll
  for (int n = 0; n < kAhead; ++n)
    if (works && first + n * step < heads) x[n] = load(first + n * step);
  const Place pl = place_row(p, row);
  if (threadIdx.x == 0) status_or(p.dev_status, pl.st);
  if (!pl.owned || !works) return;
  float c[8], s[8];
  if (turns && pl.page >= 0) {
    const float4 *cs = reinterpret_cast<const float4 *>(
        p.cos_sin + (long long)pl.pos * p.rot + i * 8);
    const float4 *sn = reinterpret_cast<const float4 *>(
        p.cos_sin + (long long)pl.pos * p.rot + p.rot / 2 + i * 8);
    const float4 u = __ldg(cs), v = __ldg(cs + 1);
    const float4 y = __ldg(sn), z = __ldg(sn + 1);
    c[0] = u.x, c[1] = u.y, c[2] = u.z, c[3] = u.w;
    c[4] = v.x, c[5] = v.y, c[6] = v.z, c[7] = v.w;
    s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
    s[4] = z.x, s[5] = z.y, s[6] = z.z, s[7] = z.w;
  }
  const long long at =
      pl.page * p.page_stride + pl.token * p.token_stride;
  auto put = [&](int h, Double d) {
    T *dst;
    if (h < p.Hq) {
      dst = (T *)p.q_out + ((long long)row * p.Hq + h) * p.D;
      if (pl.page < 0) d.a = d.b = make_uint4(0, 0, 0, 0);
    } else {
      if (pl.page < 0) return;
      const bool is_k = h < p.Hq + p.Hkv;
      dst = (T *)(is_k ? p.k_cache : p.v_cache) + at +
            (h - p.Hq - (is_k ? 0 : p.Hkv)) * p.head_stride;
    }
    const bool pairs = turns && h < p.Hq + p.Hkv;
    if (pairs && pl.page >= 0) d = turn<T, NEIGHBOURS>(d, c, s);
    *reinterpret_cast<uint4 *>(dst + (pairs ? a : i * 16)) = d.a;
    *reinterpret_cast<uint4 *>(dst + (pairs ? b : i * 16 + 8)) = d.b;
  };
#pragma unroll
  for (int n = 0; n < kAhead; ++n)
    if (first + n * step < heads) put(first + n * step, x[n]);
  for (int h = first + kAhead * step; h < heads; h += step) put(h, load(h));
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
  const bool wide =
      D % 16 == 0 && p.rot % 16 == 0 && D / 16 <= kThreads && aligned16(k) &&
      aligned16(v) && aligned16(q) && aligned16(q_out) &&
      aligned16(cache->k) && aligned16(cache->v) && aligned16(cos_sin) &&
      (k_stride | v_stride | q_stride | cache->page_stride |
       cache->token_stride | cache->head_stride) % 8 == 0;
  const bool bf = cache->dt == SD_BF16;
  const void *kernel;
  int threads = kThreads;
  if (wide) {
    // few or small heads in small CTAs: 11k tokens of 6 heads of 64 take
    // 9.4 us, with 256 threads a row 38.8
    const long long all = (Hq + 2LL * cache->heads) * (D / 16);
    if (all < kThreads) threads = (int)(all + 31) / 32 * 32;
    p.by_half = fast_div(D / 16);
    kernel = interleaved
                 ? (bf ? (const void *)append_kernel<__nv_bfloat16, true>
                       : (const void *)append_kernel<__half, true>)
                 : (bf ? (const void *)append_kernel<__nv_bfloat16, false>
                       : (const void *)append_kernel<__half, false>);
  } else {
    p.by_half = fast_div((D + 1) / 2);
    kernel = bf ? (const void *)append_any_kernel<__nv_bfloat16>
                : (const void *)append_any_kernel<__half>;
  }
  void *args[] = {&p};
  return launch_pdl(kernel, (unsigned)total, threads, 0,
                    static_cast<cudaStream_t>(stream), args);
}
