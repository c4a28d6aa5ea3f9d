// sdv_kv4_append.cu -- sd_kv4_append: new tokens' keys and values quantised
// to 4 bits as they go into the paged cache, keys and queries rotated by
// position on the way; sd_kv4_read: tokens of the cache back as 16-bit rows.
//
// With lo and hi the least and greatest of a group's values,
//   a = fp16((hi - lo) / 15), b = fp16(lo - 64 a),
//   n = rint((x - b) / a) - 64, kept inside 0 .. 15,
// values x first brought inside -6144 .. 6144, and each step rounded to fp32 by
// itself (no contraction), 1 / 15 and 1 / a being rounded first: the codes are
// the same numbers wherever they are computed.
//
// Where rows are many, what they wait for is HBM: 28k tokens of 48 heads of
// 128, fp16, neighbours turned, are 611 MB in 133 us, 0.69 of the measured copy
// rate, with 0.6 of the issue slots; of 12.2 warps at an issue 6.4 wait for a
// load, and registers are all taken.  Halves turned take 186 us (a second load
// a piece, which the registers do not hold: 112 bytes of spills, and 8.5 of
// 14.4 warps wait), none turned 164; rows that are not whole 16-byte pieces
// 302.  99k tokens of 8 heads are read back, 0.52 GB, in 87 us, 0.89.  Where
// rows are few it is the chain sequence -> page -> store.
#include "sdv_kv4.cuh"

namespace sdv {
namespace {

struct Append4Params {
  const void *k, *v, *q;
  long long k_stride, v_stride, q_stride;
  const int32_t *q_start, *kv_len, *positions, *block_table;
  const float *cos_sin;
  int max_pos, rot, warps;
  int B, total, Hq, Hkv;
  int page_size, max_pages;
  FastDiv by_page;
  Kv4Cache c;
  bool angles_wide;  // cos_sin can be read 16 bytes at a time
  void *q_out;
  int32_t *dev_status;
};

// Where one packed row goes: its page (negative: nowhere), token in the page
// and row of the angles; st: the status bits it sets; owned: it belongs to a
// sequence.
struct Place {
  int page, token, pos, st;
  bool owned;
};

template <class P>
__device__ __forceinline__ Place place_row(const P &p, int row) {
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
  r.pos = c.kv - c.n + (row - c.start);
  const int n = div_by(r.pos, p.by_page);
  const int page = __ldg(p.block_table + (long long)b * p.max_pages + n);
  if (page < 0 || page >= p.c.num_pages) r.st = SD_DEV_BAD_PAGE;
  else r.page = page;
  r.token = r.pos - n * p.page_size;
  return r;
}

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

// min and max that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  return __fmul2_rn(a, b);
}

// Codes of eight neighbours, one word, and their group's pair; `lanes`
// neighbouring lanes hold a group.  The whole warp calls.
__device__ __forceinline__ uint32_t quantise8(const float2 (&x)[4], int lanes,
                                              uint32_t &pair) {
  float lo = min_nan(x[0].x, x[0].y, x[1].x), hi = max_nan(x[0].x, x[0].y,
                                                           x[1].x);
  lo = min_nan(lo, x[1].y, x[2].x), hi = max_nan(hi, x[1].y, x[2].x);
  lo = min_nan(lo, x[2].y, x[3].x), hi = max_nan(hi, x[2].y, x[3].x);
  lo = min_nan(lo, x[3].y, x[3].y), hi = max_nan(hi, x[3].y, x[3].y);
  for (int d = 1; d < lanes; d <<= 1) {
    const float a = __shfl_xor_sync(~0u, lo, d);
    const float b = __shfl_xor_sync(~0u, hi, d);
    lo = min_nan(lo, a, a);
    hi = max_nan(hi, b, b);
  }
  if (!(lo > -kInf && hi < kInf)) {  // a group that holds NaN or infinity
    pair = 0x7e007e00u;
    return 0;
  }
  lo = fminf(fmaxf(lo, -kKv4Most), kKv4Most);
  hi = fminf(fmaxf(hi, -kKv4Most), kKv4Most);
  const __half a = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f));
  const float af = __half2float(a);
  const __half b = __float2half_rn(__fsub_rn(lo, 64.f * af));
  const float bf = __half2float(b);
  const float inv = af > 0.f ? __frcp_rn(af) : 0.f;
  // 1.5 x 2^23 + t is t rounded to a whole number, in the low bits: added up
  // with their shifts, what lies above the codes is a constant modulo 2^32
  const float2 minus_b = make_float2(-bf, -bf), inv2 = make_float2(inv, inv);
  const float2 magic = make_float2(12582912.f, 12582912.f);
  // Numbers beyond lo and hi count as these: every step here keeps the order,
  // so their places are the limits, two a group for two operations a number.
  auto place = [&](float y) {
    return fminf(fmaxf(__fmul_rn(__fadd_rn(y, -bf), inv), 64.f), 79.f);
  };
  const float least = place(lo), most = place(hi);
  uint32_t w = 0u - (0x4b400000u + 64) * 0x11111111u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 t = mul2(add2(x[e], minus_b), inv2);
    t.x = fminf(fmaxf(t.x, least), most);
    t.y = fminf(fmaxf(t.y, least), most);
    t = add2(t, magic);
    w += __float_as_uint(t.x) << 4 * e;
    w += __float_as_uint(t.y) << 4 * (e + 4);
  }
  pair = (uint32_t)__half_as_ushort(b) << 16 | __half_as_ushort(a);
  return w;
}

// Eight neighbours of a head, and the elements they are turned with.
struct Piece {
  uint4 own, other;
};

// p.warps warps per packed row (one where there are many rows, up to eight
// where there are few); a thread takes eight neighbours of every step-th head,
// so that it reads its cosines and sines once.  Queries first, which are only
// turned, then keys and values, kBatch heads at a time; the first ones are on
// their way before the row's place is looked for.  WIDE: rot_dim is a multiple
// of 16 and rows are 16-byte aligned, so that pieces are whole 16-byte loads
// and turn as a whole; otherwise elements are loaded one by one.  (A CTA a row
// looked up the row's place and read its angles in each of eight warps: 208 us
// on the 28k tokens, and 133 with a warp a row.)  Four CTAs an SM: with three,
// where no instance of whole pieces spills, neighbours take 143 us, halves 195
// and rows without a turn 179; with two 143, 259 and 238.
constexpr int kBatch = 4;
template <class T, int D, bool WIDE, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads, 4)
append4_kernel(const __grid_constant__ Append4Params p) {
  griddep_wait();
  constexpr int PER = D / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kWarps / p.warps) + warp / p.warps;
  if (row >= p.total) return;  // the whole warp
  const int at = warp % p.warps * 32 + lane;
  const int i = lane % PER, first = at / PER, step = p.warps * 32 / PER;
  const int half = p.rot / 2;
  // element (or piece's first element) e is turned with other(e)
  auto other = [&](int e) {
    return NEIGHBOURS ? e ^ 1 : e < half ? e + half : e - half;
  };
  const bool turns = 8 * i < p.rot;
  auto load = [&](const T *src, bool turned) {
    Piece x;
    if (WIDE) {
      x.own = ld_nc_v4(src + 8 * i);
      x.other = x.own;
      if (turned && !NEIGHBOURS) x.other = ld_nc_v4(src + other(8 * i));
    } else {
      alignas(16) T own[8], oth[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int n = 8 * i + e;
        own[e] = src[n];
        oth[e] = turned && n < p.rot ? src[other(n)] : own[e];
      }
      x.own = *reinterpret_cast<const uint4 *>(own);
      x.other = *reinterpret_cast<const uint4 *>(oth);
    }
    return x;
  };
  const T *q_row = (const T *)p.q + row * p.q_stride;
  const T *k_row = (const T *)p.k + row * p.k_stride;
  const T *v_row = (const T *)p.v + row * p.v_stride;
  Piece x[kBatch];
  auto load_q = [&](int h0) {
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int h = h0 + n * step + first;
      if (h < p.Hq) x[n] = load(q_row + h * D, turns);
    }
  };
  auto load_kv = [&](int h0) {  // keys, then values
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int h = h0 + n * step + first;
      if (h < 2 * p.Hkv)
        x[n] = load(h < p.Hkv ? k_row + h * D : v_row + (h - p.Hkv) * D,
                    turns && h < p.Hkv);
    }
  };
  if (p.Hq > 0) load_q(0);
  else load_kv(0);
  Place pl = place_row(p, row);
  if (pl.st == 0 && pl.owned && p.cos_sin) {
    if (p.positions) pl.pos = __ldg(p.positions + row);
    if (pl.pos < 0 || pl.pos >= p.max_pos) {
      pl.st = SD_DEV_BAD_POSITION;
      pl.page = -1;
    }
  }
  if (at == 0) status_or(p.dev_status, pl.st);
  if (!pl.owned) return;
  // x' = x c + x_other s: the sine of the first of a pair is negative
  float2 c[4], s[4];
  const float *cs = p.cos_sin + (long long)pl.pos * p.rot;
  if (WIDE && turns && pl.page >= 0 && p.angles_wide) {
    const bool head = 8 * i < half;
    const int angle = NEIGHBOURS ? 4 * i : head ? 8 * i : 8 * i - half;
    float4 a = __ldg(reinterpret_cast<const float4 *>(cs + angle));
    float4 b = __ldg(reinterpret_cast<const float4 *>(cs + half + angle));
    if (NEIGHBOURS) {
      c[0] = make_float2(a.x, a.x), s[0] = make_float2(-b.x, b.x);
      c[1] = make_float2(a.y, a.y), s[1] = make_float2(-b.y, b.y);
      c[2] = make_float2(a.z, a.z), s[2] = make_float2(-b.z, b.z);
      c[3] = make_float2(a.w, a.w), s[3] = make_float2(-b.w, b.w);
    } else {
      const float4 u =
          __ldg(reinterpret_cast<const float4 *>(cs + angle + 4));
      const float4 v =
          __ldg(reinterpret_cast<const float4 *>(cs + half + angle + 4));
      const float k = head ? -1.f : 1.f;
      c[0] = make_float2(a.x, a.y), s[0] = make_float2(k * b.x, k * b.y);
      c[1] = make_float2(a.z, a.w), s[1] = make_float2(k * b.z, k * b.w);
      c[2] = make_float2(u.x, u.y), s[2] = make_float2(k * v.x, k * v.y);
      c[3] = make_float2(u.z, u.w), s[3] = make_float2(k * v.z, k * v.w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = 8 * i + e;
      float u = 1.f, v = 0.f;
      if (n < p.rot && pl.page >= 0) {
        const bool head = NEIGHBOURS ? !(n & 1) : n < half;
        const int angle = NEIGHBOURS ? n / 2 : head ? n : n - half;
        u = __ldg(cs + angle);
        v = head ? -__ldg(cs + half + angle) : __ldg(cs + half + angle);
      }
      if (e & 1) c[e / 2].y = u, s[e / 2].y = v;
      else c[e / 2].x = u, s[e / 2].x = v;
    }
  }
  // Products and sums are rounded one by one: packed ones would be fused.
  auto turn = [&](const Piece &in, bool turned, float2 (&y)[4]) {
    const uint32_t own[4] = {in.own.x, in.own.y, in.own.z, in.own.w};
    const uint32_t oth[4] = {in.other.x, in.other.y, in.other.z, in.other.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = unpack2<T>(own[e]);
      if (!turned) continue;
      const float2 v = WIDE && NEIGHBOURS ? make_float2(y[e].y, y[e].x)
                                          : unpack2<T>(oth[e]);
      const float2 z =
          make_float2(__fadd_rn(__fmul_rn(y[e].x, c[e].x),
                                __fmul_rn(v.x, s[e].x)),
                      __fadd_rn(__fmul_rn(y[e].y, c[e].y),
                                __fmul_rn(v.y, s[e].y)));
      // (an odd piece may end its turn in the middle)
      if (WIDE || 8 * i + 2 * e < p.rot) y[e].x = z.x;
      if (WIDE || 8 * i + 2 * e + 1 < p.rot) y[e].y = z.y;
    }
  };
  T *q_to = (T *)p.q_out + (long long)row * p.Hq * D + 8 * i;
  for (int h0 = 0; h0 < p.Hq; h0 += kBatch * step) {
    if (h0) load_q(h0);
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int h = h0 + n * step + first;
      if (h >= p.Hq) break;
      uint4 w = x[n].own;  // where nothing turns it is copied
      if (turns) {
        float2 y[4];
        turn(x[n], true, y);
        w = make_uint4(pack2<T>(y[0]), pack2<T>(y[1]), pack2<T>(y[2]),
                       pack2<T>(y[3]));
      }
      if (pl.page < 0) w = make_uint4(0, 0, 0, 0);
      T *to = q_to + h * D;
      if (WIDE) {
        *reinterpret_cast<uint4 *>(to) = w;
      } else {
        const T *y = reinterpret_cast<const T *>(&w);
#pragma unroll
        for (int e = 0; e < 8; ++e) to[e] = y[e];
      }
    }
  }
  if (pl.page < 0) return;  // the whole warp
  const int lanes = 1 << (p.c.shift - 3);
  const long long page_c = pl.page * p.c.page_stride + 4 * i;
  const long long page_s =
      pl.page * p.c.scale_stride + 4 * (8 * i >> p.c.shift);
  // every lane makes the same rounds
  for (int h0 = 0; h0 < 2 * p.Hkv; h0 += kBatch * step) {
    if (h0 || p.Hq > 0) load_kv(h0);
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      if (h0 + n * step >= 2 * p.Hkv) break;
      const int h = h0 + n * step + first;
      const bool is_k = h < p.Hkv;
      float2 y[4];
      turn(x[n], turns && is_k, y);
      uint32_t pair;
      const uint32_t word = quantise8(y, lanes, pair);  // the whole warp
      if (h >= 2 * p.Hkv) continue;
      const int slot = (is_k ? h : h - p.Hkv) * p.page_size + pl.token;
      char *codes = const_cast<char *>(is_k ? p.c.k : p.c.v);
      char *pairs = const_cast<char *>(is_k ? p.c.k_scale : p.c.v_scale);
      *reinterpret_cast<uint32_t *>(codes + page_c +
                                    (long long)slot * (D / 2)) = word;
      if ((i & (lanes - 1)) == 0)
        *reinterpret_cast<uint32_t *>(
            pairs + page_s + (long long)slot * p.c.scale_bytes) = pair;
    }
  }
}

struct Read4Params {
  const int32_t *q_start, *kv_len, *block_table;
  int B, total, Hkv, page_size, max_pages;
  FastDiv by_page;
  Kv4Cache c;
  void *k_out, *v_out;
  long long k_stride, v_stride;
  int32_t *dev_status;
};

// A warp per packed row, a lane for 16 elements of every (512 / D)-th head:
// eight bytes of codes, the pair, and 32 bytes written.
constexpr int kReadAhead = 4;
template <class T, int D>
__global__ void __launch_bounds__(kThreads)
read4_kernel(const __grid_constant__ Read4Params p) {
  griddep_wait();
  constexpr int PER = D / 16, STEP = 32 / PER;
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.total) return;  // the whole warp
  const int lane = threadIdx.x & 31, i = lane % PER, first = lane / PER;
  const Place pl = place_row(p, row);
  if (lane == 0) status_or(p.dev_status, pl.st);
  if (!pl.owned) return;
  const int group = 16 * i >> p.c.shift;
  for (int h0 = 0; h0 < 2 * p.Hkv; h0 += kReadAhead * STEP) {
    uint2 w[kReadAhead];
    uint32_t pair[kReadAhead];
#pragma unroll
    for (int n = 0; n < kReadAhead; ++n) {
      const int h = h0 + n * STEP + first;
      w[n] = make_uint2(0, 0);
      pair[n] = 0x7e007e00u;  // NaN
      if (h < 2 * p.Hkv && pl.page >= 0) {
        const bool is_k = h < p.Hkv;
        const long long at =
            (long long)(is_k ? h : h - p.Hkv) * p.page_size + pl.token;
        w[n] = __ldg(reinterpret_cast<const uint2 *>(
            (is_k ? p.c.k : p.c.v) + pl.page * p.c.page_stride +
            at * (D / 2) + 8 * i));
        pair[n] = __ldg(reinterpret_cast<const uint32_t *>(
            (is_k ? p.c.k_scale : p.c.v_scale) +
            pl.page * p.c.scale_stride + at * p.c.scale_bytes + 4 * group));
      }
    }
#pragma unroll
    for (int n = 0; n < kReadAhead; ++n) {
      const int h = h0 + n * STEP + first;
      if (h >= 2 * p.Hkv) continue;
      const bool is_k = h < p.Hkv;
      T *to = is_k ? (T *)p.k_out + row * p.k_stride + (long long)h * D
                   : (T *)p.v_out + row * p.v_stride +
                         (long long)(h - p.Hkv) * D;
      const uint32_t a = both_lo(pair[n]), b = both_hi(pair[n]);
      const uint32_t words[2] = {w[n].x, w[n].y};
      uint32_t y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = kv4_fma(kv4_codes(words[e / 4], e % 4), a, b);
        if (!std::is_same<T, __half>::value)
          y[e] = pack2<T>(unpack2<__half>(y[e]));
      }
      asm volatile(
          "st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
              to + 16 * i),
          "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]),
          "r"(y[6]), "r"(y[7])
          : "memory");
    }
  }
}

template <class T, int D>
const void *append_of(bool wide, bool neighbours) {
  if (neighbours)
    return wide ? (const void *)append4_kernel<T, D, true, true>
                : (const void *)append4_kernel<T, D, false, true>;
  return wide ? (const void *)append4_kernel<T, D, true, false>
              : (const void *)append4_kernel<T, D, false, false>;
}

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" sd_status sd_kv4_append(
    const sd_paged_kv4 *cache, const void *k, long long k_stride,
    const void *v, long long v_stride, const void *q, long long q_stride,
    int q_heads, const int32_t *q_start, const int32_t *kv_len,
    const int32_t *positions, const float *cos_sin, int max_pos, int rot_dim,
    int interleaved, int B, int total, void *q_out, int32_t *dev_status,
    void *stream) {
  sd_status st = check_kv4(cache);
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
  SDV_REQUIRE(k && v && cache->k && cache->v && cache->k_scale &&
                  cache->v_scale && q_start && kv_len,
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
  Append4Params p;
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
  p.B = B;
  p.total = total;
  p.Hq = Hq;
  p.Hkv = cache->heads;
  p.page_size = cache->page_size;
  p.by_page = fast_div(cache->page_size);
  p.max_pages = cache->max_pages;
  p.c = kv4_cache(cache);
  p.angles_wide = aligned16(cos_sin);
  p.q_out = q_out;
  p.dev_status = dev_status;
  const bool wide = p.rot % 16 == 0 && aligned16(k) && aligned16(v) &&
                    aligned16(q) && aligned16(q_out) &&
                    (k_stride | v_stride | (q ? q_stride : 0)) % 8 == 0;
  const bool bf = cache->dt == SD_BF16;
  const bool nb = interleaved != 0;
  const void *kernel =
      D == 64 ? (bf ? append_of<__nv_bfloat16, 64>(wide, nb)
                    : append_of<__half, 64>(wide, nb))
              : (bf ? append_of<__nv_bfloat16, 128>(wide, nb)
                    : append_of<__half, 128>(wide, nb));
  // as many warps a row as find a place (32 an SM are resident at a time), but
  // no more than it has work for: 1216 tokens, halves turned, take 10.8 us with
  // four warps a row, 14.5 with two and 12.9 with eight
  const long long most = Hq > 2 * cache->heads ? Hq : 2 * cache->heads;
  p.warps = 1;
  while (p.warps < kWarps && (long long)total * p.warps < 32 * sms &&
         p.warps * 32 < most * (D / 8))
    p.warps *= 2;
  const unsigned rows = kWarps / p.warps;
  void *args[] = {&p};
  return launch_pdl(kernel, (unsigned)((total + rows - 1LL) / rows), kThreads,
                    0, static_cast<cudaStream_t>(stream), args);
}

extern "C" sd_status sd_kv4_read(const sd_paged_kv4 *cache,
                                 const int32_t *q_start,
                                 const int32_t *kv_len, int B, int total,
                                 void *k_out, long long k_stride, void *v_out,
                                 long long v_stride, int32_t *dev_status,
                                 void *stream) {
  sd_status st = check_kv4(cache);
  if (st != SD_OK) return st;
  const int D = cache->head_dim;
  SDV_REQUIRE(B >= 0 && total >= 0, "B < 0 or total < 0");
  if (B == 0 || total == 0) return SD_OK;
  SDV_REQUIRE(cache->k && cache->v && cache->k_scale && cache->v_scale &&
                  q_start && kv_len && k_out && v_out,
              "null pointer");
  SDV_REQUIRE(cache->max_pages == 0 || cache->block_table,
              "block_table is null");
  SDV_REQUIRE(k_stride >= (long long)cache->heads * D &&
                  v_stride >= (long long)cache->heads * D,
              "tokens overlap: a stride is below heads x head_dim");
  SDV_REQUIRE((reinterpret_cast<uintptr_t>(k_out) & 31) == 0 &&
                  (reinterpret_cast<uintptr_t>(v_out) & 31) == 0 &&
                  k_stride % 16 == 0 && v_stride % 16 == 0,
              "k_out and v_out must be 32-byte aligned, their strides "
              "multiples of 16");
  int sms = 0;
  st = check_device(&sms);
  if (st != SD_OK) return st;
  Read4Params p;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.block_table = cache->block_table;
  p.B = B;
  p.total = total;
  p.Hkv = cache->heads;
  p.page_size = cache->page_size;
  p.by_page = fast_div(cache->page_size);
  p.max_pages = cache->max_pages;
  p.c = kv4_cache(cache);
  p.k_out = k_out;
  p.v_out = v_out;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.dev_status = dev_status;
  const bool bf = cache->dt == SD_BF16;
  const void *kernel =
      D == 64 ? (bf ? (const void *)read4_kernel<__nv_bfloat16, 64>
                    : (const void *)read4_kernel<__half, 64>)
              : (bf ? (const void *)read4_kernel<__nv_bfloat16, 128>
                    : (const void *)read4_kernel<__half, 128>);
  void *args[] = {&p};
  return launch_pdl(kernel, (unsigned)((total + kWarps - 1LL) / kWarps),
                    kThreads, 0, static_cast<cudaStream_t>(stream), args);
}
