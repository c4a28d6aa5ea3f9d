// sdv_attention.cuh -- the tensor-core kernel of chunk attention over a paged
// cache of 16-bit or 4-bit keys and values.
//
//   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j)
//
// in one pass over the keys with a running reference m and sum l: a new
// reference m' scales what is summed so far by exp(m - m').
//
// A row is one (token, query head); the rows of a sequence that read one
// cache head are token-major, so the G query heads of a group share each key
// tile.  A unit of work is (sequence, cache head, 128 or 256 rows), its
// length the tiles of 128 keys its rows see.  All units laid end to end are
// cut into equal shares, one per SM, whatever the lengths are; a unit that
// is cut leaves partial sums in the workspace, which a second kernel joins
// in key order.
//
// In a CTA, two warps load key and value tiles by TMA through the block
// table, two issue the tensor-core products, and two warpgroups ("streams")
// turn scores into weights, a thread per row.  S = Q K^T goes to tensor
// memory; the weights, as 16-bit numbers (the tensor cores take two operands
// of one type), go back there over S and are the first operand of O += W V.
// With 256 rows each stream has 128 of them; with up to 128 rows (a few
// drafts) both have the same rows and every other key tile, and their sums
// are joined at the end of the unit.
//
// With up to 128 rows a weight is the sum of two 16-bit numbers and O takes a
// product of each (with one the tensor pipe is busy a third of the time, with
// two 41 to 48 %), so that the result is off by little more than its own
// rounding (fp16's range has its limits: see Scale).
// Weights rounded once were 0.0022 to 0.0026 off in bf16, by the inputs, where
// that rounding is 0.0017 (a few heavy keys of a few rows decide it); 9 tokens
// over 131072 keys took 94 us so and take 96, 64 sequences of one token 220
// and 229, 32 of nine 133 and 141.  With 256 rows, where the products are what
// it waits for, weights are rounded once (0.0023).
//
// The plain loop over keys with a warp per (token, head) took 14 ms on 64
// sequences of one token and 219 ms on two prompt chunks; this takes 230 us
// and 561 us.
//
// What bounds it: HBM for a few rows a unit (1.41 GB of keys and values of 64
// sequences in 230 us, 0.92 of the measured copy rate; a CTA keeps six tiles,
// 192 KB, on their way), and for many rows the chain score product, softmax,
// value product of a stream: 2750 cycles for two streams' 128 x 128 tiles
// where the products alone take 2048 (1.45 PFLOP/s on chunks of 4096 and 2250
// tokens, 0.76 of the measured bf16 rate; with D = 64 the products halve, the
// softmax stays, and the call takes 509 us).
//
// Over a 4-bit cache (CODES) two warps load codes and pairs as they lie, half a
// tile of 64 keys at a time, and four more make fp16 tiles of them in the same
// swizzle; products are of fp16 numbers, bf16 queries are scaled to them.  Up
// to 128 rows (SPLIT): both streams have every tile, a half of its keys each,
// and one warp issues all products, so that the next tile's scores are made
// beside this one's weights (32 chunks of 9 tokens 131 us with every other tile
// a stream, so 116).  Beside fp16 rows a weight there is two numbers as above;
// beside bf16 rows fp16's bits are enough (0.00167 off, with two 0.00166; the
// chunks of 9 tokens take 116 us and would take 131).  One warp that loaded and
// made a tile took 6400 cycles for it, half of them loading (246 us); 2000
// cycles of makers, 1800 of softmax and 1700 of products, in rings of two
// tiles, make 2800 a tile now, where the tile's bytes take 700: the stages wait
// for one another.  With 256 rows 690 us on the two prompt chunks (1.2 PFLOP/s,
// tensor pipe 0.50), where 16-bit keys take 557: not for the makers, which
// could make a quarter as much in the same time.
//
// A wait that gives up (see role_wait) stops the loads and the products; all
// other steps go on over meaningless data to the end of the share, so that
// every barrier between warps is reached.
#pragma once

#include <cuda.h>

#include <atomic>

#include "sdv_kv4.cuh"
#include "sdv_tcgen05.cuh"
#include "sdv_units.cuh"

namespace sdv {
namespace {

constexpr int kHalf = kTile / 2;  // keys a softmax thread weighs at a time
constexpr int kMaxGrid = 160;    // CTAs the workspace is laid out for
// Two warpgroups of softmax, one of roles; over a cache in 4 bits one that
// makes tiles of its codes.
template <bool CODES> constexpr int attn_threads() { return CODES ? 512 : 384; }
constexpr int kMmaWarp = 9;  // and 10; warps 8 and 11 load
constexpr int kBadRing = 64;     // units whose bad-page mark is kept
// A row's weights are 2^kBias at its reference m, and m moves up only when the
// scores' maximum is 2^kSlack above it: weights stay at or below 2^15, inside
// fp16's range, and hardly a tile rescales anything.  (With a slack of 2^8 the
// rows of a prompt tile did so in one tile of ten, for half a tile's time
// each.)  bf16 has fp32's exponents: its weights keep their bits at any scale.
// fp16 weights below 2^-14 lose bits and those below 2^-25 are gone, while l
// counts them in full.  So in fp16 a reference is worth 2^3, and it moves DOWN
// to the maximum of a half tile whose weights all lie 2^kDrop below it (one of
// thousands, perhaps, that matter beside a key far above them).  A weight is
// off by its own rounding, or by 2^-17 of the largest of its 64 keys; beside
// a key that set the reference, and in a half that hides keys, by 2^-28 of the
// reference's.  Sums grow by a move down, so none is made once they are kTop,
// nor by more than 2^kMost: what lies below is then no part of the result.
// For this, fp16 takes 2 to 5 % more (without bias and moves down, two prompt
// chunks of D = 128 took 559 us and take 588, 16 trees of 64 nodes 69 and 72,
// 9 tokens over 131072 keys 97 and 99).
template <class T> struct Scale {
  static constexpr float kSlack = 15.f, kBias = 0.f, kDrop = kInf;
};
template <> struct Scale<__half> {
  static constexpr float kSlack = 12.f, kBias = 3.f, kDrop = 11.f;
};
constexpr float kTop = 0x1p50f, kMost = 60.f;

struct AttnParams : UnitParams {
  const void *q;
  long long q_stride;
  int num_pages;
  int box;  // rows of one TMA box: a power of two that divides the page
  float scale_log2;  // scale x log2(e)
  // over a cache in 4 bits
  Kv4Cache c;
  bool bf16;  // type of q and out; fp16 otherwise
};

// --------------------------------------------------------- shared memory
// PAIR: 256 rows a unit, 128 a stream; otherwise both streams share 128.
template <int D, bool PAIR, bool CODES> struct Layout {
  static constexpr int kRows = PAIR ? 256 : 128;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQBytes = (PAIR ? 2 : 1) * kTileBytes;
  // Two rings of tiles, as many as fit: what is in flight covers the latency
  // of HBM.  PAIR and CODES: ring 0 holds the key tiles, ring 1 the value
  // tiles, read by both streams.  Otherwise ring st holds stream st's tiles in the order
  // it uses them (key, value, key, ...): a ring with one writer and one
  // reader, so that a stream that is ahead never takes a slot's earlier
  // filling for its own.
  static constexpr int kN0 = CODES       ? (D == 128 ? 2 : 4)
                             : D == 128 ? 3
                             : PAIR     ? 4
                                        : 5;
  static constexpr int kN1 = CODES       ? (D == 128 ? 2 : 4)
                             : D == 128 ? (PAIR ? 2 : 3)
                             : PAIR     ? 4
                                        : 5;
  // CODES: codes and pairs of 64 keys (or values), half a tile, in a ring of
  // their own for each ring of tiles: six halves where they fit (32 chunks of 9
  // tokens 115 us, with three 119), three beside 256 rows of queries.
  static constexpr int kRaw = D == 128 ? (PAIR ? 3 : 6) : 6;
  static constexpr int kRawBytes = 64 * (D / 2 + D / 8);
  static constexpr size_t kTiles =
      kQBytes + (size_t)kTileBytes * (kN0 + kN1) +
      (CODES ? 2 * kRaw * kRawBytes : 0);
};

template <int D, bool PAIR, bool CODES> struct Shared {
  using L = Layout<D, PAIR, CODES>;
  uint64_t full[2][L::kN0], empty[2][L::kN0];
  uint64_t raw_full[2][L::kRaw], raw_empty[2][L::kRaw];
  uint64_t q_full[2], s_full[2], turn[2], drain[2];
  uint64_t w_full[2][2], o_full[2][2];  // of a stream's tile halves; SPLIT:
                                        // w_full of its two buffers
  uint64_t idle;  // stream 1 has no tile: its product warp saw the queries
  uint32_t tmem;
  volatile int abort;
  int bad[kBadRing];  // unit count whose pages were bad
  float2 ml[2][PAIR ? 1 : kTile];
  float q_sl[2][CODES ? L::kRows : 1];  // factor of a row's scores
  Plan plan;
};
template <int D, bool PAIR, bool CODES> constexpr size_t attn_smem() {
  return Layout<D, PAIR, CODES>::kTiles + sizeof(Shared<D, PAIR, CODES>);
}

// A barrier of the two softmax warpgroups alone; of one of them.
__device__ __forceinline__ void streams_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}
__device__ __forceinline__ void stream_sync(int st) {
  if (st) asm volatile("bar.sync 3, 128;" ::: "memory");
  else asm volatile("bar.sync 2, 128;" ::: "memory");
}

// A pair as a sum of two 16-bit pairs.  bf16: the first is cut off, not
// rounded (a byte permutation), and the second holds the 8 bits after it.
template <class T>
__device__ __forceinline__ void split2(float2 z, uint32_t &w, uint32_t &rest);
template <>
__device__ __forceinline__ void split2<__nv_bfloat16>(float2 z, uint32_t &w,
                                                      uint32_t &rest) {
  const uint32_t x = __float_as_uint(z.x), y = __float_as_uint(z.y);
  w = __byte_perm(x, y, 0x7632);
  const float2 r = fma2(make_float2(__uint_as_float(x & 0xffff0000u),
                                    __uint_as_float(y & 0xffff0000u)),
                        make_float2(-1.f, -1.f), z);
  rest = pack2<__nv_bfloat16>(r.x, r.y);
}
template <>
__device__ __forceinline__ void split2<__half>(float2 z, uint32_t &w,
                                               uint32_t &rest) {
  w = pack2<__half>(z.x, z.y);
  const float2 r =
      fma2(__half22float2(*reinterpret_cast<const __half2 *>(&w)),
           make_float2(-1.f, -1.f), z);
  rest = pack2<__half>(r.x, r.y);
}

__device__ __forceinline__ float max32(const uint32_t *x) {
  const float *f = reinterpret_cast<const float *>(x);
  float a = fmaxf(f[0], f[1]), b = fmaxf(f[2], f[3]);
#pragma unroll
  for (int e = 4; e < 32; e += 4) {
    a = max3f(a, f[e], f[e + 1]);
    b = max3f(b, f[e + 2], f[e + 3]);
  }
  return fmaxf(a, b);
}

// Scores a row does not see become -inf.
__device__ __forceinline__ void hide32(uint32_t *x, uint32_t seen) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(seen >> e & 1)) x[e] = 0xff800000u;
}

// The largest of a row's 128 scores (of those it sees, where `cuts`).
__device__ __forceinline__ float row_max(uint32_t s_addr, bool cuts,
                                         const uint32_t *seen) {
  float m = -kInf;
#pragma unroll
  for (int c = 0; c < kTile; c += 64) {
    uint32_t x[64];
    tmem_ld32(s_addr + c, x);
    tmem_ld32(s_addr + c + 32, x + 32);
    tmem_wait_ld();
    if (cuts) {
      hide32(x, seen[c / 32]);
      hide32(x + 32, seen[c / 32 + 1]);
    }
    m = max3f(m, max32(x), max32(x + 32));
  }
  return m;
}

// 32 weights 2^(s sl + off) as 16-bit pairs, with REST as two (see split2);
// their sums before that are added to `sum`.
template <class T, bool REST>
__device__ __forceinline__ void weigh32(const uint32_t *x, float sl,
                                        float off, uint32_t *w,
                                        uint32_t *rest, float2 (&sum)[2]) {
  const float2 k2 = make_float2(sl, sl), o2 = make_float2(off, off);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float2 z = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
    z = fma2(z, k2, o2);
    z.x = ex2(z.x);
    z.y = ex2(z.y);
    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], z);
    if (REST) split2<T>(z, w[e >> 1], rest[e >> 1]);
    else w[e >> 1] = pack2<T>(z.x, z.y);
  }
}

// Columns of the score tile where the weights of half a tile go: over the
// scores of that half, which have been read by then.  With REST their second
// numbers follow them.
template <bool REST> constexpr int weight_col(int hf) {
  return hf * (REST ? kHalf : kHalf / 2);
}

// A softmax thread's row: where its scores and sums lie, its reference m
// and sum l.
struct Row {
  uint32_t s_addr, o_addr;
  float sl, m, l;
};

// The weights of one row in one tile, half a tile at a time, so that the
// values of one half are summed while the other is weighed.  They are taken
// against the reference at hand while the scores' maximum is still being
// found; where it turns out too far above or, in fp16, below (both rare), the
// sums are scaled and the half is weighed once more.  Chunks of 32 scores are
// fetched one ahead.  first: nothing is summed yet; parity: of the tile in the
// stream; w_full, o_full: of the tile's halves.  Tiles that hide scores have a
// copy of their own: a warp here runs on its scheduler's issue slots.
// CODES: the halves in a loop, since with the warps that make tiles an SM runs
// four kinds of code at a time and waits for instructions (two prompt chunks
// 804 us, so 681; with 16-bit keys 557 and 574).
template <class T, int D, bool HIDE, bool REST, bool CODES>
__device__ __forceinline__ bool weigh_tile(Row &row, const uint32_t *seen,
                                           uint64_t *w_full, uint64_t *o_full,
                                           bool first, uint32_t parity,
                                           volatile int *abort,
                                           int32_t *dev_status) {
  using S = Scale<T>;
  uint32_t x[2][32];
  tmem_ld32(row.s_addr, x[0]);
#pragma unroll (CODES && !HIDE ? 1 : 2)
  for (int hf = 0; hf < 2; ++hf) {
    uint32_t w[kHalf / 2], rest[REST ? kHalf / 2 : 32];
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    float mt = -kInf;
    const float off = row.m == -kInf ? 0.f : S::kBias - row.m * row.sl;
#pragma unroll
    for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
      uint32_t *xc = x[c & 1];
      tmem_wait_ld();
      if (c < 3) tmem_ld32(row.s_addr + 32 * (c + 1), x[(c + 1) & 1]);
      if (HIDE) hide32(xc, seen[c]);
      mt = fmaxf(mt, max32(xc));
      weigh32<T, REST>(xc, row.sl, off, w + 16 * (c & 1),
                       rest + 16 * (c & 1), sum);
    }
    constexpr bool DROPS = S::kDrop < kInf;
    const float up = (mt - row.m) * row.sl;
    bool move = mt > -kInf && !(up <= S::kSlack);
    if (DROPS && (!HIDE || (seen[2 * hf] & seen[2 * hf + 1]) == ~0u))
      move = move || (up < -S::kDrop && up > -kMost && row.l < kTop);
    if (__any_sync(~0u, move)) {
      float f = 1.f;
      if (move) {
        f = row.m == -kInf ? 1.f : ex2(-up);
        row.m = mt;
      }
      row.l *= f;
      if (hf || !first) {
        // all sums before this half are complete when the last of them are
        const bool fine =
            role_wait(&o_full[hf ^ 1], parity ^ (hf ^ 1), abort, dev_status);
        if (!__all_sync(~0u, fine)) return false;
        tmem_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(row.o_addr + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st32(row.o_addr + c, o);
        }
      }
      const float to = row.m == -kInf ? 0.f : S::kBias - row.m * row.sl;
      sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
        uint32_t y[32];
        tmem_ld32(row.s_addr + 32 * c, y);
        tmem_wait_ld();
        if (HIDE) hide32(y, seen[c]);
        weigh32<T, REST>(y, row.sl, to, w + 16 * (c & 1),
                         rest + 16 * (c & 1), sum);
      }
      __syncwarp();
    }
    tmem_st32(row.s_addr + weight_col<REST>(hf), w);
    if (REST) tmem_st32(row.s_addr + weight_col<REST>(hf) + kHalf / 2, rest);
    const float2 t = add2(sum[0], sum[1]);
    row.l += t.x + t.y;
    tmem_wait_st();
    tmem_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&w_full[hf]);
  }
  return true;
}

// The weights of one row in half a tile, where the stream has a half of each
// (SPLIT): the maximum first, then the weights in a second pass over the
// scores, in loops as short as they can be, for the same reason (32 chunks of
// 9 tokens 116 us; weighed while the maximum is being found 122).
template <class T, int D, bool REST>
__device__ __forceinline__ bool weigh_half(Row &row, bool cuts,
                                           const uint32_t (&seen)[2],
                                           uint64_t *w_full, uint64_t *o_full,
                                           bool first, uint32_t parity,
                                           volatile int *abort,
                                           int32_t *dev_status) {
  using S = Scale<T>;
  float mt = -kInf;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t x[32];
    tmem_ld32(row.s_addr + 32 * c, x);
    tmem_wait_ld();
    if (cuts) hide32(x, seen[c]);
    mt = fmaxf(mt, max32(x));
  }
  const float up = (mt - row.m) * row.sl;
  bool move = mt > -kInf && !(up <= S::kSlack);
  if (!cuts || (seen[0] & seen[1]) == ~0u)
    move = move || (up < -S::kDrop && up > -kMost && row.l < kTop);
  if (__any_sync(~0u, move)) {
    float f = 1.f;
    if (move) {
      f = row.m == -kInf ? 1.f : ex2(-up);
      row.m = mt;
    }
    row.l *= f;
    if (!first) {
      // all sums before this half are complete when the last of them are
      const bool fine = role_wait(o_full, parity ^ 1, abort, dev_status);
      if (!__all_sync(~0u, fine)) return false;
      tmem_fence_after();
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(row.o_addr + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st32(row.o_addr + c, o);
      }
    }
    __syncwarp();
  }
  const float off = row.m == -kInf ? 0.f : S::kBias - row.m * row.sl;
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t x[32], w[16], rest[16];
    tmem_ld32(row.s_addr + 32 * c, x);
    tmem_wait_ld();
    if (cuts) hide32(x, c ? seen[1] : seen[0]);
    weigh32<T, REST>(x, row.sl, off, w, rest, sum);
    // over the scores that they are the weights of
    tmem_st16(row.s_addr + 32 * c, w);
    if (REST) tmem_st16(row.s_addr + 32 * c + 16, rest);
  }
  const float2 t = add2(sum[0], sum[1]);
  row.l += t.x + t.y;
  tmem_wait_st();
  tmem_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(w_full);
  return true;
}

// A thread's part of a query row that LANES neighbouring lanes hold, to fp16
// pairs; returns the factor of the row's scores.  bf16 rows are multiplied by
// the power of two that takes the row's largest element to [2^14, 2^15): exact
// but for elements 2^-28 of that and below.  The power stops at 2^126, whose
// inverse is still a normal number: rows below 2^-112 are taken to below 2^14,
// where bf16's least number, 2^-133, is 2^-7, and nothing is lost at all.  A
// factor beyond fp32's numbers becomes the greatest of them: times a score of
// 0 it has to be 0.  A row with NaN or infinity gets a NaN factor.
template <int LANES, int N>
__device__ __forceinline__ float fit_query(uint32_t (&w)[N], bool bf16,
                                           float scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1)
    top = max(top, __shfl_xor_sync(~0u, top, d));
  float f = scale;
  if (bf16) {
    const int exp = max((int)(top >> 7), 15) - 127;
    const float up = __uint_as_float((uint32_t)(14 - exp + 127) << 23);
    f *= __uint_as_float((uint32_t)(exp - 14 + 127) << 23);
    f = fminf(f, 0x1.fffffep127f);
    if (top >= 0x7f80u) f = __int_as_float(0x7fc00000);
#pragma unroll
    for (int i = 0; i < N; ++i)
      w[i] = pack2<__half>(__uint_as_float(w[i] << 16) * up,
                           __uint_as_float(w[i] & 0xffff0000u) * up);
  } else if (top >= 0x7c00u) {
    f = __int_as_float(0x7fc00000);
  }
  return f;
}

// Codes and pairs of the key tiles (ring 0) or value tiles (1), half a tile at
// a time, by one warp.
template <int D, bool PAIR, int ROWS>
__device__ __forceinline__ void load_codes(const AttnParams &p,
                                           Shared<D, PAIR, true> &s,
                                           char *raw, int me) {
  using L = Layout<D, PAIR, true>;
  constexpr int CODE_BYTES = 32 * D;
  const int lane = threadIdx.x & 31, sb = p.c.scale_bytes;
  const uint32_t to = smem_addr(raw) + 16 * lane;
  const int chunk = 16 * (lane & (D / 4 - 1));
  const int pair_at = 16 * (lane & (sb / 2 - 1)), pair_8 = lane / (sb / 2);
  bool fine = true;
  RingAt at(L::kRaw);
  Units<ROWS> u(p, s.plan);
  for (; u.left && fine; u.next()) {
    const int32_t *table = p.block_table + (long long)u.b * p.max_pages;
    auto look_up = [&](int j) {  // page of keys 8 (lane % 16) to + 7 of tile j
      const int key = j * kTile + 8 * (lane & 15);
      return j < u.j1 && key < u.c.kv ? __ldg(table + div_by(key, p.by_page))
                                      : -1;
    };
    int id = look_up(u.j0);
    for (int j = u.j0; j < u.j1 && fine; ++j) {
      const int key = j * kTile + 8 * (lane & 15);
      long long code = -1, pair = -1;  // negative: none
      if (id >= 0 && id < p.num_pages) {
        const int row = (u.h - div_by(key, p.by_page)) * p.page_size + key;
        code = id * p.c.page_stride + (long long)row * (D / 2);
        pair = id * p.c.scale_stride + (long long)row * sb;
      } else if (key < u.c.kv) {
        s.bad[u.count % kBadRing] = u.count;
        status_or(p.dev_status, SD_DEV_BAD_PAGE);
      }
      id = look_up(j + 1);
#pragma unroll 1
      for (int first = 0; first < 16; first += 8) {  // halves of the tile
        fine = role_wait(&s.raw_empty[me][at.slot], at.parity ^ 1, &s.abort,
                         p.dev_status);
        if (!__all_sync(~0u, fine)) {
          fine = false;
          break;
        }
        const char *from = (me ? p.c.v : p.c.k) + chunk;
        const uint32_t dst = to + at.slot * L::kRawBytes;
        long long c[D / 16];
#pragma unroll
        for (int o = 0; o < D / 16; ++o)
          c[o] = __shfl_sync(
              ~0u, code, first + (D == 128 ? o : 2 * o + (lane >> 4)));
        const long long c0 = __shfl_sync(~0u, pair, first + (pair_8 & 7));
        // 64 / sb lanes hold eight keys' pairs
        const long long c1 =
            __shfl_sync(~0u, pair, first + (pair_8 + 64 / sb & 7));
#pragma unroll
        for (int o = 0; o < D / 16; ++o)
          cp16(dst + 512 * o, from + c[o], c[o] >= 0);
        const char *pairs = (me ? p.c.v_scale : p.c.k_scale) + pair_at;
        cp16(dst + CODE_BYTES, pairs + c0, pair_8 < 8 && c0 >= 0);
        cp16(dst + CODE_BYTES + 512, pairs + c1,
             pair_8 + 64 / sb < 8 && c1 >= 0);
        cp_arrive(smem_addr(&s.raw_full[me][at.slot]));
        at.next();
      }
    }
  }
  cp_commit();
  cp_wait<0>();
}

// Half `hf` of the tiles of ring `me`, as fp16 numbers in the swizzle, by one
// warp: a word of codes, eight neighbours, becomes the 16 bytes of a chunk.
// What lies past a sequence's keys becomes zeros.
template <int D, bool PAIR, int ROWS>
__device__ __forceinline__ void make_tiles(const AttnParams &p,
                                           Shared<D, PAIR, true> &s,
                                           char *ring, const char *raw,
                                           int me, int hf) {
  using L = Layout<D, PAIR, true>;
  constexpr int W = D / 32;  // words of a key a thread
  constexpr int CODE_BYTES = 32 * D;
  const int lane = threadIdx.x & 31, sb = p.c.scale_bytes;
  const int row = lane >> 2, t = lane & 3;
  // Chunk i of the thread's W is the (W t + i)-th of the row, eight to a
  // column half.  A store's threads, two rows of four, would meet the same
  // banks for both halves: the second half's take their words in another
  // order.  (Addresses of shared memory as such: a pointer that may be to
  // either ring would be a generic one.)
  const int turn = D == 128 ? t & 2 : 0;
  const uint32_t code_from =
      smem_addr(raw) + row * (D / 2) + t * (D / 8) + 4 * turn;
  const uint32_t pair_from = smem_addr(raw) + CODE_BYTES + row * sb +
                             4 * ((t * (D / 4)) >> p.c.shift);
  const uint32_t tile_at = smem_addr(ring) +
                           (D == 128 ? (t >> 1) * (kTile * 128) : 0) +
                           (64 * hf + row) * 128;
  uint32_t chunk[W];
#pragma unroll
  for (int i = 0; i < W; ++i)
    chunk[i] = (((W * t + (i ^ turn)) & 7) ^ row) * 16;
  bool fine = true;
  RingAt at(me ? L::kN1 : L::kN0), from(L::kRaw);
  if (hf) from.next();
  Units<ROWS> u(p, s.plan);
  for (; u.left && fine; u.next())
    for (int j = u.j0; j < u.j1; ++j) {
      fine = role_wait(&s.empty[me][at.slot], at.parity ^ 1, &s.abort,
                       p.dev_status) &&
             role_wait(&s.raw_full[me][from.slot], from.parity, &s.abort,
                       p.dev_status);
      if (!__all_sync(~0u, fine)) {
        fine = false;
        break;
      }
      const uint32_t tile = tile_at + at.slot * L::kTileBytes;
      const uint32_t codes = code_from + from.slot * L::kRawBytes;
      const uint32_t pairs = pair_from + from.slot * L::kRawBytes;
      const int left = u.c.kv - (j * kTile + 64 * hf + row);
      // Eight keys at a time, the next ones' words loaded first (the
      // compiler may not move a load past a store).
      uint32_t w[2][W], x[2];
      auto load = [&](int b, int o) {
        const uint32_t at = codes + o * 8 * (D / 2);
        lds_pair(at, w[b]);
        if (D == 128) lds_pair(at + 8 - 8 * turn, w[b] + W - 2);
        x[b] = lds_word(pairs + o * 8 * sb);
      };
      auto make = [&](int k, int o) {
        if (8 * o >= left) x[k] = 0;
        const uint32_t a = both_lo(x[k]), b = both_hi(x[k]);
        uint4 y[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          y[i].x = kv4_fma(kv4_codes(w[k][i], 0), a, b);
          y[i].y = kv4_fma(kv4_codes(w[k][i], 1), a, b);
          y[i].z = kv4_fma(kv4_codes(w[k][i], 2), a, b);
          y[i].w = kv4_fma(kv4_codes(w[k][i], 3), a, b);
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
          sts_v4(tile + o * 8 * 128 + chunk[i], y[i]);
      };
      load(0, 0);
#pragma unroll 1
      for (int o = 0; o < 8; o += 2) {
        load(1, o + 1);
        make(0, o);
        if (o < 6) load(0, o + 2);
        make(1, o + 1);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.full[me][at.slot]);
        mbar_arrive(&s.raw_empty[me][from.slot]);
      }
      at.next();
      from.next();
      from.next();
    }
}

// ------------------------------------------------------------- the kernel
// T: type of the products.  CODES: the cache is in 4 bits, T is fp16, q and
// out are of the type that p.bf16 says.  REST: weights are two numbers each.
template <class T, int D, bool PAIR, bool CODES, bool REST>
__global__ void __launch_bounds__(attn_threads<CODES>(), 1)
attention_kernel(const __grid_constant__ AttnParams p,
                 const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map) {
  using L = Layout<D, PAIR, CODES>;
  constexpr int ROWS = L::kRows;
  // Up to 128 rows over a 4-bit cache: both streams have every key tile, half
  // of its keys each, and the next tile's scores are made meanwhile.
  constexpr bool SPLIT = CODES && !PAIR;
  constexpr bool BF16 = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) char dyn[];  // swizzled tiles first
  using S = Shared<D, PAIR, CODES>;
  S &s = *reinterpret_cast<S *>(dyn + L::kTiles);
  char *q_tile = dyn;
  char *ring[2] = {q_tile + L::kQBytes,
                   q_tile + L::kQBytes + L::kN0 * L::kTileBytes};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i)
      for (int k = 0; k < L::kN0; ++k) {
        mbar_init(&s.full[i][k], CODES ? 2 : 1);
        mbar_init(&s.empty[i][k], PAIR ? 2 : 1);  // the streams that read it
      }
    for (int i = 0; i < 2 && CODES; ++i)
      for (int k = 0; k < L::kRaw; ++k) {
        mbar_init(&s.raw_full[i][k], 32);
        mbar_init(&s.raw_empty[i][k], 1);
      }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.q_full[i], PAIR ? 4 : 8);
      mbar_init(&s.s_full[i], 1);
      for (int hf = 0; hf < 2; ++hf) {
        mbar_init(&s.w_full[i][hf], 4);
        mbar_init(&s.o_full[i][hf], 1);
      }
      mbar_init(&s.turn[i], 1);
    }
    mbar_init(&s.idle, 1);
    mbar_init(&s.drain[0], 1);
    mbar_init(&s.drain[1], 1);
    s.abort = 0;
    fence_mbar_init();
  }
  if (tid < kBadRing) s.bad[tid] = 0;
  if (warp == kMmaWarp) tmem_alloc_all(&s.tmem);
  if (!CODES && warp == 8 && lane == 0) {
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }
  griddep_wait();  // nothing before this reads or writes what a grid before
                   // this one may still write or read
  make_plan<ROWS>(p, s.plan);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem;
  bool fine = true;

  // 384 threads start with 168 registers each, 512 with 128; a softmax thread
  // holds much of a row, a role next to nothing: 256 x 208 + 128 x 88 = 384 x
  // 168, and 256 x 168 + 256 x 88 = 512 x 128.
  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  else if (CODES) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  // (the branch has to be on the same condition: code that both kinds reach
  // has the smaller number)
  if (warp >= 8) {
    const bool maker = CODES && (warp == 8 || warp >= 11);
    if constexpr (CODES) {
      char *raw = q_tile + L::kQBytes + (L::kN0 + L::kN1) * L::kTileBytes;
      const int me = warp == 8 || warp == 12 || warp == 13 ? 0 : 1;
      raw += me * L::kRaw * L::kRawBytes;
      if (warp == 8 || warp == 11)
        load_codes<D, PAIR, ROWS>(p, s, raw, me);
      else if (maker)
        make_tiles<D, PAIR, ROWS>(p, s, ring[me], raw, me, warp & 1);
    }
    Units<ROWS> u(p, s.plan);
    if (maker) {
      // done
    } else if (!CODES && (warp == 8 || warp == 11)) {
      // ---- ring `me`, a box of page rows at a time
      const int me = warp == 8 ? 0 : 1;
      const int per = kTile / p.box;  // boxes of a tile and column half
      const bool has = lane < per * (D / 64);
      const int a = lane % per, half = lane / per;
      const uint32_t to = half * (kTile * 128) + a * p.box * 128;
      RingAt at(me ? L::kN1 : L::kN0);
      unsigned filled = 0;
      int page = 0, tok = 0;
      auto load = [&](const CUtensorMap *map) {
        fine = role_wait(&s.empty[me][at.slot], at.parity ^ 1, &s.abort,
                         p.dev_status);
        if (!__all_sync(~0u, fine)) {
          fine = false;
          return;
        }
        uint64_t *full = &s.full[me][at.slot];
        if (lane == 0) mbar_expect_tx(full, L::kTileBytes);
        __syncwarp();
        if (has)
          tma_load_4d(ring[me] + at.slot * L::kTileBytes + to, map, half * 64,
                      tok, u.h, page, full);
        at.next();
        ++filled;
      };
      for (; u.left && fine; u.next()) {
        const int32_t *table = p.block_table + (long long)u.b * p.max_pages;
        const int step = PAIR ? 1 : 2;
        for (int j = u.j0 + (PAIR ? 0 : me); j < u.j1 && fine; j += step) {
          bool bad = false;
          if (has) {
            const int key = j * kTile + a * p.box;
            page = p.num_pages > 0 ? p.num_pages : 1;  // out of range: zeros
            tok = 0;
            if (key < u.c.kv) {
              const int n = div_by(key, p.by_page);
              const int id = __ldg(table + n);
              if (id >= 0 && id < p.num_pages) page = id;
              else bad = true;
              tok = key - n * p.page_size;
            }
          }
          if (__any_sync(~0u, bad) && lane == 0) {
            s.bad[u.count % kBadRing] = u.count;
            status_or(p.dev_status, SD_DEV_BAD_PAGE);
          }
          if (!PAIR || me == 0) load(&k_map);
          if ((!PAIR || me == 1) && fine) load(&v_map);
        }
      }
      if (!fine) {  // give up: let the copies in flight land first
        for (int i = 0; i < at.n; ++i)
          if (filled > (unsigned)i) {
            const unsigned last = (filled - 1 - i) / at.n;
            for (unsigned it = 0; it < (1u << 20); ++it)
              if (mbar_try_wait(&s.full[me][i], last & 1)) break;
          }
      }
    } else if constexpr (SPLIT) {
      // ---- tensor-core products, all by one warp: the next tile's scores go
      // out before this one's weights are waited for.  Products run in the
      // order issued, so a buffer's scores are made after the values of the
      // tile before last, whose weights it held.
      constexpr uint32_t S_DESC = umma_idesc(BF16, false, kTile, kTile);
      constexpr uint32_t O_DESC = umma_idesc(BF16, true, kTile, D);
      constexpr uint32_t HI = umma_desc_hi(1024);
      const uint32_t q_lo = umma_desc_lo(q_tile, 16);
      const uint32_t k_lo = umma_desc_lo(ring[0], 16);
      const uint32_t v_lo = umma_desc_lo(ring[1], kTile * 128);
      RingAt k_at(L::kN0), v_at(L::kN1);
      uint32_t qp = 0, wp = 0, buf = 0;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        fine = fine && role_wait(bar, parity, &s.abort, p.dev_status);
      };
      auto scores = [&](uint32_t to) {
        wait(&s.full[0][k_at.slot], k_at.parity);
        if (elect_one() && fine) {
          const uint32_t b = k_lo + k_at.slot * (L::kTileBytes / 16);
          tmem_fence_after();
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int at = ((i / 4) * (kTile * 128) + (i % 4) * 32) / 16;
            umma_ss<HI>(tmem + to * kTile, q_lo + at, b + at, S_DESC, i > 0);
          }
          umma_commit(&s.s_full[to]);
          umma_commit(&s.empty[0][k_at.slot]);
        }
        __syncwarp();
        k_at.next();
      };
      if (warp == kMmaWarp) {
        for (; u.left; u.next()) {
          const int cnt = u.j1 - u.j0;
          wait(&s.q_full[0], qp);
          qp ^= 1;
          scores(buf);
          for (int i = 0; i < cnt; ++i) {
            if (i + 1 < cnt) scores(buf ^ 1);
            wait(&s.full[1][v_at.slot], v_at.parity);
            for (int st = 0; st < 2; ++st) {
              wait(&s.w_full[st][buf], wp >> buf & 1);
              if (elect_one() && fine) {
                const uint32_t b = v_lo + v_at.slot * (L::kTileBytes / 16) +
                                   st * (kHalf * 128 / 16);
                const uint32_t w = tmem + buf * kTile + st * kHalf;
                tmem_fence_after();
#pragma unroll
                for (int k = 0; k < kHalf / 16; ++k)
#pragma unroll
                  for (int rest = 0; rest < (REST ? 2 : 1); ++rest)
                    umma_ts<HI>(tmem + 2 * kTile + st * D,
                                w + k / 2 * 32 + k % 2 * 8 + rest * 16,
                                b + k * 16 * 128 / 16, O_DESC,
                                i > 0 || k > 0 || rest > 0);
                umma_commit(&s.o_full[st][0]);
                if (st) umma_commit(&s.empty[1][v_at.slot]);
              }
              __syncwarp();
            }
            wp ^= 1u << buf;  // (weights may be a buffer ahead of this)
            v_at.next();
            buf ^= 1;
          }
        }
        if (__any_sync(~0u, !fine)) {
          // tensor memory is freed below: let products in flight end
          if (elect_one()) umma_commit(&s.drain[0]);
          __syncwarp();
          for (unsigned it = 0; it < (1u << 20); ++it)
            if (mbar_try_wait(&s.drain[0], 0)) break;
        }
      }
    } else {
      // ---- tensor-core products of stream st, a warp each: while one is held
      // up issuing (products queue some 200 cycles deep) the other waits for
      // its weights
      const int st = warp - kMmaWarp;
      constexpr uint32_t S_DESC = umma_idesc(BF16, false, kTile, kTile);
      constexpr uint32_t O_DESC = umma_idesc(BF16, true, kTile, D);
      constexpr uint32_t HI = umma_desc_hi(1024);
      const uint32_t s_addr = tmem + st * kTile;
      const uint32_t o_addr = tmem + 2 * kTile + st * D;
      const uint32_t q_lo =
          umma_desc_lo(q_tile + (PAIR ? st : 0) * L::kTileBytes, 16);
      // where the stream reads keys and values next
      const int kr = PAIR ? 0 : st, vr = PAIR ? 1 : st;
      const uint32_t k_lo = umma_desc_lo(ring[kr], 16);
      const uint32_t v_lo = umma_desc_lo(ring[vr], kTile * 128);
      RingAt ring_k(kr ? L::kN1 : L::kN0), ring_v(L::kN1);
      RingAt &k_at = ring_k, &v_at = PAIR ? ring_v : ring_k;
      uint32_t wp = 0, qp = 0;
      // After a wait that gives up nothing more is issued, but the loops go on
      // to their ends: lanes may disagree about it, and elect_one() and
      // __syncwarp() want them all.
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        fine = fine && role_wait(bar, parity, &s.abort, p.dev_status);
      };
      // S against the next key tile
      auto wait_k = [&] { wait(&s.full[kr][k_at.slot], k_at.parity); };
      auto scores = [&] {
        if (elect_one() && fine) {
          const uint32_t b = k_lo + k_at.slot * (L::kTileBytes / 16);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int at = ((i / 4) * (kTile * 128) + (i % 4) * 32) / 16;
            umma_ss<HI>(s_addr, q_lo + at, b + at, S_DESC, i > 0);
          }
          umma_commit(&s.s_full[st]);
          umma_commit(&s.empty[kr][k_at.slot]);
        }
        __syncwarp();
        k_at.next();
      };
      // Wait for the value tile of key tile j.  What lies past the sequence's
      // keys becomes zero, so that 0 x NaN of a stale page cannot reach the
      // sums (both streams may write the same zeros).
      auto wait_v = [&](int j) {
        wait(&s.full[vr][v_at.slot], v_at.parity);
        const int from = u.c.kv - j * kTile;
        if (!CODES && from < kTile) {
          const int to = (from + p.box - 1) / p.box * p.box;
          char *v = ring[vr] + v_at.slot * L::kTileBytes;
          for (int i = lane; i < (to - from) * 8 * (D / 64); i += 32) {
            const int row = from + i / 8 % (to - from);
            const int half = i / 8 / (to - from);
            *reinterpret_cast<uint4 *>(v + half * (kTile * 128) + row * 128 +
                                       (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
        }
      };
      // O with half hf of that tile
      auto values = [&](int hf, bool first) {
        if (elect_one() && fine) {
          const uint32_t b = v_lo + v_at.slot * (L::kTileBytes / 16) +
                             hf * (kHalf * 128 / 16);
          const uint32_t w = s_addr + weight_col<REST>(hf);
          tmem_fence_after();
#pragma unroll
          for (int i = 0; i < kHalf / 16; ++i)
            umma_ts<HI>(o_addr, w + i * 8, b + i * 16 * 128 / 16, O_DESC,
                        !first || i > 0);
          if (REST) {
#pragma unroll
            for (int i = 0; i < kHalf / 16; ++i)
              umma_ts<HI>(o_addr, w + kHalf / 2 + i * 8,
                          b + i * 16 * 128 / 16, O_DESC, true);
          }
          umma_commit(&s.o_full[st][hf]);
          if (hf) umma_commit(&s.empty[vr][v_at.slot]);
        }
        __syncwarp();
        if (hf) v_at.next();
      };
      // 256 rows: the streams take strict turns, a value and a score product
      // at a time, so that one's softmax runs under the other's products
      // (left to themselves they fall into step, and both wait for both)
      uint32_t tp = st ^ 1;
      auto take_turn = [&] {
        wait(&s.turn[st], tp);
        tp ^= 1;
      };
      auto pass_turn = [&] {
        if (elect_one() && fine) mbar_arrive(&s.turn[st ^ 1]);
        __syncwarp();
      };
      for (; u.left; u.next()) {
        const int cnt = u.j1 - u.j0;
        if (PAIR && st == 1 && u.rows <= kTile) {
          // no rows: let go of every tile as it comes
          for (int i = 0; i < cnt; ++i) {
            wait(&s.full[kr][k_at.slot], k_at.parity);
            if (fine && lane == 0) mbar_arrive(&s.empty[kr][k_at.slot]);
            k_at.next();
            wait(&s.full[vr][v_at.slot], v_at.parity);
            if (fine && lane == 0) mbar_arrive(&s.empty[vr][v_at.slot]);
            v_at.next();
          }
          continue;
        }
        wait(&s.q_full[PAIR ? st : 0], qp);
        qp ^= 1;
        const int i0 = PAIR ? 0 : st, step = PAIR ? 1 : 2;
        const bool turns = PAIR && u.rows > kTile;
        if (i0 < cnt) {
          wait_k();
          if (turns) take_turn();
          tmem_fence_after();
          scores();
          if (turns) pass_turn();
        } else if (!PAIR) {
          if (elect_one() && fine) mbar_arrive(&s.idle);
          __syncwarp();
        }
        for (int i = i0; i < cnt; i += step) {
          const bool more = i + step < cnt;
          wait_v(u.j0 + i);
          if (PAIR && more) wait_k();
          wait(&s.w_full[st][0], wp);
          if (turns) take_turn();
          values(0, i == i0);
          wait(&s.w_full[st][1], wp);
          wp ^= 1;
          values(1, false);
          if (!PAIR && more) wait_k();
          if (more) scores();
          if (turns) pass_turn();
        }
      }
      if (__any_sync(~0u, !fine)) {
        // tensor memory is freed below: let products in flight end
        if (elect_one()) umma_commit(&s.drain[st]);
        __syncwarp();
        for (unsigned it = 0; it < (1u << 20); ++it)
          if (mbar_try_wait(&s.drain[st], 0)) break;
      }
    }
  } else {
    Units<ROWS> u(p, s.plan);
    // ---- softmax: stream st, a thread per row
    const int st = warp >> 2, r = tid & (kTile - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes << 16
    float sl = p.scale_log2;
    int sl_at = 0;  // CODES: where load_q leaves the rows' factors
    unsigned tn = 0;  // tiles of this stream seen
    uint32_t idle_p = 0;
    if (tid == 0) p.cut[blockIdx.x].parts = 0;
    const int base_row = PAIR ? st * kTile : 0;
    // a stream without rows takes no part in a unit
    auto active = [&](const Units<ROWS> &v) {
      return !PAIR || v.rows > base_row;
    };
    // a unit's queries, in the tiles' swizzle
    auto load_q = [&](const Units<ROWS> &v) {
      if (!active(v)) return;
      constexpr int CH = D / 8, NT = PAIR ? 128 : 256;
      const int me = PAIR ? r : tid, ch = me % CH;
      const uint16_t *src = (const uint16_t *)p.q + v.c.start * p.q_stride +
                            (long long)v.h * p.G * D + ch * 8;
      char *dst = q_tile + (PAIR ? st : 0) * L::kTileBytes +
                  (ch >> 3) * (kTile * 128);
      uint4 x[kTile * CH / NT];
#pragma unroll
      for (int i = 0; i < kTile * CH / NT; ++i) {
        const int n = base_row + me / CH + i * (NT / CH);
        x[i] = make_uint4(0, 0, 0, 0);
        if (n < v.rows) {
          const int at = v.t * ROWS + n, tok = div_by(at, p.by_G);
          x[i] = __ldg(reinterpret_cast<const uint4 *>(
              src + tok * p.q_stride + (at - tok * p.G) * D));
        }
      }
#pragma unroll
      for (int i = 0; i < kTile * CH / NT; ++i) {
        const int n = me / CH + i * (NT / CH);
        if constexpr (CODES) {
          uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          const float f = fit_query<CH>(w, p.bf16, p.scale_log2);
          x[i] = make_uint4(w[0], w[1], w[2], w[3]);
          if (ch == 0) s.q_sl[sl_at][base_row + n] = f;
        }
        *reinterpret_cast<uint4 *>(dst + n * 128 +
                                   (((ch & 7) ^ (n & 7)) << 4)) = x[i];
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_full[PAIR ? st : 0]);
    };
    if (u.left) load_q(u);
    if (CODES && !PAIR) streams_sync();
    while (u.left) {
      if constexpr (CODES) {
        if (PAIR) stream_sync(st);
        sl = s.q_sl[sl_at][base_row + r];
        sl_at ^= 1;
      }
      if (tid == 0 && u.j0 == 0 && u.j1 < u.nk) {
        // this CTA's last unit goes on in the CTAs up to the one whose
        // share holds the unit's last tile
        const unsigned long long end =
            s.plan.x1 + (unsigned)(u.nk - u.j1);
        CutUnit cut;
        cut.parts = (int)((end * s.plan.n - 1) / s.plan.total) -
                    (int)blockIdx.x + 1;
        cut.rows = u.rows;
        cut.start = u.c.start;
        cut.head = u.h;
        cut.first = u.t * ROWS;
        p.cut[blockIdx.x] = cut;
      }
      Units<ROWS> next(u);
      next.next();
      if (next.left && active(next)) {  // its queries on their way to L2
        const int n = base_row + r, at = next.t * ROWS + n;
        if (n < next.rows && (PAIR || st == 0)) {
          const int tok = div_by(at, p.by_G);
          const uint16_t *q = (const uint16_t *)p.q +
                              (next.c.start + tok) * p.q_stride +
                              (next.h * p.G + at - tok * p.G) * D;
#pragma unroll
          for (int e = 0; e < D; e += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q + e));
        }
      }
      const int cnt_all = u.j1 - u.j0;
      const int cnt = !active(u)        ? 0
                      : PAIR || SPLIT ? cnt_all
                                      : (cnt_all - st + 1) / 2;
      const int row_at = u.t * ROWS + base_row + r;
      const bool mine = base_row + r < u.rows;
      const bool warp_rows = base_row + (warp & 3) * 32 < u.rows;
      const int token = mine ? div_by(row_at, p.by_G) : 0;
      const int ctx = u.c.kv - u.c.n, limit = ctx + token;
      Row row = {tmem + lanes + st * kTile,
                 tmem + lanes + 2 * kTile + st * D, sl, -kInf, 0.f};
      for (int i = 0; i < cnt; ++i, ++tn) {
        // SPLIT: tiles alternate between two buffers of scores
        const int j = u.j0 + (PAIR || SPLIT ? i : 2 * i + st);
        const int buf = SPLIT ? tn & 1 : st;
        fine = role_wait(&s.s_full[buf], (SPLIT ? tn >> 1 : tn) & 1, &s.abort,
                         p.dev_status);
        if (!__all_sync(~0u, fine)) { fine = false; break; }
        constexpr int KEYS = SPLIT ? kHalf : kTile;
        if (SPLIT) row.s_addr = tmem + lanes + buf * kTile + st * kHalf;
        if (warp_rows) {
          tmem_fence_after();
          // only tiles past the row's last key hide anything
          const int key = j * kTile + (SPLIT ? st * kHalf : 0);
          const bool cuts = __any_sync(
              ~0u, key + KEYS - 1 > (p.mask ? ctx - 1 : limit));
          uint32_t seen[KEYS / 32] = {};
          if (cuts) {
#pragma unroll
            for (int c = 0; c < KEYS / 32; ++c)
              seen[c] =
                  mine ? seen_bits(p, u.c, token, limit, key + 32 * c) : 0;
          }
          __syncwarp();
          if constexpr (SPLIT) {
            fine = weigh_half<T, D, REST>(
                row, cuts, seen, &s.w_full[st][buf], &s.o_full[st][0], i == 0,
                tn & 1, &s.abort, p.dev_status);
          } else {
            if (i == 0) row.m = row_max(row.s_addr, cuts, seen);
            fine = cuts ? weigh_tile<T, D, true, REST, CODES>(
                              row, seen, s.w_full[st], s.o_full[st], i == 0,
                              tn & 1, &s.abort, p.dev_status)
                        : weigh_tile<T, D, false, REST, CODES>(
                              row, seen, s.w_full[st], s.o_full[st], i == 0,
                              tn & 1, &s.abort, p.dev_status);
          }
          if (!fine) break;
        } else if (lane == 0) {
          mbar_arrive(&s.w_full[st][SPLIT ? buf : 0]);
          if (!SPLIT) mbar_arrive(&s.w_full[st][1]);
        }
      }
      // ---- the end of the unit.  The last scores are out, so the next
      // unit's queries may replace this one's: its first scores are under
      // way while this one's rows are written
      if (PAIR && next.left) load_q(next);
      if (cnt > 0) {
        role_wait(&s.o_full[st][SPLIT ? 0 : 1], (tn - 1) & 1, &s.abort,
                  p.dev_status);
        __syncwarp();
        tmem_fence_after();
      } else if (!PAIR) {
        // One tile, and it is stream 0's: nothing else holds the queries back
        // until product warp 1 has seen these.  Were they replaced twice
        // before it looks, their barrier would show it the parity that it is
        // waiting to see end.
        role_wait(&s.idle, idle_p, &s.abort, p.dev_status);
        idle_p ^= 1;
        __syncwarp();
      }
      // the two streams' sums of the same rows are joined; stream st then
      // writes column half st.  256 rows: each its own rows, all columns.
      float f0 = 1.f, f1 = 0.f, m = row.m, l = row.l;
      if (!PAIR) {
        s.ml[st][r] = make_float2(m, l);
        tmem_fence_before();
        streams_sync();
        tmem_fence_after();
        if (next.left) load_q(next);
        const float2 other = s.ml[st ^ 1][r];
        const float mj = fmaxf(m, other.x);
        const float fm = m == -kInf ? 0.f : ex2((m - mj) * sl);
        const float fo = other.x == -kInf ? 0.f : ex2((other.x - mj) * sl);
        l = l * fm + other.y * fo;
        m = mj;
        f0 = st ? fo : fm;
        f1 = st ? fm : fo;
      }
      if (s.bad[u.count % kBadRing] == u.count) l = __int_as_float(0x7fc00000);
      const bool whole = u.j0 == 0 && u.j1 == u.nk;
      const int c_lo = PAIR ? 0 : st * (D / 2), c_n = PAIR ? D : D / 2;
      const uint32_t o_addr =
          tmem + lanes + 2 * kTile + (PAIR ? st * D : 0) + c_lo;
      const bool second = !PAIR && (SPLIT || cnt_all > 1);
      if (warp_rows) {
        const long long to = (long long)(u.c.start + token) * p.Hq +
                             u.h * p.G + (mine ? row_at - token * p.G : 0);
        const long long part =
            ((long long)blockIdx.x * 2 + (u.j0 == 0 ? 1 : 0)) * ROWS +
            base_row + r;
        // no key seen: 0, also where O has 0 times another row's infinity; a
        // NaN sum stays NaN
        if (l == 0.f) f0 = f1 = 0.f;
        else if (whole) f0 *= 1.f / l, f1 *= 1.f / l;
        if (mine && (PAIR || st == 0)) {
          // l counts 2^kBias for a weight of 1
          const float ref = m * sl - Scale<T>::kBias;
          if (!whole) p.part_ml[part] = make_float2(ref, l);
          else if (p.lse)
            p.lse[to] = l == 0.f ? -kInf : (ref + log2f(l)) * kLn2;
        }
        uint16_t *out = (uint16_t *)p.out + to * D + c_lo;
        float *part_o = p.part_o + part * D + c_lo;
#pragma unroll
        for (int c = 0; c < c_n; c += 32) {
          __syncwarp();  // tcgen05.ld wants the whole warp
          uint32_t a[32];
          tmem_ld32(o_addr + c, a);
          tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = f0 == 0.f ? 0.f : __uint_as_float(a[e]) * f0;
          if (second) {
            tmem_ld32(o_addr + D + c, a);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = f1 == 0.f ? o[e] : fmaf(__uint_as_float(a[e]), f1, o[e]);
          }
          if (!mine) {
            // no such row
          } else if (whole) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w[e] = !CODES || !p.bf16
                         ? pack2<T>(o[2 * e], o[2 * e + 1])
                         : pack2<__nv_bfloat16>(o[2 * e], o[2 * e + 1]);
            st_v8(out + c, w);
            st_v8(out + c + 16, w + 8);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(o[e]);
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_v8(part_o + c + e, a + e);
          }
        }
      }
      __syncwarp();
      tmem_fence_before();
      if (!PAIR) streams_sync();  // O, m and l may be overwritten
      u.to(next);
    }
  }

  if (s.plan.any_unusable) {
    // NaN for the sequences that cannot be read
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      const Chunk c = attn_chunk(p, b);
      if (c.usable || c.n == 0) continue;
      if (tid == 0) status_or(p.dev_status, SD_DEV_BAD_LENGTH);
      const long long lo = (long long)c.start * p.Hq,
                      n = (long long)c.n * p.Hq;
      for (long long i = tid; i < n * D; i += attn_threads<CODES>())
        ((uint16_t *)p.out)[lo * D + i] = 0x7fff;  // NaN of either type
      if (p.lse)
        for (long long i = tid; i < n; i += attn_threads<CODES>())
          p.lse[lo + i] = __int_as_float(0x7fc00000);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_free_all(tmem);
}

// 256 rows a unit where a chunk has more than 128 of them.
bool pair_rows(int max_q, int G) { return (long long)max_q * G > kTile; }

template <class T, int D, bool PAIR, bool CODES, bool REST>
sd_status launch(AttnParams &p, const CUtensorMap &k_map,
                 const CUtensorMap &v_map, int sms, char *ws,
                 cudaStream_t s) {
  using L = Layout<D, PAIR, CODES>;
  set_workspace(p, ws_layout(kMaxGrid, L::kRows, D), ws);
  const void *kernel = (const void *)attention_kernel<T, D, PAIR, CODES, REST>;
  int dev = 0;
  SDV_CUDA(cudaGetDevice(&dev));
  static std::atomic<unsigned long long> ready{0};
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    SDV_CUDA(cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)attn_smem<D, PAIR, CODES>()));
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  const unsigned grid = sms < kMaxGrid ? sms : kMaxGrid;
  void *args[] = {&p, const_cast<CUtensorMap *>(&k_map),
                  const_cast<CUtensorMap *>(&v_map)};
  sd_status st = launch_pdl(kernel, grid, attn_threads<CODES>(),
                            attn_smem<D, PAIR, CODES>(), s, args);
  if (st != SD_OK) return st;
  if (CODES && p.bf16)
    return launch_join<__nv_bfloat16, D, L::kRows>(p, grid, s);
  return launch_join<T, D, L::kRows>(p, grid, s);
}

}  // namespace
}  // namespace sdv
