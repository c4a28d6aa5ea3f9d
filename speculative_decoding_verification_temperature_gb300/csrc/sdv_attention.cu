// sdv_attention.cu -- sd_paged_attention: a chunk of new tokens attends
// over the paged cache.
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
// A wait that gives up (see role_wait) stops the loads and the products; all
// other steps go on over meaningless data to the end of the share, so that
// every barrier between warps is reached.
#include <cuda.h>

#include <atomic>

#include "sdv_paged.cuh"
#include "sdv_tcgen05.cuh"

namespace sdv {
namespace {

constexpr int kTile = 128;       // keys per tile, rows per stream
constexpr int kHalf = kTile / 2;  // keys a softmax thread weighs at a time
constexpr int kMaxGrid = 160;    // CTAs the workspace is laid out for
constexpr int kAttnThreads = 384;  // two warpgroups of softmax, one of roles
constexpr int kMmaWarp = 9;  // and 10; warps 8 and 11 load
constexpr int kBadRing = 64;     // units whose bad-page mark is kept
constexpr float kLn2 = 0.693147180559945f;
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

struct AttnParams {
  const void *q;
  long long q_stride;
  const int32_t *q_start, *kv_len, *block_table, *mask;
  int mask_words;
  int B, total, Hq, Hkv, G;
  FastDiv by_G, by_page;
  int num_pages, page_size, max_pages;
  int box;  // rows of one TMA box: a power of two that divides the page
  float scale_log2;  // scale x log2(e)
  void *out;
  float *lse;
  int32_t *dev_status;
  // workspace: records of cut units, (m, l) and O of the parts
  struct CutUnit *cut;
  float2 *part_ml;
  float *part_o;
};

// A unit whose key range is cut: part 0 is slot 1 of the CTA that starts
// it, part k slot 0 of the k-th CTA after it.
struct CutUnit {
  int parts, rows;     // rows: valid rows of the tile
  int start, head;     // packed row of the sequence, cache head
  int first;           // first row of the tile in (token, group) order
};

// ------------------------------------------------------------ work units
__device__ __forceinline__ Chunk attn_chunk(const AttnParams &p, int b) {
  Chunk c = load_chunk(p.q_start, p.kv_len, b, p.total,
                       (long long)p.max_pages * p.page_size);
  if (p.mask && c.n > 32LL * p.mask_words) c.usable = false;
  return c;
}

template <int ROWS>
__device__ __forceinline__ int row_tiles(const AttnParams &p,
                                         const Chunk &c) {
  return c.usable ? (c.n * p.G + ROWS - 1) / ROWS : 0;
}

// Key tiles that row tile t sees.
template <int ROWS>
__device__ __forceinline__ int key_tiles(const AttnParams &p, const Chunk &c,
                                         int t) {
  int last = c.kv - 1;
  if (!p.mask) {
    const int i = div_by((t + 1) * ROWS - 1, p.by_G);
    if (i < c.n - 1) last = c.kv - c.n + i;
  }
  return last / kTile + 1;
}

template <int ROWS>
__device__ unsigned long long head_tiles(const AttnParams &p,
                                         const Chunk &c) {
  const int T = row_tiles<ROWS>(p, c);
  unsigned long long s = 0;
  for (int t = 0; t < T; ++t) s += key_tiles<ROWS>(p, c, t);
  return s;
}

// Starting and ending a unit costs a CTA about as much as this many key
// tiles: it counts into the shares, so that many short units and few long
// ones take the same time (two prompt chunks, one over 8192 cached keys and
// one over 2385: 589 us by tiles alone, 549 with 8, 554 with 12; 8 trees of
// 64 nodes 53 and 48, 8 prompts of up to 700 tokens 99 and 83).
template <int ROWS> constexpr int unit_cost() { return ROWS == 256 ? 8 : 1; }

// The plan of one CTA.  All units are laid end to end, each `extra` places
// for itself and then one for each key tile; the CTA's share is [x0, x1).
struct Plan {
  unsigned long long total, x0, x1;
  unsigned long long warp_sum[8], warp_units[8];
  int n, b, h, t, at;  // shares; the unit where x0 lies, and the place in it
  int any_unusable;
};

template <int ROWS>
__device__ void make_plan(const AttnParams &p, Plan &s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // key tiles and units of this thread's sequences; of its first one
  unsigned long long tiles = 0, units = 0, first_tiles = 0, first_units = 0;
  bool unusable = false;
  if (tid < 256)
    for (int b = tid; b < p.B; b += 256) {
      const Chunk c = attn_chunk(p, b);
      if (c.n > 0 && !c.usable) unusable = true;
      if (!c.rows_ok) {
        unusable = true;
        if (blockIdx.x == 0) status_or(p.dev_status, SD_DEV_BAD_LENGTH);
      }
      const unsigned long long w = head_tiles<ROWS>(p, c) * p.Hkv;
      const unsigned long long k =
          (unsigned long long)row_tiles<ROWS>(p, c) * p.Hkv;
      if (b == tid) first_tiles = w, first_units = k;
      tiles += w;
      units += k;
    }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    tiles += __shfl_xor_sync(~0u, tiles, d);
    units += __shfl_xor_sync(~0u, units, d);
  }
  if (lane == 0 && warp < 8) {
    s.warp_sum[warp] = tiles;
    s.warp_units[warp] = units;
  }
  if (tid == 0) s.b = -1;
  const int any = __syncthreads_or(unusable);
  if (tid == 0) {
    unsigned long long w = 0, k = 0;
    for (int i = 0; i < 8; ++i) {
      w += s.warp_sum[i];
      k += s.warp_units[i];
    }
    w += k * unit_cost<ROWS>();
    s.total = w;
    s.any_unusable = any;
    s.n = w < gridDim.x ? (int)w : (int)gridDim.x;
    s.x0 = s.x1 = 0;
    if ((int)blockIdx.x < s.n) {
      s.x0 = w * blockIdx.x / s.n;
      s.x1 = w * (blockIdx.x + 1) / s.n;
    }
  }
  __syncthreads();
  if (s.x0 == s.x1) return;
  constexpr unsigned long long extra = unit_cost<ROWS>();
  unsigned long long carry = 0;
  for (int base = 0; base < p.B; base += 256) {
    unsigned long long w = first_tiles + extra * first_units;
    if (base > 0) {
      w = 0;
      if (tid < 256 && base + tid < p.B) {
        const Chunk c = attn_chunk(p, base + tid);
        w = (head_tiles<ROWS>(p, c) + extra * row_tiles<ROWS>(p, c)) * p.Hkv;
      }
    }
    unsigned long long inc = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long o = __shfl_up_sync(~0u, inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 31 && warp < 8) s.warp_sum[warp] = inc;
    __syncthreads();
    unsigned long long all = 0, before = carry;
    for (int i = 0; i < 8; ++i) {
      if (i < warp) before += s.warp_sum[i];
      all += s.warp_sum[i];
    }
    const unsigned long long lo = before + inc - w;
    if (tid < 256 && s.x0 >= lo && s.x0 < lo + w) {
      const Chunk c = attn_chunk(p, base + tid);
      const unsigned long long per =
          head_tiles<ROWS>(p, c) + extra * row_tiles<ROWS>(p, c);
      unsigned long long r = s.x0 - lo;
      s.h = (int)(r / per);
      r %= per;
      int t = 0;
      for (;; ++t) {
        const int k = key_tiles<ROWS>(p, c, t) + (int)extra;
        if (r < (unsigned long long)k) break;
        r -= k;
      }
      s.b = base + tid;
      s.t = t;
      s.at = (int)r;
    }
    carry += all;
    __syncthreads();
    if (s.b >= 0) break;
  }
}

// Walks the units of a CTA's share that it has key tiles of; every warp
// walks the same ones.
template <int ROWS> struct Units {
  const AttnParams &p;
  unsigned long long left;  // places of the share from `at` on
  Chunk c;
  static constexpr int extra = unit_cost<ROWS>();
  int b, h, t, T, at;
  int j0, j1, nk;   // key tiles [j0, j1) of the unit's nk
  int rows;         // valid rows of the tile
  int count;        // units begun

  __device__ Units(const AttnParams &p_, const Plan &s)
      : p(p_), left(s.x1 - s.x0), b(s.b), h(s.h), t(s.t), T(0), at(s.at),
        count(0) {
    if (!left) return;
    c = attn_chunk(p, b);
    T = row_tiles<ROWS>(p, c);
    set();
    if (j0 == j1) next();
  }
  __device__ void to(const Units &o) {  // o walks the same share
    left = o.left, c = o.c, b = o.b, h = o.h, t = o.t, T = o.T, at = o.at;
    j0 = o.j0, j1 = o.j1, nk = o.nk, rows = o.rows, count = o.count;
  }
  __device__ int places() const {  // of the unit that are in the share
    const int n = nk + extra - at;
    return (unsigned long long)n < left ? n : (int)left;
  }
  __device__ void set() {
    ++count;
    nk = key_tiles<ROWS>(p, c, t);
    j0 = max(0, at - extra);
    j1 = max(0, at + places() - extra);
    rows = min(c.n * p.G - t * ROWS, ROWS);
  }
  __device__ void next() {
    do {  // past units of which the share has no tile
      left -= places();
      if (!left) return;
      at = 0;
      if (++t == T) {
        t = 0;
        if (++h == p.Hkv) {
          h = 0;
          do {  // left > 0: a later sequence has units
            c = attn_chunk(p, ++b);
            T = row_tiles<ROWS>(p, c);
          } while (T == 0);
        }
      }
      set();
    } while (j0 == j1);
  }
};

// --------------------------------------------------------- shared memory
// PAIR: 256 rows a unit, 128 a stream; otherwise both streams share 128.
template <int D, bool PAIR> struct Layout {
  static constexpr int kRows = PAIR ? 256 : 128;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQBytes = (PAIR ? 2 : 1) * kTileBytes;
  // Two rings of tiles, as many as fit: what is in flight covers the latency
  // of HBM.  PAIR: ring 0 holds the key tiles, ring 1 the value tiles, read
  // by both streams.  Otherwise ring st holds stream st's tiles in the order
  // it uses them (key, value, key, ...): a ring with one writer and one
  // reader, so that a stream that is ahead never takes a slot's earlier
  // filling for its own.
  static constexpr int kN0 = D == 128 ? 3 : PAIR ? 4 : 5;
  static constexpr int kN1 = D == 128 ? (PAIR ? 2 : 3) : PAIR ? 4 : 5;
  static constexpr size_t kTiles =
      kQBytes + (size_t)kTileBytes * (kN0 + kN1);
};

template <int D, bool PAIR> struct Shared {
  using L = Layout<D, PAIR>;
  uint64_t full[2][L::kN0], empty[2][L::kN0];
  uint64_t q_full[2], s_full[2], turn[2], drain[2];
  uint64_t w_full[2][2], o_full[2][2];  // of a stream's tile halves
  uint64_t idle;  // stream 1 has no tile: its product warp saw the queries
  uint32_t tmem;
  volatile int abort;
  int bad[kBadRing];  // unit count whose pages were bad
  float2 ml[2][PAIR ? 1 : kTile];
  Plan plan;
};
template <int D, bool PAIR> constexpr size_t attn_smem() {
  return Layout<D, PAIR>::kTiles + sizeof(Shared<D, PAIR>);
}

// A barrier of the two softmax warpgroups alone.
__device__ __forceinline__ void streams_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

// 32 bytes, at a multiple of 32: whole sectors even where each lane writes
// a row of its own.
__device__ __forceinline__ void st_v8(void *to, const uint32_t *x) {
  asm volatile(
      "st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to),
      SDV_I8(x, 0)
      : "memory");
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t u;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
  return u;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t u;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(hi), "f"(lo));
  return u;
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

// Bits of the 32 keys from `key` on that a row sees.  Causal: keys up to
// `limit`.  Tree: the prefix, and the chunk's tokens in its mask.
__device__ __forceinline__ uint32_t seen_bits(const AttnParams &p,
                                              const Chunk &c, int token,
                                              int limit, int key) {
  const int ctx = c.kv - c.n;
  const int end = (p.mask ? c.kv - 1 : limit) - key;  // last bit in range
  if (end < 0) return 0;
  const uint32_t in = end >= 31 ? ~0u : (2u << end) - 1;
  if (!p.mask) return in;
  const int x = key - ctx;  // the chunk's token at bit 0
  if (x <= -32) return in;
  const int32_t *m = p.mask + (long long)(c.start + token) * p.mask_words;
  uint32_t bits;
  if (x < 0) {
    bits = ((1u << -x) - 1) | (uint32_t)__ldg(m) << -x;
  } else {
    const int w = x >> 5;
    const uint32_t lo = w < p.mask_words ? (uint32_t)__ldg(m + w) : 0;
    const uint32_t hi = w + 1 < p.mask_words ? (uint32_t)__ldg(m + w + 1) : 0;
    bits = __funnelshift_r(lo, hi, x & 31);
  }
  return bits & in;
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
template <class T, int D, bool HIDE, bool REST>
__device__ __forceinline__ bool weigh_tile(Row &row, const uint32_t *seen,
                                           uint64_t *w_full, uint64_t *o_full,
                                           bool first, uint32_t parity,
                                           volatile int *abort,
                                           int32_t *dev_status) {
  using S = Scale<T>;
  uint32_t x[2][32];
  tmem_ld32(row.s_addr, x[0]);
#pragma unroll
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

// ------------------------------------------------------------- the kernel
template <class T, int D, bool PAIR>
__global__ void __launch_bounds__(kAttnThreads, 1)
attention_kernel(const __grid_constant__ AttnParams p,
                 const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map) {
  using L = Layout<D, PAIR>;
  constexpr int ROWS = L::kRows;
  constexpr bool REST = !PAIR;
  constexpr bool BF16 = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) char dyn[];  // swizzled tiles first
  Shared<D, PAIR> &s = *reinterpret_cast<Shared<D, PAIR> *>(dyn + L::kTiles);
  char *q_tile = dyn;
  char *ring[2] = {q_tile + L::kQBytes,
                   q_tile + L::kQBytes + L::kN0 * L::kTileBytes};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i)
      for (int k = 0; k < L::kN0; ++k) {
        mbar_init(&s.full[i][k], 1);
        mbar_init(&s.empty[i][k], PAIR ? 2 : 1);  // the streams that read it
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
  if (warp == 8 && lane == 0) {
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

  // 384 threads start with 168 registers each; a softmax thread holds much of
  // a row, a role next to nothing: 256 x 208 + 128 x 88 = 384 x 168
  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  if (warp >= 8) {
    Units<ROWS> u(p, s.plan);
    if (warp == 8 || warp == 11) {
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
        if (from < kTile) {
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
    const float sl = p.scale_log2;
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
      const T *src = (const T *)p.q + v.c.start * p.q_stride +
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
        *reinterpret_cast<uint4 *>(dst + n * 128 +
                                   (((ch & 7) ^ (n & 7)) << 4)) = x[i];
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_full[PAIR ? st : 0]);
    };
    if (u.left) load_q(u);
    while (u.left) {
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
          const T *q = (const T *)p.q + (next.c.start + tok) * p.q_stride +
                       (next.h * p.G + at - tok * p.G) * D;
#pragma unroll
          for (int e = 0; e < D; e += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q + e));
        }
      }
      const int cnt_all = u.j1 - u.j0;
      const int cnt =
          !active(u) ? 0 : PAIR ? cnt_all : (cnt_all - st + 1) / 2;
      const int row_at = u.t * ROWS + base_row + r;
      const bool mine = base_row + r < u.rows;
      const bool warp_rows = base_row + (warp & 3) * 32 < u.rows;
      const int token = mine ? div_by(row_at, p.by_G) : 0;
      const int ctx = u.c.kv - u.c.n, limit = ctx + token;
      Row row = {tmem + lanes + st * kTile,
                 tmem + lanes + 2 * kTile + st * D, sl, -kInf, 0.f};
      for (int i = 0; i < cnt; ++i, ++tn) {
        const int j = u.j0 + (PAIR ? i : 2 * i + st);
        fine = role_wait(&s.s_full[st], tn & 1, &s.abort, p.dev_status);
        if (!__all_sync(~0u, fine)) { fine = false; break; }
        if (warp_rows) {
          tmem_fence_after();
          // only tiles past the row's last key hide anything
          const int key = j * kTile;
          const bool cuts = __any_sync(
              ~0u, key + kTile - 1 > (p.mask ? ctx - 1 : limit));
          uint32_t seen[kTile / 32] = {};
          if (cuts) {
#pragma unroll
            for (int c = 0; c < kTile / 32; ++c)
              seen[c] =
                  mine ? seen_bits(p, u.c, token, limit, key + 32 * c) : 0;
          }
          __syncwarp();
          if (i == 0) row.m = row_max(row.s_addr, cuts, seen);
          fine = cuts ? weigh_tile<T, D, true, REST>(row, seen, s.w_full[st],
                                               s.o_full[st], i == 0, tn & 1,
                                               &s.abort, p.dev_status)
                      : weigh_tile<T, D, false, REST>(row, seen, s.w_full[st],
                                                s.o_full[st], i == 0, tn & 1,
                                                &s.abort, p.dev_status);
          if (!fine) break;
        } else if (lane == 0) {
          mbar_arrive(&s.w_full[st][0]);
          mbar_arrive(&s.w_full[st][1]);
        }
      }
      // ---- the end of the unit.  The last scores are out, so the next
      // unit's queries may replace this one's: its first scores are under
      // way while this one's rows are written
      if (PAIR && next.left) load_q(next);
      if (cnt > 0) {
        role_wait(&s.o_full[st][1], (tn - 1) & 1, &s.abort, p.dev_status);
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
      const bool second = !PAIR && cnt_all > 1;
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
        T *out = (T *)p.out + to * D + c_lo;
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
              w[e] = pack2<T>(o[2 * e], o[2 * e + 1]);
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
      for (long long i = tid; i < n * D; i += kAttnThreads)
        ((T *)p.out)[lo * D + i] = narrow<T>(__int_as_float(0x7fc00000));
      if (p.lse)
        for (long long i = tid; i < n; i += kAttnThreads)
          p.lse[lo + i] = __int_as_float(0x7fc00000);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_free_all(tmem);
}

// A row of a cut unit from its parts (a warp), kAhead of them read at once.
template <class T, int D, int ROWS, int kAhead>
__device__ __forceinline__ void join_row(const AttnParams &p,
                                         const CutUnit &cut, int r,
                                         int lane) {
  auto slot = [&](int k) {
    return ((long long)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * ROWS + r;
  };
  constexpr int E = D / 32;
  auto part = [&](int k) {
    return k < cut.parts ? p.part_ml[slot(k)] : make_float2(-kInf, 0.f);
  };
  float2 ml = part(lane);
  float m = ml.x;
  for (int k = lane + 32; k < cut.parts; k += 32) m = fmaxf(m, part(k).x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  float l = 0.f, o[E] = {};
  for (int k0 = 0; k0 < cut.parts; k0 += 32) {
    if (k0) ml = part(k0 + lane);
    // lane k has the weight of part k0 + k: 0 for one that saw nothing (or
    // is none), NaN for one with a NaN sum
    const float w = ml.x == -kInf ? (ml.y == ml.y ? 0.f : ml.y)
                                  : ex2(ml.x - m);
    l += ml.y * w;
    const int n = min(cut.parts - k0, 32);
    for (int k = 0; k < n; k += kAhead) {
      float x[kAhead][E];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float *src =
            p.part_o + slot(min(k0 + k + i, cut.parts - 1)) * D + lane * E;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4 *>(src);
          x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2 *>(src);
          x[i][0] = v.x, x[i][1] = v.y;
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float wk = __shfl_sync(~0u, w, k + i);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(x[i][e], wk, o[e]);
      }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
  const int at = cut.first + r, tok = div_by(at, p.by_G);
  const long long row = (long long)(cut.start + tok) * p.Hq +
                        cut.head * p.G + (at - tok * p.G);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t *dst = reinterpret_cast<uint32_t *>((T *)p.out + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    dst[e / 2] = pack2<T>(o[e] * inv, o[e + 1] * inv);
  if (p.lse && lane == 0)
    p.lse[row] = l == 0.f ? -kInf : (m + log2f(l)) * kLn2;
}

// Joins the parts of cut units: a warp per row.  Block (x, y): the unit that
// CTA x began, rows 8 y to 8 y + 7.  Where a long axis was cut into many parts
// it is a chain of waits for L2: one head of 64 with 81 tokens behind 40k, the
// whole call 50 us with parts read two at a time and 43 with sixteen.  Units
// of two or three parts, which most are, would read more than they have that
// way (64 tree nodes of 16 sequences: 73 us, two at a time 67).
template <class T, int D, int ROWS>
__global__ void __launch_bounds__(kThreads)
attention_join_kernel(const __grid_constant__ AttnParams p) {
  griddep_wait();
  const CutUnit cut = p.cut[blockIdx.x];
  const int r = blockIdx.y * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (cut.parts < 2 || r >= cut.rows) return;
  if (cut.parts > 4)
    join_row<T, D, ROWS, 16>(p, cut, r, lane);
  else
    join_row<T, D, ROWS, 2>(p, cut, r, lane);
}

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

struct WsLayout {
  size_t cut, ml, o, bytes;
};
WsLayout ws_layout(int rows, int D) {
  WsLayout w;
  w.cut = 0;
  w.ml = (kMaxGrid * sizeof(CutUnit) + 255) / 256 * 256;
  w.o = w.ml + (size_t)kMaxGrid * 2 * rows * sizeof(float2);
  w.bytes = w.o + (size_t)kMaxGrid * 2 * rows * D * sizeof(float);
  return w;
}

// 256 rows a unit where a chunk has more than 128 of them.
bool pair_rows(int max_q, int G) { return (long long)max_q * G > kTile; }

template <class T, int D, bool PAIR>
sd_status launch(AttnParams &p, const CUtensorMap &k_map,
                 const CUtensorMap &v_map, int sms, char *ws,
                 cudaStream_t s) {
  using L = Layout<D, PAIR>;
  const WsLayout w = ws_layout(L::kRows, D);
  p.cut = reinterpret_cast<CutUnit *>(ws + w.cut);
  p.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
  p.part_o = reinterpret_cast<float *>(ws + w.o);
  const void *kernel = (const void *)attention_kernel<T, D, PAIR>;
  int dev = 0;
  SDV_CUDA(cudaGetDevice(&dev));
  static std::atomic<unsigned long long> ready{0};
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    SDV_CUDA(cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)attn_smem<D, PAIR>()));
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  const unsigned grid = sms < kMaxGrid ? sms : kMaxGrid;
  void *args[] = {&p, const_cast<CUtensorMap *>(&k_map),
                  const_cast<CUtensorMap *>(&v_map)};
  sd_status st = launch_pdl(kernel, grid, kAttnThreads,
                            attn_smem<D, PAIR>(), s, args);
  if (st != SD_OK) return st;
  // a sequence whose table holds one key tile has no unit that can be cut
  if ((long long)p.max_pages * p.page_size <= kTile) return SD_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, L::kRows / kWarps, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *jargs[] = {&p};
  SDV_CUDA(cudaLaunchKernelExC(
      &cfg, (const void *)attention_join_kernel<T, D, L::kRows>, jargs));
  return SD_OK;
}

template <class T>
sd_status dispatch(AttnParams &p, int D, bool pair, const CUtensorMap &km,
                   const CUtensorMap &vm, int sms, char *ws, cudaStream_t s) {
  if (D == 64)
    return pair ? launch<T, 64, true>(p, km, vm, sms, ws, s)
                : launch<T, 64, false>(p, km, vm, sms, ws, s);
  return pair ? launch<T, 128, true>(p, km, vm, sms, ws, s)
              : launch<T, 128, false>(p, km, vm, sms, ws, s);
}

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_paged_attention_workspace(int q_heads, int heads,
                                               int head_dim, int max_q) {
  if (heads < 1 || q_heads < heads || (head_dim != 64 && head_dim != 128))
    return 256;
  return ws_layout(pair_rows(max_q, q_heads / heads) ? 256 : 128, head_dim)
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
