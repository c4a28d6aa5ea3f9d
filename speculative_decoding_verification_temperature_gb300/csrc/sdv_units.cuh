// sdv_units.cuh -- what the kernels of chunk attention over a paged cache
// share, whatever type the cache holds: the units of work, their equal shares
// per CTA, the keys a row sees, and the kernel that joins the parts of units
// that were cut.
#pragma once

#include "sdv_paged.cuh"
#include "sdv_tcgen05.cuh"

namespace sdv {
namespace {

constexpr int kTile = 128;  // keys per tile
constexpr float kLn2 = 0.693147180559945f;

struct UnitParams {
  const int32_t *q_start, *kv_len, *block_table, *mask;
  int mask_words;
  int B, total, Hq, Hkv, G;
  FastDiv by_G, by_page;
  int page_size, max_pages;
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
__device__ __forceinline__ Chunk attn_chunk(const UnitParams &p, int b) {
  Chunk c = load_chunk(p.q_start, p.kv_len, b, p.total,
                       (long long)p.max_pages * p.page_size);
  if (p.mask && c.n > 32LL * p.mask_words) c.usable = false;
  return c;
}

template <int ROWS>
__device__ __forceinline__ int row_tiles(const UnitParams &p,
                                         const Chunk &c) {
  return c.usable ? (c.n * p.G + ROWS - 1) / ROWS : 0;
}

// Key tiles that row tile t sees.
template <int ROWS, int KEYS = kTile>
__device__ __forceinline__ int key_tiles(const UnitParams &p, const Chunk &c,
                                         int t) {
  int last = c.kv - 1;
  if (!p.mask) {
    const int i = div_by((t + 1) * ROWS - 1, p.by_G);
    if (i < c.n - 1) last = c.kv - c.n + i;
  }
  return last / KEYS + 1;
}

template <int ROWS, int KEYS = kTile>
__device__ unsigned long long head_tiles(const UnitParams &p,
                                         const Chunk &c) {
  const int T = row_tiles<ROWS>(p, c);
  unsigned long long s = 0;
  for (int t = 0; t < T; ++t) s += key_tiles<ROWS, KEYS>(p, c, t);
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

template <int ROWS, int KEYS = kTile>
__device__ void make_plan(const UnitParams &p, Plan &s) {
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
      const unsigned long long w = head_tiles<ROWS, KEYS>(p, c) * p.Hkv;
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
        w = (head_tiles<ROWS, KEYS>(p, c) + extra * row_tiles<ROWS>(p, c)) *
            p.Hkv;
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
          head_tiles<ROWS, KEYS>(p, c) + extra * row_tiles<ROWS>(p, c);
      unsigned long long r = s.x0 - lo;
      s.h = (int)(r / per);
      r %= per;
      int t = 0;
      for (;; ++t) {
        const int k = key_tiles<ROWS, KEYS>(p, c, t) + (int)extra;
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
template <int ROWS, int KEYS = kTile> struct Units {
  const UnitParams &p;
  unsigned long long left;  // places of the share from `at` on
  Chunk c;
  static constexpr int extra = unit_cost<ROWS>();
  int b, h, t, T, at;
  int j0, j1, nk;   // key tiles [j0, j1) of the unit's nk
  int rows;         // valid rows of the tile
  int count;        // units begun

  __device__ Units(const UnitParams &p_, const Plan &s)
      : p(p_), left(s.x1 - s.x0), b(s.b), h(s.h), t(s.t), T(0), at(s.at),
        count(0) {
    if (!left) return;
    c = attn_chunk(p, b);
    T = row_tiles<ROWS>(p, c);
    set();
    if (j0 == j1) next();
  }
  // The part of the share from place `from` on, `n` places long.
  __device__ Units(const UnitParams &p_, const Plan &s,
                   unsigned long long from, unsigned long long n)
      : p(p_), left(s.x1 - s.x0), b(s.b), h(s.h), t(s.t), T(0), at(s.at),
        count(0) {
    if (!n) left = 0;
    if (!left) return;
    c = attn_chunk(p, b);
    T = row_tiles<ROWS>(p, c);
    for (;;) {
      set();
      const int here = nk + extra - at;
      if (from < (unsigned long long)here) break;
      from -= here;
      step();
    }
    at += (int)from;
    left = n;
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
    nk = key_tiles<ROWS, KEYS>(p, c, t);
    j0 = max(0, at - extra);
    j1 = max(0, at + places() - extra);
    rows = min(c.n * p.G - t * ROWS, ROWS);
  }
  __device__ void step() {  // to the start of the unit after this one
    at = 0;
    if (++t == T) {
      t = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {  // there is one: a later sequence has units
          c = attn_chunk(p, ++b);
          T = row_tiles<ROWS>(p, c);
        } while (T == 0);
      }
    }
  }
  __device__ void next() {
    do {  // past units of which the share has no tile
      left -= places();
      if (!left) return;
      step();
      set();
    } while (j0 == j1);
  }
};

// Bits of the 32 keys from `key` on that a row sees.  Causal: keys up to
// `limit`.  Tree: the prefix, and the chunk's tokens in its mask.
__device__ __forceinline__ uint32_t seen_bits(const UnitParams &p,
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

// What a part with reference ml.x and sum ml.y counts beside a reference m: 0
// if it saw nothing (or is none), NaN if its sum is NaN.
__device__ __forceinline__ float part_weight(float2 ml, float m) {
  return ml.x == -kInf ? (ml.y == ml.y ? 0.f : ml.y) : ex2(ml.x - m);
}

// A row of a cut unit from its parts (a warp), kAhead of them read at once.
template <class T, int D, int ROWS, int kAhead>
__device__ __forceinline__ void join_row(const UnitParams &p,
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
    const float w = part_weight(ml, m);  // of part k0 + lane
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
join_kernel(const __grid_constant__ UnitParams p) {
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

// The join after an attention kernel of `grid` CTAs.
template <class T, int D, int ROWS, int KEYS = kTile>
sd_status launch_join(UnitParams &p, unsigned grid, cudaStream_t s) {
  // a sequence whose table holds one key tile has no unit that can be cut
  if ((long long)p.max_pages * p.page_size <= KEYS) return SD_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, ROWS / kWarps, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *args[] = {&p};
  SDV_CUDA(cudaLaunchKernelExC(&cfg, (const void *)join_kernel<T, D, ROWS>,
                               args));
  return SD_OK;
}

// Workspace of an attention kernel of up to `grid` CTAs: a record, and (m, l)
// and O of two cut units, per CTA.
struct WsLayout {
  size_t ml, o, bytes;
};
inline WsLayout ws_layout(int grid, int rows, int D) {
  WsLayout w;
  w.ml = (grid * sizeof(CutUnit) + 255) / 256 * 256;
  w.o = w.ml + (size_t)grid * 2 * rows * sizeof(float2);
  w.bytes = w.o + (size_t)grid * 2 * rows * D * sizeof(float);
  return w;
}
inline void set_workspace(UnitParams &p, const WsLayout &w, void *ws) {
  char *at = static_cast<char *>(ws);
  p.cut = reinterpret_cast<CutUnit *>(at);
  p.part_ml = reinterpret_cast<float2 *>(at + w.ml);
  p.part_o = reinterpret_cast<float *>(at + w.o);
}

}  // namespace
}  // namespace sdv
