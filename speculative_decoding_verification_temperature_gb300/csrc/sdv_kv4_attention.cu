// sdv_kv4_attention.cu -- sd_kv4_attention: a chunk of new tokens attends
// over the 4-bit paged cache.
#include <atomic>

#include "sdv_kv4.cuh"
#include "sdv_units.cuh"

namespace sdv {
namespace {

struct Attn4Params : UnitParams {
  const void *q;
  long long q_stride;
  Kv4Cache c;
  float scale_log2;  // scale x log2(e)
};

// ------------------------------------------------------- few rows a head
//
// Where a cache head has few rows (one token of a group of query heads), a
// warp takes 16 keys at a time from the cache straight into registers and
// makes them operands there, with the keys as the rows of the products:
//   S^T [16 keys x 8 rows] = K [16 x D] Q^T,   O^T [D x 8] += V^T [D x 16] W
// so that 8 rows are not padded to more.  A thread's four neighbours hold one
// key's row: which elements of it a step of a product takes is free as long
// as the queries' operand takes the same.
//
// A row's weights are fp16, 2^kBias at its reference m, which moves up only
// when a score is 2^kSlack above it: at most 2^15, and a weight 2^-24 of the
// reference's still has all its bits.
constexpr float kBias = 10.f, kSlack = 5.f;
constexpr int kBlock = 16;  // keys of a warp's step

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0,
                                         uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 tile of 16-bit numbers, rows across lane groups, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D> struct Words {  // a thread's share of a key's row
  uint32_t w[D / 32];
};
template <int D>
__device__ __forceinline__ Words<D> ld_words(const char *p) {
  Words<D> r;
  if constexpr (D == 128) {
    asm("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
        : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
        : "l"(p));
  } else {
    asm("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
        : "=r"(r.w[0]), "=r"(r.w[1])
        : "l"(p));
  }
  return r;
}
template <int D>
__device__ __forceinline__ void ld_half_words(const char *p, uint32_t *w) {
  if constexpr (D == 128) {
    asm("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
        : "=r"(w[0]), "=r"(w[1])
        : "l"(p));
  } else {
    asm("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
  }
}

// 16 keys on their way: the thread's quarter of keys g and g + 8, and its
// eighth of the values 2 t, 2 t + 1, 2 t + 8, 2 t + 9.
template <int D> struct Stage {
  Words<D> k[2];
  uint32_t ks[2];
  uint32_t v[4][D / 64];
  uint32_t vs[4];
};

template <int ROWS, int D, int WARPS> struct Shared4 {
  Plan plan;
  int bad;
  float q_scale[ROWS];
  float2 ml[WARPS][ROWS];
  uint32_t q[ROWS][D / 2 + 4];
  alignas(16) float o[WARPS][ROWS][D + 4];
};

// The queries of a unit as fp16 rows in shared memory (rows that are none:
// zeros), bf16 ones times a power of two that takes the row's largest to
// [2^14, 2^15): exact but for elements 2^-28 of that and below.  A row with
// NaN or infinity gets a NaN factor.
template <class T, int D, int ROWS, int WARPS>
__device__ __forceinline__ void load_queries(const Attn4Params &p,
                                             const Units<ROWS> &u,
                                             Shared4<ROWS, D, WARPS> &s) {
  constexpr int E = D / 64;  // words a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < ROWS; r += WARPS) {
    uint32_t w[E] = {};
    float f = p.scale_log2;
    if (r < u.rows) {
      const int at = u.t * ROWS + r, tok = div_by(at, p.by_G);
      const T *src = (const T *)p.q + (u.c.start + tok) * p.q_stride +
                     (long long)(u.h * p.G + at - tok * p.G) * D;
      const uint32_t *x = reinterpret_cast<const uint32_t *>(src) + lane * E;
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        w[e] = __ldg(x + e);
        top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
      }
      top = __reduce_max_sync(~0u, top);
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        // exponents above -86: the power is a normal number
        const int exp = max((int)(top >> 7), 41) - 127;
        const float up = __uint_as_float((uint32_t)(14 - exp + 127) << 23);
        f *= __uint_as_float((uint32_t)(exp - 14 + 127) << 23);
        if (top >= 0x7f80u) f = __int_as_float(0x7fc00000);
#pragma unroll
        for (int e = 0; e < E; ++e)
          w[e] = pack2<__half>(__uint_as_float(w[e] << 16) * up,
                               __uint_as_float(w[e] & 0xffff0000u) * up);
      } else if (top >= 0x7c00u) {
        f = __int_as_float(0x7fc00000);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s.q[r][lane * E + e] = w[e];
    if (lane == 0) s.q_scale[r] = f;
  }
}

template <class T, int D, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, NT == 1 ? 2 : 1)
kv4_rows_kernel(const __grid_constant__ Attn4Params p) {
  constexpr int ROWS = 8 * NT, W = D / 32;  // W: words of a key a thread
  using S = Shared4<ROWS, D, WARPS>;
  extern __shared__ __align__(16) char dyn[];
  S &s = *reinterpret_cast<S *>(dyn);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  griddep_wait();
  make_plan<ROWS>(p, s.plan);
  if (tid == 0) {
    s.bad = 0;
    p.cut[blockIdx.x].parts = 0;
  }
  __syncthreads();
  Units<ROWS> u(p, s.plan);
  const int k_group = (t * (D / 4)) >> p.c.shift;
  const int v_group = (g * (D / 8)) >> p.c.shift;
  for (; u.left; u.next()) {
    if (tid == 0 && u.j0 == 0 && u.j1 < u.nk) {
      // this CTA's last unit goes on in the CTAs up to the one whose share
      // holds the unit's last tile
      const unsigned long long end = s.plan.x1 + (unsigned)(u.nk - u.j1);
      CutUnit cut;
      cut.parts = (int)((end * s.plan.n - 1) / s.plan.total) -
                  (int)blockIdx.x + 1;
      cut.rows = u.rows;
      cut.start = u.c.start;
      cut.head = u.h;
      cut.first = u.t * ROWS;
      p.cut[blockIdx.x] = cut;
    }
    load_queries<T, D, ROWS, WARPS>(p, u, s);
    __syncthreads();
    const int32_t *table = p.block_table + (long long)u.b * p.max_pages;
    const int end = min(u.j1 * kTile, u.c.kv);
    bool bad = false;

    auto page_of = [&](int key, int &tok) {  // key: a multiple of 8
      const int n = div_by(key, p.by_page);
      tok = key - n * p.page_size;
      if (key >= end) return -1;
      const int id = __ldg(table + n);
      return id >= 0 && id < p.c.num_pages ? id : -2;
    };
    auto fetch = [&](int key, Stage<D> &x, const int (&page)[2],
                     const int (&tok)[2]) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        x.ks[hf] = x.vs[2 * hf] = x.vs[2 * hf + 1] = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) x.k[hf].w[i] = 0;
#pragma unroll
        for (int i = 0; i < W / 2; ++i)
          x.v[2 * hf][i] = x.v[2 * hf + 1][i] = 0;
        if (page[hf] >= 0) {
          const long long at = (long long)u.h * p.page_size + tok[hf];
          const char *kc =
              p.c.k + page[hf] * p.c.page_stride + at * (D / 2);
          const char *vc =
              p.c.v + page[hf] * p.c.page_stride + at * (D / 2);
          const char *kp = p.c.k_scale + page[hf] * p.c.scale_stride +
                           at * p.c.scale_bytes;
          const char *vp = p.c.v_scale + page[hf] * p.c.scale_stride +
                           at * p.c.scale_bytes;
          x.k[hf] = ld_words<D>(kc + g * (D / 2) + t * (D / 8));
          ld_half_words<D>(vc + 2 * t * (D / 2) + g * (D / 16), x.v[2 * hf]);
          ld_half_words<D>(vc + (2 * t + 1) * (D / 2) + g * (D / 16),
                           x.v[2 * hf + 1]);
          // what lies past the sequence's keys counts as zeros
          const int k0 = key + 8 * hf;
          if (k0 + g < end)
            x.ks[hf] = __ldg(reinterpret_cast<const uint32_t *>(
                kp + g * p.c.scale_bytes + 4 * k_group));
          if (k0 + 2 * t < end)
            x.vs[2 * hf] = __ldg(reinterpret_cast<const uint32_t *>(
                vp + 2 * t * p.c.scale_bytes + 4 * v_group));
          if (k0 + 2 * t + 1 < end)
            x.vs[2 * hf + 1] = __ldg(reinterpret_cast<const uint32_t *>(
                vp + (2 * t + 1) * p.c.scale_bytes + 4 * v_group));
        } else if (page[hf] == -2) {
          bad = true;
        }
      }
    };

    // the queries' operand: the thread's quarter of rows g (and g + 8)
    uint32_t qf[NT][2 * W * 2];
    float rs[NT][2], m[NT][2], l[NT][2];
    int limit[NT][2];
    const int ctx = u.c.kv - u.c.n;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 4 * W; ++i) qf[n][i] = s.q[8 * n + g][t * 4 * W + i];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        rs[n][e] = s.q_scale[r];
        m[n][e] = -kInf;
        l[n][e] = 0.f;
        limit[n][e] =
            ctx + div_by(u.t * ROWS + min(r, u.rows - 1), p.by_G);
      }
    }
    float o[NT][W * 2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2 * W; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    const int open = p.mask ? ctx : ctx + div_by(u.t * ROWS, p.by_G) + 1;

    auto use = [&](int key, const Stage<D> &x) {
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
      const uint32_t a0 = both_lo(x.ks[0]), b0 = both_hi(x.ks[0]);
      const uint32_t a1 = both_lo(x.ks[1]), b1 = both_hi(x.ks[1]);
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const uint32_t f0 = kv4_fma(kv4_codes(x.k[0].w[i], j), a0, b0);
          const uint32_t f1 = kv4_fma(kv4_codes(x.k[1].w[i], j), a1, b1);
          const uint32_t f2 = kv4_fma(kv4_codes(x.k[0].w[i], j + 1), a0, b0);
          const uint32_t f3 = kv4_fma(kv4_codes(x.k[1].w[i], j + 1), a1, b1);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816(sc[n], f0, f1, f2, f3, qf[n][4 * i + j],
                     qf[n][4 * i + j + 1]);
        }
      // scores in powers of two; those a row does not see become -inf
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] *= rs[n][e & 1];
      if (key + kBlock > open) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = key + g + (e >> 1) * 8;
            bool see = k <= limit[n][e & 1];
            if (p.mask) {
              see = k < end;
              const int i = k - ctx;
              if (see && i >= 0)
                see = i < 32 * p.mask_words &&
                      (__ldg(p.mask +
                             (long long)(u.c.start + limit[n][e & 1] - ctx) *
                                 p.mask_words +
                             (i >> 5)) >>
                           (i & 31) &
                       1);
            }
            if (!see) sc[n][e] = -kInf;
          }
      }
      bool move = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          move = move || fmaxf(sc[n][e], sc[n][e + 2]) > m[n][e] + kSlack;
      if (__any_sync(~0u, move)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(sc[n][e], sc[n][e + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
              top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            if (top > m[n][e] + kSlack) {
              const float f = ex2(m[n][e] - top);  // 0 from -inf
              m[n][e] = top;
              l[n][e] *= f;
#pragma unroll
              for (int i = 0; i < 2 * W; ++i) {
                o[n][i][e] *= f;
                o[n][i][e + 2] *= f;
              }
            }
          }
      }
      uint32_t w[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[n][e & 1];
          z[e] = ex2(sc[n][e] - (ref == -kInf ? 0.f : ref - kBias));
          l[n][e & 1] += z[e];
        }
        w[n][0] = transpose8(pack2<__half>(z[0], z[1]));
        w[n][1] = transpose8(pack2<__half>(z[2], z[3]));
      }
      // values of two keys at a time: their codes are brought together first
      uint32_t va[2], vb[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        va[hf] = __byte_perm(x.vs[2 * hf], x.vs[2 * hf + 1], 0x5410);
        vb[hf] = __byte_perm(x.vs[2 * hf], x.vs[2 * hf + 1], 0x7632);
      }
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        uint32_t lo[2], hi[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          lo[hf] = __byte_perm(x.v[2 * hf][i], x.v[2 * hf + 1][i], 0x5410);
          hi[hf] = __byte_perm(x.v[2 * hf][i], x.v[2 * hf + 1][i], 0x7632);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // elements 8 i + 2 j (rows g) and 8 i + 2 j + 1 (rows g + 8)
          const uint32_t f0 = kv4_fma(kv4_codes(lo[0], j), va[0], vb[0]);
          const uint32_t f1 = kv4_fma(kv4_codes(hi[0], j), va[0], vb[0]);
          const uint32_t f2 = kv4_fma(kv4_codes(lo[1], j), va[1], vb[1]);
          const uint32_t f3 = kv4_fma(kv4_codes(hi[1], j), va[1], vb[1]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816(o[n][4 * i + j], f0, f1, f2, f3, w[n][0], w[n][1]);
        }
      }
    };

    // a warp's blocks are WARPS apart; two are on their way, and the pages of
    // a third
    constexpr int STEP = WARPS * kBlock;
    Stage<D> x[2];
    int page[2], tok[2];
    int key = u.j0 * kTile + warp * kBlock;
    auto look = [&](int at) {
      page[0] = page_of(at, tok[0]);
      page[1] = page_of(at + 8, tok[1]);
    };
    look(key);
    fetch(key, x[0], page, tok);
    look(key + STEP);
    while (key < end) {
      fetch(key + STEP, x[1], page, tok);
      look(key + 2 * STEP);
      use(key, x[0]);
      key += STEP;
      if (key >= end) break;
      fetch(key + STEP, x[0], page, tok);
      look(key + 2 * STEP);
      use(key, x[1]);
      key += STEP;
    }

    // ---- the warps' sums of the unit are joined
    if (__any_sync(~0u, bad) && lane == 0) {
      s.bad = 1;
      status_or(p.dev_status, SD_DEV_BAD_PAGE);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
          sum += __shfl_xor_sync(~0u, sum, d);
        const int r = 8 * n + 2 * t + e;
        if (g == 0) s.ml[warp][r] = make_float2(m[n][e], sum);
        // element 2 i of the thread's eighth is in o[i][e], 2 i + 1 in
        // o[i][e + 2]
#pragma unroll
        for (int i = 0; i < 2 * W; i += 2)
          *reinterpret_cast<float4 *>(
              &s.o[warp][r][g * (D / 8) + 2 * i]) =
              make_float4(o[n][i][e], o[n][i][e + 2], o[n][i + 1][e],
                          o[n][i + 1][e + 2]);
      }
    __syncthreads();
    const bool whole = u.j0 == 0 && u.j1 == u.nk;
    constexpr int E = D / 32;
    for (int r = warp; r < u.rows; r += WARPS) {
      float top = -kInf, sum = 0.f, out[E] = {};
#pragma unroll
      for (int k = 0; k < WARPS; ++k) top = fmaxf(top, s.ml[k][r].x);
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        const float2 a = s.ml[k][r];
        // 0 for a warp that saw nothing, NaN for one with a NaN sum
        const float f = a.x == -kInf ? (a.y == a.y ? 0.f : a.y)
                                     : ex2(a.x - top);
        sum += a.y * f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float y = s.o[k][r][lane * E + e];
          if (f != 0.f) out[e] = fmaf(y, f, out[e]);
        }
      }
      if (s.bad) sum = __int_as_float(0x7fc00000);
      const int at = u.t * ROWS + r, token = div_by(at, p.by_G);
      if (whole) {
        const long long to = (long long)(u.c.start + token) * p.Hq +
                             u.h * p.G + at - token * p.G;
        const float inv = 1.f / sum;
        uint32_t *dst =
            reinterpret_cast<uint32_t *>((T *)p.out + to * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2)
          dst[e / 2] = sum == 0.f ? 0 : pack2<T>(out[e] * inv,
                                                 out[e + 1] * inv);
        if (p.lse && lane == 0)
          p.lse[to] = sum == 0.f ? -kInf : (top - kBias + log2f(sum)) * kLn2;
      } else {
        const long long part =
            ((long long)blockIdx.x * 2 + (u.j0 == 0 ? 1 : 0)) * ROWS + r;
        if (lane == 0) p.part_ml[part] = make_float2(top - kBias, sum);
#pragma unroll
        for (int e = 0; e < E; ++e)
          p.part_o[part * D + lane * E + e] = out[e];
      }
    }
    __syncthreads();
    if (tid == 0) s.bad = 0;
  }

  if (s.plan.any_unusable) {
    // NaN for the sequences that cannot be read
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      const Chunk c = attn_chunk(p, b);
      if (c.usable || c.n == 0) continue;
      if (tid == 0) status_or(p.dev_status, SD_DEV_BAD_LENGTH);
      const long long lo = (long long)c.start * p.Hq,
                      n = (long long)c.n * p.Hq;
      for (long long i = tid; i < n * D; i += WARPS * 32)
        ((T *)p.out)[lo * D + i] = narrow<T>(__int_as_float(0x7fc00000));
      if (p.lse)
        for (long long i = tid; i < n; i += WARPS * 32)
          p.lse[lo + i] = __int_as_float(0x7fc00000);
    }
  }
}

// ------------------------------------------------------------------- host
constexpr int kMaxGrid4 = 320;  // CTAs the workspace is laid out for

int rows_tile(int max_q, int G) {
  return (long long)max_q * G <= 8 ? 1 : 2;
}

template <class T, int D, int NT>
sd_status launch_rows(Attn4Params &p, int sms, void *ws, cudaStream_t s) {
  constexpr int WARPS = 8;
  constexpr size_t smem = sizeof(Shared4<8 * NT, D, WARPS>);
  set_workspace(p, ws_layout(kMaxGrid4, 8 * NT, D), ws);
  const void *kernel = (const void *)kv4_rows_kernel<T, D, NT, WARPS>;
  int dev = 0;
  SDV_CUDA(cudaGetDevice(&dev));
  static std::atomic<unsigned long long> ready{0};
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    SDV_CUDA(cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  const int want = NT == 1 ? 2 * sms : sms;
  const unsigned grid = want < kMaxGrid4 ? want : kMaxGrid4;
  void *args[] = {&p};
  const sd_status st = launch_pdl(kernel, grid, WARPS * 32, smem, s, args);
  return st != SD_OK ? st : launch_join<T, D, 8 * NT>(p, grid, s);
}

template <class T>
sd_status dispatch4(Attn4Params &p, int D, int nt, int sms, void *ws,
                    cudaStream_t s) {
  if (D == 64)
    return nt == 1 ? launch_rows<T, 64, 1>(p, sms, ws, s)
                   : launch_rows<T, 64, 2>(p, sms, ws, s);
  return nt == 1 ? launch_rows<T, 128, 1>(p, sms, ws, s)
                 : launch_rows<T, 128, 2>(p, sms, ws, s);
}

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_kv4_attention_workspace(int q_heads, int heads,
                                             int head_dim, int max_q) {
  if (heads < 1 || q_heads < heads || (head_dim != 64 && head_dim != 128))
    return 256;
  return ws_layout(kMaxGrid4, 8 * rows_tile(max_q, q_heads / heads), head_dim)
      .bytes;
}

extern "C" sd_status sd_kv4_attention(
    const void *q, long long q_stride, int q_heads, const sd_paged_kv4 *cache,
    const int32_t *q_start, const int32_t *kv_len, const int32_t *tree_mask,
    int mask_words, int B, int total, int max_q, float scale, void *out,
    float *lse, int32_t *dev_status, void *workspace, size_t ws_bytes,
    void *stream) {
  sd_status st = check_kv4(cache);
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
  if (B == 0 || total == 0) return SD_OK;
  SDV_REQUIRE(q && cache->k && cache->v && cache->k_scale &&
                  cache->v_scale && q_start && kv_len && out,
              "null pointer");
  SDV_REQUIRE(cache->max_pages == 0 || cache->block_table,
              "block_table is null");
  SDV_REQUIRE(q_stride >= (long long)q_heads * D,
              "tokens overlap: q_stride is below q_heads x head_dim");
  SDV_REQUIRE(aligned16(q) && q_stride % 8 == 0,
              "q must be 16-byte aligned, q_stride a multiple of 8");
  SDV_REQUIRE((reinterpret_cast<uintptr_t>(out) & 31) == 0,
              "out must be 32-byte aligned");
  SDV_REQUIRE((long long)total * q_heads < (1LL << 31) - 256,
              "total x q_heads does not fit 31 bits");
  const size_t need =
      sd_kv4_attention_workspace(q_heads, cache->heads, D, max_q);
  SDV_REQUIRE(workspace && ws_bytes >= need &&
                  (reinterpret_cast<uintptr_t>(workspace) & 31) == 0,
              "a 32-byte aligned workspace of >= %zu bytes required", need);
  int sms = 0;
  st = check_device(&sms);
  if (st != SD_OK) return st;
  Attn4Params p;
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
  p.G = q_heads / cache->heads;
  p.Hkv = cache->heads;
  p.by_G = fast_div(p.G);
  p.by_page = fast_div(cache->page_size);
  p.page_size = cache->page_size;
  p.max_pages = cache->max_pages;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.out = out;
  p.lse = lse;
  p.dev_status = dev_status;
  p.c = kv4_cache(cache);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int nt = rows_tile(max_q, p.G);
  return cache->dt == SD_BF16
             ? dispatch4<__nv_bfloat16>(p, D, nt, sms, workspace, s)
             : dispatch4<__half>(p, D, nt, sms, workspace, s);
}
