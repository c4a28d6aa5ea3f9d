// sdv_kv4_attention.cu -- sd_kv4_attention: a chunk of new tokens attends
// over the 4-bit paged cache.
//
// With more than 16 rows a head, the kernel of sdv_attention.cuh; with up to 8
// or 16, the one below, whose products are small ones of a warp's own: tiles
// of 128 rows there would be written to and read from shared memory as 16-bit
// numbers, four times the cache's bytes, and take 2.2 times as long for 8 rows
// (64 sequences of up to 8192 keys: 88 us here; 16 rows 136, and 195 there).
#include "sdv_attention.cuh"

namespace sdv {
namespace {

// ------------------------------------------------------- few rows a head
//
// Where a cache head has few rows (one token of a group of query heads), a
// warp takes 32 keys at a time, makes their codes operands in registers, and
// has the keys as the rows of its products:
//   S^T [16 keys x 8 rows] = K [16 x D] Q^T,   O^T [D x 8] += V^T [D x 16] W
// so that 8 rows are not padded to more.  Four neighbouring threads hold a
// key's row: which of its elements a step of a product takes is free as long
// as the queries' operand takes the same.  Each warp has a ring of such blocks
// in shared memory, which it fills itself with asynchronous copies, codes and
// pairs as they lie: no other warp is waited for until a unit ends.  (A warp
// that brought tiles of 128 keys by bulk copies, four a page, was held up by
// their number: 56 cycles a copy, 154 us on 64 sequences of pages of 16.)
//
// What it spends its time on: making numbers of codes.  A word, eight values,
// is 4 masks, a shift, 2 subtractions and 4 fmas; 16 keys of 128 are 16 words a
// lane and 340 instructions in all, 41 ns of an SM's issue slots (2.07 GHz),
// where their bytes take 52 at the measured copy rate.  No pipe is full: four
// warps a scheduler issue in 0.6 of the slots, and of 6.1 warps at an issue 1.3
// wait for the result before, 1.0 for a pipe and 0.7 to be dispatched, 0.3 for
// memory.  88 us on 64 sequences (0.40 GB, 4.5 TB/s, 0.67 of the copy rate), 67
// us and a join of 8 on one token behind 262144 keys.
//
// The units' shares are per warp, in places of 32 keys; what the warps of a CTA
// have of one unit they join in shared memory at the end, what CTAs have of one
// the join kernel.  (With a share a CTA, whose warps joined at every unit's
// end, 200 sequences of up to 300 keys took 49 us; this takes 30.)
//
// A row's weights are fp16, 2^kBias at its reference m, which moves up only
// when a score is 2^kSlack above it: at most 2^15, and a weight 2^-24 of the
// reference's still has all its bits.  Beside rows in fp16 a weight is the sum
// of two such numbers and O takes a product of each (REST), so that the result
// is off by little more than its own rounding; one would be as coarse as that
// (0.00029 off where the rounding is 0.00021).  Beside bf16 rows one number's
// rounding is an eighth of the result's: two are 0.00165 off and one 0.00166,
// and 64 sequences take 98 us with two and 88 with one, one token behind
// 262144 keys 82 and 75.
constexpr float kBias = 10.f, kSlack = 5.f;
constexpr float kNone = 3e38f;  // in place of kBias - m: no reference yet
constexpr int kBlock = 32;  // keys of a warp's step, two products' rows

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0,
                                         uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
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

// A part of a unit that a warp leaves to be joined with others: (m, l) and O
// of its rows.
template <int ROWS, int D> struct Part {
  float2 ml[ROWS];
  alignas(16) float o[ROWS][D];
};
struct PartInfo {
  int there;          // there is one
  int begun, ended;   // it has the unit's first, its last key
  int rows, start, head, first, ahead;  // ahead: places to the unit's end
};

template <int ROWS, int D, int WARPS> struct Shared4 {
  Plan plan;
  PartInfo info[WARPS][2];
  Part<ROWS, D> part[WARPS];  // of the warp's first unit
};

// A thread's part of a query row, D / 4 elements, as fp16 pairs, and the
// factor of its scores (see fit_query).
template <int N>
__device__ __forceinline__ float load_query(const void *src, bool valid,
                                            bool bf16, float scale,
                                            uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (valid) x = __ldg(reinterpret_cast<const uint4 *>(src) + i / 4);
    w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
  }
  return fit_query<4>(w, bf16, scale);
}

constexpr int kKeys = kBlock;  // keys of a place in the shares

// SB: bytes of a key's pairs.  REST: weights are two numbers each.
template <int D, int SB, int NT, int WARPS, bool REST>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 2 : 1)
kv4_rows_kernel(const __grid_constant__ AttnParams p) {
  constexpr int ROWS = 8 * NT, W = D / 32;  // W: words of a key a thread
  constexpr int CODES = kBlock * D / 2;     // bytes of a block's key codes
  static_assert(sizeof(Part<ROWS, D>) <= 2 * (2 * CODES + 8 * kBlock),
                "a part does not fit the smallest ring");
  using S = Shared4<ROWS, D, WARPS>;
  using U = Units<ROWS, kKeys>;
  extern __shared__ __align__(1024) char dyn[];
  S &s = *reinterpret_cast<S *>(dyn);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  constexpr int sb = SB, slot_bytes = 2 * CODES + 2 * kBlock * SB;
  constexpr int GROUP = 4 * D / SB;
  auto ring_of = [&](int w) {
    return dyn + (sizeof(S) + 127) / 128 * 128 + w * 2 * slot_bytes;
  };
  char *ring = ring_of(warp);
  griddep_wait();
  make_plan<ROWS, kKeys>(p, s.plan);
  if (tid == 0) p.cut[blockIdx.x].parts = 0;
  if (lane < 2) s.info[warp][lane].there = 0;
  __syncthreads();

  // ---- the warp's blocks of a unit: where the next ones lie.  Lane 4 i + o
  // holds the places in bytes of the codes and pairs of keys 8 o to 8 o + 7 of
  // the i-th block of a batch of eight; negative: nothing to be had.
  struct Places {
    long long code, pair;
  };
  bool bad = false;
  auto look_up = [&](const U &v, int first) {  // the batch's first block
    const int key = v.j0 * kKeys + first * kBlock + 8 * lane;
    Places x{-1, -1};
    if (key < min(v.j1 * kKeys, v.c.kv)) {
      const int n = div_by(key, p.by_page);
      const int page =
          __ldg(p.block_table + (long long)v.b * p.max_pages + n);
      if (page >= 0 && page < p.c.num_pages) {
        const int row = (v.h - n) * p.page_size + key;
        x.code = page * p.c.page_stride + (long long)row * (D / 2);
        x.pair = page * p.c.scale_stride + (long long)row * sb;
      } else {
        bad = true;
      }
    }
    return x;
  };
  // A lane's part of the copies of a block: 16 bytes of the codes of each
  // eight keys (D = 64: of every other eight), and of pairs.
  const uint32_t to = smem_addr(ring) + 16 * lane;
  constexpr int CHUNKS = 4 * SB;  // of 16 bytes of pairs, keys' first
  const int which = lane / (2 * SB), pair_8 = lane / (SB / 2) & 3;
  const char *pairs = (which ? p.c.v_scale : p.c.k_scale) +
                      16 * (lane & (SB / 2 - 1));
  const char *k_codes = p.c.k + 16 * (lane & (D / 4 - 1));
  const char *v_codes = p.c.v + 16 * (lane & (D / 4 - 1));
  int fill = 0;  // where to fill next
  auto fetch = [&](const Places &x, int i) {
    const uint32_t at = to + fill;
#pragma unroll
    for (int o = 0; o < D / 32; ++o) {
      const long long c = __shfl_sync(
          ~0u, x.code, 4 * i + (D == 128 ? o : 2 * o + (lane >> 4)));
      cp16(at + 512 * o, k_codes + c, c >= 0);
      cp16(at + CODES + 512 * o, v_codes + c, c >= 0);
    }
    const long long c = __shfl_sync(~0u, x.pair, 4 * i + pair_8);
    cp16(at + 2 * CODES, pairs + c, lane < CHUNKS && c >= 0);
    if (CHUNKS > 32)  // the values' pairs: the same places
      cp16(at + 2 * CODES + 512, p.c.v_scale + 16 * (lane & (SB / 2 - 1)) + c,
           c >= 0);
    cp_commit();
    fill ^= slot_bytes;
  };
  // Row g of a product's keys is key (g >> 1) + 4 (g & 1) of eight, so that
  // the two whose values a thread pairs are t and t + 4: four rows of 64
  // bytes in a row, which share banks two by two instead of all four.
  const int kg = (g >> 1) + 4 * (g & 1);
  const int k_at = kg * (D / 2) + t * (D / 8);
  const int ks_at = kg * sb + 4 * (t * (D / 4) / GROUP);
  const int v_at = t * (D / 2) + g * (D / 16);
  const int vs_at = t * sb + 4 * (g * (D / 8) / GROUP);

  auto pack = [&](float a, float b) {
    return p.bf16 ? pack2<__nv_bfloat16>(a, b) : pack2<__half>(a, b);
  };

  // the warp's share of the CTA's
  const unsigned long long all = s.plan.x1 - s.plan.x0;
  const unsigned long long from = all * warp / WARPS;
  U u(p, s.plan, from, all * (warp + 1) / WARPS - from);
  Places now{-1, -1};
  int slot = 0;  // where to use next
  if (u.left) {
    now = look_up(u, 0);
    fetch(now, 0);
  }
  while (u.left) {
    // the queries' operand: the thread's quarter of rows g (and g + 8)
    uint32_t qf[NT][4 * W];
    float rs[NT][2], off[NT][2], l[NT][2];
    const int ctx = u.c.kv - u.c.n;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = u.t * ROWS + 8 * n + g, tok = div_by(r, p.by_G);
      const float f = load_query<4 * W>(
          (const uint16_t *)p.q + (u.c.start + tok) * p.q_stride +
              (long long)(u.h * p.G + r - tok * p.G) * D + t * (D / 4),
          8 * n + g < u.rows, p.bf16, p.scale_log2, qf[n]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        rs[n][e] = __shfl_sync(~0u, f, 4 * (2 * t + e));  // of row 2 t + e
        off[n][e] = kNone;
        l[n][e] = 0.f;
      }
    }
    float o[NT][2 * W][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2 * W; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    // keys that every row of the unit sees
    const int open = p.mask ? ctx : ctx + div_by(u.t * ROWS, p.by_G) + 1;

    const char *k_from = ring + k_at, *ks_from = ring + 2 * CODES + ks_at;
    const char *v_from = ring + CODES + v_at;
    const char *vs_from = ring + 2 * CODES + kBlock * SB + vs_at;
    // NB times 16 keys, from the b0-th of the block on.  With 16 rows there
    // are no registers for both at once (188 us where 147 were taken so).
    constexpr int NB = NT == 1 ? 2 : 1;
    auto use = [&](auto hides, int key, int b0) {
      constexpr bool HIDE = decltype(hides)::value;
      // scores: [16 keys][rows]
      float sc[NB][NT][4];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[b][n][e] = 0.f;
        uint32_t k[2][W], a[2], c[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          lds_words(k_from + slot + 8 * (D / 2) * (2 * (b0 + b) + hf), k[hf]);
          uint32_t x = *reinterpret_cast<const uint32_t *>(
              ks_from + slot + 8 * SB * (2 * (b0 + b) + hf));
          // what lies past the sequence's keys counts as zeros
          if (HIDE && key + 16 * (b0 + b) + 8 * hf + kg >= u.c.kv) x = 0;
          a[hf] = both_lo(x);
          c[hf] = both_hi(x);
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const uint32_t f0 = kv4_fma(kv4_codes(k[0][i], j), a[0], c[0]);
            const uint32_t f1 = kv4_fma(kv4_codes(k[1][i], j), a[1], c[1]);
            const uint32_t f2 =
                kv4_fma(kv4_codes(k[0][i], j + 1), a[0], c[0]);
            const uint32_t f3 =
                kv4_fma(kv4_codes(k[1][i], j + 1), a[1], c[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(sc[b][n], f0, f1, f2, f3, qf[n][4 * i + j],
                       qf[n][4 * i + j + 1]);
          }
      }
      // exponents of the weights; of keys a row does not see -inf
      float y[NB][NT][4];
      float most = -kInf;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[b][n][e] = fmaf(sc[b][n][e], rs[n][e & 1], off[n][e & 1]);
            if (HIDE) {
              const int r = min(8 * n + 2 * t + (e & 1), u.rows - 1);
              const int token = div_by(u.t * ROWS + r, p.by_G);
              const int i = key + 16 * (b0 + b) + kg + (e >> 1) * 8 - ctx;
              bool see = i <= token;
              if (p.mask) {
                see = i < u.c.n;
                if (see && i >= 0)
                  see = __ldg(p.mask +
                              (long long)(u.c.start + token) * p.mask_words +
                              (i >> 5)) >>
                            (i & 31) &
                        1;
              }
              if (!see) y[b][n][e] = -kInf;
            }
          }
          most = max3f(most, y[b][n][0], y[b][n][1]);
          most = max3f(most, y[b][n][2], y[b][n][3]);
        }
      if (__any_sync(~0u, most > kBias + kSlack)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // (from kNone the exponents say nothing but which keys count)
            float x[2 * NB], top = -kInf;
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
              x[i] = y[i >> 1][n][e + 2 * (i & 1)];
              if (x[i] != -kInf)
                x[i] = sc[i >> 1][n][e + 2 * (i & 1)] * rs[n][e];
              top = fmaxf(top, x[i]);
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
              top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            if (top + off[n][e] > kBias + kSlack) {
              const float up = kBias - top, f = ex2(up - off[n][e]);
              off[n][e] = up;
#pragma unroll
              for (int i = 0; i < 2 * NB; ++i)
                y[i >> 1][n][e + 2 * (i & 1)] = x[i] + up;
              l[n][e] *= f;
#pragma unroll
              for (int i = 0; i < 2 * W; ++i) {
                o[n][i][e] *= f;
                o[n][i][e + 2] *= f;
              }
            }
          }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        // values of two keys at a time: their codes are brought together
        uint32_t v[4][W / 2], va[2], vc[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const char *from = v_from + slot + 8 * (D / 2) * (2 * (b0 + b) + hf);
          lds_words(from, v[2 * hf]);
          lds_words(from + 4 * (D / 2), v[2 * hf + 1]);
          from = vs_from + slot + 8 * SB * (2 * (b0 + b) + hf);
          uint32_t x = *reinterpret_cast<const uint32_t *>(from);
          uint32_t z = *reinterpret_cast<const uint32_t *>(from + 4 * SB);
          if (HIDE && key + 16 * (b0 + b) + 8 * hf + t >= u.c.kv) x = 0;
          if (HIDE && key + 16 * (b0 + b) + 8 * hf + t + 4 >= u.c.kv) z = 0;
          va[hf] = __byte_perm(x, z, 0x5410);
          vc[hf] = __byte_perm(x, z, 0x7632);
        }
        uint32_t w[NT][2], rest[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float2 z = make_float2(ex2(y[b][n][2 * hf]),
                                         ex2(y[b][n][2 * hf + 1]));
            l[n][0] += z.x;
            l[n][1] += z.y;
            if (REST) {
              split2<__half>(z, w[n][hf], rest[n][hf]);
              rest[n][hf] = transpose8(rest[n][hf]);
            } else {
              w[n][hf] = pack2<__half>(z.x, z.y);
            }
            w[n][hf] = transpose8(w[n][hf]);
          }
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
          uint32_t lo[2], hi[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            lo[hf] = __byte_perm(v[2 * hf][i], v[2 * hf + 1][i], 0x5410);
            hi[hf] = __byte_perm(v[2 * hf][i], v[2 * hf + 1][i], 0x7632);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // elements 8 i + 2 j (rows g) and 8 i + 2 j + 1 (rows g + 8)
            const uint32_t f0 = kv4_fma(kv4_codes(lo[0], j), va[0], vc[0]);
            const uint32_t f1 = kv4_fma(kv4_codes(hi[0], j), va[0], vc[0]);
            const uint32_t f2 = kv4_fma(kv4_codes(lo[1], j), va[1], vc[1]);
            const uint32_t f3 = kv4_fma(kv4_codes(hi[1], j), va[1], vc[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(o[n][4 * i + j], f0, f1, f2, f3, w[n][0], w[n][1]);
              if (REST)
                mma16816(o[n][4 * i + j], f0, f1, f2, f3, rest[n][0],
                         rest[n][1]);
            }
          }
        }
      }
    };
    const int key0 = u.j0 * kKeys;
    const int blocks = (min(u.j1 * kKeys, u.c.kv) - key0 + kBlock - 1) /
                       kBlock;
    for (int i = 0; i < blocks; ++i) {
      cp_wait<0>();
      __syncwarp();
      // the next block goes where the one before this was
      if (((i + 1) & 7) == 0) now = look_up(u, i + 1);
      fetch(now, (i + 1) & 7);
      const int key = key0 + i * kBlock;
#pragma unroll 1
      for (int b0 = 0; b0 < 2; b0 += NB)
        if (key + kBlock > open) use(std::true_type{}, key, b0);
        else use(std::false_type{}, key, b0);
      slot ^= slot_bytes;
    }

    // ---- the end of the part.  The block past it was fetched as an empty
    // one: the next unit's first takes its place
    cp_wait<0>();
    fill = slot;
    const bool was_bad = __any_sync(~0u, bad);
    bad = false;
    const bool begun = u.j0 == 0, ended = u.j1 == u.nk;
    const int start = u.c.start, first = u.t * ROWS, head = u.h;
    const int rows = u.rows, ahead = u.nk - u.j1;
    u.next();
    if (u.left) {
      now = look_up(u, 0);
      fetch(now, 0);
    }
    if (was_bad && lane == 0) status_or(p.dev_status, SD_DEV_BAD_PAGE);
    // The last part may go where the ring was: nothing is on its way there.
    Part<ROWS, D> &part =
        begun ? *reinterpret_cast<Part<ROWS, D> *>(ring) : s.part[warp];
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
          sum += __shfl_xor_sync(~0u, sum, d);
        if (was_bad) sum = __int_as_float(0x7fc00000);
        // element 2 i of the thread's eighth is in o[i][e], 2 i + 1 in
        // o[i][e + 2]
        const int r = 8 * n + 2 * t + e;
        if (!begun || !ended) {
          if (g == 0)
            part.ml[r] = make_float2(
                off[n][e] == kNone ? -kInf : -off[n][e], sum);
#pragma unroll
          for (int i = 0; i < 2 * W; i += 2)
            *reinterpret_cast<float4 *>(&part.o[r][g * (D / 8) + 2 * i]) =
                make_float4(o[n][i][e], o[n][i][e + 2], o[n][i + 1][e],
                            o[n][i + 1][e + 2]);
        } else if (r < rows) {
          const int tok = div_by(first + r, p.by_G);
          const long long row = (long long)(start + tok) * p.Hq +
                                head * p.G + first + r - tok * p.G;
          // no key seen: 0, whatever O has of another row's infinity
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          uint32_t w[2 * W];
#pragma unroll
          for (int i = 0; i < 2 * W; ++i)
            w[i] = sum == 0.f ? 0
                              : pack(o[n][i][e] * inv, o[n][i][e + 2] * inv);
          uint16_t *dst = (uint16_t *)p.out + row * D + g * (D / 8);
          if constexpr (D == 128) {
            st_v8(dst, w);
          } else {
            *reinterpret_cast<uint4 *>(dst) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (p.lse && g == 0)
            p.lse[row] =
                sum == 0.f ? -kInf : (log2f(sum) - off[n][e]) * kLn2;
        }
      }
    if (lane == 0 && (!begun || !ended))
      s.info[warp][begun] = PartInfo{1,     begun, ended, rows,
                                     start, head,  first, ahead};
  }
  __syncthreads();

  // ---- parts of one unit lie in warps one after the other; what they make
  // together is the unit, or the CTA's part of it.  A warp per row.
  for (int w0 = 0; w0 < WARPS; ++w0)
    for (int second = 0; second < 2; ++second) {
      // where a chain of parts starts
      const PartInfo &f = s.info[w0][second];
      if (!f.there || (!second && all * w0 / WARPS > 0)) continue;
      int w1 = w0;  // its last warp (some may have no share at all)
      bool ended = f.ended;
      for (int w = w0 + 1; w < WARPS && !ended; ++w)
        if (s.info[w][0].there) {
          w1 = w;
          ended = s.info[w][0].ended;
        }
      const int ahead = s.info[w1][w1 == w0 ? second : 0].ahead;
      if (tid == 0 && f.begun && !ended) {
        // the unit goes on in the CTAs up to the one whose share holds its
        // last key
        const unsigned long long end = s.plan.x1 + (unsigned)ahead;
        CutUnit cut;
        cut.parts = (int)((end * s.plan.n - 1) / s.plan.total) -
                    (int)blockIdx.x + 1;
        cut.rows = f.rows;
        cut.start = f.start;
        cut.head = f.head;
        cut.first = f.first;
        p.cut[blockIdx.x] = cut;
      }
      constexpr int E = D / 32;
      for (int r = warp; r < f.rows; r += WARPS) {
        float top = -kInf, sum = 0.f, out[E] = {};
        auto part_of = [&](int w) -> const Part<ROWS, D> & {
          return w == w0 && second
                     ? *reinterpret_cast<const Part<ROWS, D> *>(ring_of(w))
                     : s.part[w];
        };
        for (int w = w0; w <= w1; ++w)
          if (w == w0 || s.info[w][0].there)
            top = fmaxf(top, part_of(w).ml[r].x);
        for (int w = w0; w <= w1; ++w) {
          if (w > w0 && !s.info[w][0].there) continue;
          const Part<ROWS, D> &x = part_of(w);
          const float2 a = x.ml[r];
          const float k = part_weight(a, top);
          sum += a.y * k;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float y = x.o[r][lane * E + e];
            if (k != 0.f) out[e] = fmaf(y, k, out[e]);
          }
        }
        if (f.begun && ended) {
          const int tok = div_by(f.first + r, p.by_G);
          const long long row = (long long)(f.start + tok) * p.Hq +
                                f.head * p.G + f.first + r - tok * p.G;
          const float inv = 1.f / sum;
          uint32_t *dst =
              reinterpret_cast<uint32_t *>((uint16_t *)p.out + row * D +
                                           lane * E);
#pragma unroll
          for (int e = 0; e < E; e += 2)
            dst[e / 2] =
                sum == 0.f ? 0 : pack(out[e] * inv, out[e + 1] * inv);
          if (p.lse && lane == 0)
            p.lse[row] = sum == 0.f ? -kInf : (top + log2f(sum)) * kLn2;
        } else {
          const long long at =
              ((long long)blockIdx.x * 2 + (f.begun ? 1 : 0)) * ROWS + r;
          if (lane == 0) p.part_ml[at] = make_float2(top, sum);
#pragma unroll
          for (int e = 0; e < E; ++e)
            p.part_o[at * D + lane * E + e] = out[e];
        }
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
      for (long long i = tid; i < n * D; i += WARPS * 32)
        ((uint16_t *)p.out)[lo * D + i] = 0x7fff;  // NaN of either type
      if (p.lse)
        for (long long i = tid; i < n; i += WARPS * 32)
          p.lse[lo + i] = __int_as_float(0x7fc00000);
    }
  }
}

// ------------------------------------------------------------------- host
constexpr int kMaxGrid4 = 320;  // CTAs the workspace is laid out for

// The kernel of a call, by the rows a head has: 8 or 16 at a time in warps of
// their own, 128 or 256 in tiles.  Measured on 64 sequences of up to 8192 keys:
// 16 rows 136 us in warps and 195 in tiles, 32 rows 260 and 195.
int rows_of(int max_q, int G) {
  const long long n = (long long)max_q * G;
  return n <= 8 ? 8 : n <= 16 ? 16 : n <= 128 ? 128 : 256;
}
size_t workspace_of(int rows, int D) {
  return ws_layout(rows <= 16 ? kMaxGrid4 : kMaxGrid, rows, D).bytes;
}

template <int D, int SB, int NT, bool REST>
sd_status launch_rows(AttnParams &p, int sms, void *ws, cudaStream_t s) {
  // Two CTAs of eight warps an SM where their shared memory lets them (200
  // sequences of 300 keys take 29 us so, and 35 with one of sixteen); with
  // pairs of 32 elements at D = 128 it does not, and one of sixteen takes 92 us
  // on 64 sequences, one of eight 110.  16 rows a head hold twice as much a
  // warp: one CTA of twelve, as many as shared memory holds at D = 128: 137
  // us on 64 sequences (its spills of 200 bytes included; eight warps, which
  // spill nothing, take 132, ten 153), at D = 64 81 (eight 88, sixteen 81).
  constexpr int WARPS = NT == 2 ? 12 : D == 128 && SB == 16 ? 16 : 8;
  constexpr size_t smem =
      (sizeof(Shared4<8 * NT, D, WARPS>) + 127) / 128 * 128 +
      WARPS * 2 * kBlock * (D + 2 * SB);
  set_workspace(p, ws_layout(kMaxGrid4, 8 * NT, D), ws);
  const void *kernel = (const void *)kv4_rows_kernel<D, SB, NT, WARPS, REST>;
  int dev = 0;
  SDV_CUDA(cudaGetDevice(&dev));
  static std::atomic<unsigned long long> ready{0};
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    SDV_CUDA(cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  const int want = WARPS == 8 ? 2 * sms : sms;
  const unsigned grid = want < kMaxGrid4 ? want : kMaxGrid4;
  void *args[] = {&p};
  const sd_status st = launch_pdl(kernel, grid, WARPS * 32, smem, s, args);
  if (st != SD_OK) return st;
  return p.bf16 ? launch_join<__nv_bfloat16, D, 8 * NT, kKeys>(p, grid, s)
                : launch_join<__half, D, 8 * NT, kKeys>(p, grid, s);
}

template <int NT, bool REST>
sd_status dispatch_rows(AttnParams &p, int D, int sms, void *ws,
                        cudaStream_t s) {
  const int sb = p.c.scale_bytes;
  if (D == 64)
    return sb == 4 ? launch_rows<64, 4, NT, REST>(p, sms, ws, s)
                   : launch_rows<64, 8, NT, REST>(p, sms, ws, s);
  return sb == 4   ? launch_rows<128, 4, NT, REST>(p, sms, ws, s)
         : sb == 8 ? launch_rows<128, 8, NT, REST>(p, sms, ws, s)
                   : launch_rows<128, 16, NT, REST>(p, sms, ws, s);
}

template <bool PAIR, bool REST>
sd_status dispatch_tiles(AttnParams &p, int D, int sms, void *ws,
                         cudaStream_t s) {
  const CUtensorMap none = {};  // tiles are not loaded but made
  char *at = static_cast<char *>(ws);
  return D == 64 ? launch<__half, 64, PAIR, true, REST>(p, none, none, sms, at,
                                                        s)
                 : launch<__half, 128, PAIR, true, REST>(p, none, none, sms,
                                                         at, s);
}

template <bool REST>
sd_status dispatch_up_to_128(AttnParams &p, int rows, int D, int sms, void *ws,
                        cudaStream_t s) {
  return rows == 8    ? dispatch_rows<1, REST>(p, D, sms, ws, s)
         : rows == 16 ? dispatch_rows<2, REST>(p, D, sms, ws, s)
                      : dispatch_tiles<false, REST>(p, D, sms, ws, s);
}

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" size_t sd_kv4_attention_workspace(int q_heads, int heads,
                                             int head_dim, int max_q) {
  if (heads < 1 || q_heads < heads || (head_dim != 64 && head_dim != 128))
    return 256;
  return workspace_of(rows_of(max_q, q_heads / heads), head_dim);
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
  p.num_pages = cache->num_pages;
  p.c = kv4_cache(cache);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.bf16 = cache->dt == SD_BF16;
  const int rows = rows_of(max_q, p.G);
  if (rows == 256) return dispatch_tiles<true, false>(p, D, sms, workspace, s);
  return p.bf16 ? dispatch_up_to_128<false>(p, rows, D, sms, workspace, s)
                : dispatch_up_to_128<true>(p, rows, D, sms, workspace, s);
}
