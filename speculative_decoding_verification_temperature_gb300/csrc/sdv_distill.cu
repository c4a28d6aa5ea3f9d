// sdv_distill.cu -- sd_distill_topk and its gradient: distillation of a
// drafter from the target's top logits.
//
// With p the teacher's probabilities of its K entries, P their sum and q =
// softmax(z / T) of the student's row,
//   loss = sum_k p_k (log p_k - log q_k)
//   d loss / d z_j = (P q_j - sum_{k: id_k = j} p_k) / T.
//
// All three calls stream vocabulary rows: the forward call reads a row once,
// the backward call reads and writes it once, and so does the step, which
// keeps a row in the shared memory of a cluster between the pass that finds
// log sum exp and the pass that writes the gradient.
//
// A row is cut into 16-byte slots by address, whatever its own alignment:
// only its first and last slot can be partial, and those alone are read and
// written by the element.
#include <atomic>

#include "sdv_device.cuh"
#include "sdv_host.cuh"
#include "sdv_tma.cuh"

namespace sdv {
namespace {

constexpr float kLn2 = 0.693147180559945f;
constexpr int kBatch = 8;         // slots a thread has in flight

struct DistillParams {
  const void *student;
  long long row_stride;
  const float *logit, *teacher_lse, *grad_loss;
  const int32_t *id;
  int N, V, K, CL;
  float k2;     // log2(e) / T
  float inv_T;
  float *loss, *lse;
  const float *lse_in;
  void *grad;
  long long grad_stride;
  int32_t *dev_status;
};

// A row as 16-byte slots from the aligned address at or before its start:
// column j is element head + j; slots [f0, f1) are whole.
template <int DT> struct SlotRow {
  static constexpr int VW = vec_width<DT>();
  const char *base;
  int head, V, slots, f0, f1;
  __device__ SlotRow(const void *rows, long long stride, int row, int V_)
      : V(V_) {
    const char *start =
        (const char *)rows + (long long)row * stride * elt_bytes<DT>();
    head = (int)(reinterpret_cast<uintptr_t>(start) & 15) / elt_bytes<DT>();
    base = start - head * elt_bytes<DT>();
    slots = (head + V + VW - 1) / VW;
    f0 = head > 0;
    f1 = max((head + V) / VW, f0);
  }
  __device__ bool full(int s) const {
    return (unsigned)(s - f0) < (unsigned)(f1 - f0);
  }
  __device__ int first_col(int s) const { return s * VW - head; }
};

__device__ __forceinline__ uint4 ld_v4(const void *p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// A partial slot by the element; columns outside the row are -inf.
template <int DT>
__device__ __noinline__ Raw<DT, vec_width<DT>()> load_partial(
    const SlotRow<DT> &r, int s) {
  uint32_t w[4] = {};
  const int c0 = r.first_col(s);
  for (int e = 0; e < r.VW; ++e) {
    const bool in = c0 + e >= 0 && c0 + e < r.V;
    const char *at = r.base + (s * r.VW + e) * (long long)elt_bytes<DT>();
    if (DT == 0) {
      w[e] = in ? *reinterpret_cast<const uint32_t *>(at) : 0xff800000u;
    } else {
      const uint32_t h =
          in ? *reinterpret_cast<const unsigned short *>(at) : 0xff80u;
      w[e >> 1] |= h << (16 * (e & 1));
    }
  }
  Raw<DT, vec_width<DT>()> x;
  x.w = make_uint4(w[0], w[1], w[2], w[3]);
  return x;
}

template <int DT>
__device__ __forceinline__ Raw<DT, vec_width<DT>()> load_slot(
    const SlotRow<DT> &r, int s) {
  if (r.full(s)) {
    Raw<DT, vec_width<DT>()> x;
    x.w = ld_v4(r.base + (long long)s * 16);
    return x;
  }
  return load_partial(r, s);
}

// One logit (a plain load: the row may be written in this kernel, later).
template <int DT>
__device__ __forceinline__ float load_col(const SlotRow<DT> &r, int j) {
  const char *at = r.base + (long long)(r.head + j) * elt_bytes<DT>();
  if constexpr (DT == 0) return *reinterpret_cast<const float *>(at);
  const uint32_t h = *reinterpret_cast<const unsigned short *>(at);
  return __uint_as_float(h << 16);
}

template <int DT>
__device__ __forceinline__ void store_elt(void *row, int j, float x) {
  if constexpr (DT == 0) {
    ((float *)row)[j] = x;
  } else {
    uint32_t u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(u) : "f"(x));
    ((unsigned short *)row)[j] = (unsigned short)u;
  }
}

// c 2^(z k2 + nl2) of a slot's columns, as the row's type.
template <int DT>
__device__ __forceinline__ uint4 slot_grad(
    const Raw<DT, vec_width<DT>()> &x, float c, float k2, float nl2) {
  constexpr int VW = vec_width<DT>();
  const uint32_t in[4] = {x.w.x, x.w.y, x.w.z, x.w.w};
  uint32_t out[4];
  const float2 kk = make_float2(k2, k2), nn = make_float2(nl2, nl2),
               cc = make_float2(c, c);
#pragma unroll
  for (int e = 0; e < VW; e += 2) {
    float2 z = DT == 0 ? make_float2(__uint_as_float(in[e % 4]),
                                     __uint_as_float(in[(e + 1) % 4]))
                       : make_float2(__uint_as_float(in[e / 2] << 16),
                                     __uint_as_float(in[e / 2] & 0xffff0000u));
    z = fma2(z, kk, nn);
    z.x = ex2(z.x);
    z.y = ex2(z.y);
    z = mul2(z, cc);
    if constexpr (DT == 0) {
      out[e % 4] = __float_as_uint(z.x);
      out[(e + 1) % 4] = __float_as_uint(z.y);
    } else {
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
          : "=r"(out[e / 2])
          : "f"(z.y), "f"(z.x));
    }
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The columns of slot s that lie in the row, by the element.
template <int DT>
__device__ __noinline__ void store_partial(const SlotRow<DT> &r, char *grad,
                                           int s, uint4 g) {
  const uint32_t w[4] = {g.x, g.y, g.z, g.w};
  const int c0 = r.first_col(s);
  for (int e = 0; e < r.VW; ++e) {
    if (c0 + e < 0 || c0 + e >= r.V) continue;
    if (DT == 0) ((uint32_t *)grad)[c0 + e] = w[e % 4];
    else
      ((unsigned short *)grad)[c0 + e] =
          (unsigned short)(w[e / 2] >> (16 * (e & 1)));
  }
}

// Where a row's gradient goes: slot by slot where it lies like the student's
// row (`like`), else by the element.
template <int DT> struct GradRow {
  char *row, *slots;
  bool like;
  __device__ GradRow(void *grad, long long stride, int n,
                     const SlotRow<DT> &r) {
    row = (char *)grad + (long long)n * stride * elt_bytes<DT>();
    slots = row - r.head * elt_bytes<DT>();
    like = (reinterpret_cast<uintptr_t>(slots) & 15) == 0;
  }
  __device__ __forceinline__ void store(const SlotRow<DT> &r, int s,
                                        uint4 g) const {
    if (like && r.full(s))
      *reinterpret_cast<uint4 *>(slots + (long long)s * 16) = g;
    else
      store_partial(r, row, s, g);
  }
};

// The teacher's entries of one row, in shared memory: id (-1: padding or
// p = 0 by a logit of -inf), p, log2 p, the student's logit at the id, and P
// (NaN: unusable entries).
struct Teacher {
  alignas(16) int id[SD_MAX_DISTILL_K];
  float p[SD_MAX_DISTILL_K];
  float log2p[SD_MAX_DISTILL_K];
  float at[SD_MAX_DISTILL_K];
  float P;
};

// An entry as read: padding and logits of -inf lose their id, NaN and +inf
// become NaN.
__device__ __forceinline__ void put_entry(const DistillParams &p, Teacher &t,
                                          int k, int id, float z) {
  bool bad = false;
  if (id >= p.V) {
    status_or(p.dev_status, SD_DEV_BAD_TOKEN);
    id = -1;
  }
  if (id >= 0) {
    bad = z != z || z == kInf;
    if (z == -kInf) id = -1;
  }
  t.id[k] = id < 0 ? -1 : id;
  t.log2p[k] = bad ? __int_as_float(0x7fc00000) : z;
}

// Normalise a row's entries as put_entry left them (one warp).
__device__ void normalise(const DistillParams &p, int row, Teacher &t) {
  const int lane = threadIdx.x & 31;
  float m = -kInf;
  bool bad = false;
  for (int k = lane; k < p.K; k += 32)
    if (t.id[k] >= 0) {
      m = fmaxf(m, t.log2p[k]);
      bad = bad || t.log2p[k] != t.log2p[k];
    }
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  // sum of 2^((z - m) k2) over the entries
  float s = 0.f;
  for (int k = lane; k < p.K; k += 32)
    if (t.id[k] >= 0) s += ex2((t.log2p[k] - m) * p.k2);
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
  float tl = 0.f;
  if (p.teacher_lse) {
    tl = __ldg(p.teacher_lse + row);
    if (!(fabsf(tl) < kInf)) bad = true;
  }
  const float ls = log2f(s);
  float P = 0.f;
  for (int k = lane; k < p.K; k += 32) {
    const float z = t.log2p[k];
    const float l2 = p.teacher_lse ? (z * p.inv_T - tl) * (1.f / kLn2)
                                   : (z - m) * p.k2 - ls;
    const float pk = t.id[k] >= 0 ? ex2(l2) : 0.f;
    t.log2p[k] = l2;
    t.p[k] = pk;
    P += pk;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) P += __shfl_xor_sync(~0u, P, d);
  if (!p.teacher_lse) P = m == -kInf ? 0.f : 1.f;
  if (__any_sync(~0u, bad)) P = __int_as_float(0x7fc00000);
  if (lane == 0) t.P = P;
}

// Read and normalise a row's entries, and fetch the student's logits at the
// ids in [lo, hi) (one warp).
template <int DT>
__device__ void load_teacher(const DistillParams &p, int row, Teacher &t,
                             const SlotRow<DT> &r, int lo, int hi) {
  const int lane = threadIdx.x & 31;
  for (int k = lane; k < p.K; k += 32)
    put_entry(p, t, k, __ldg(p.id + (long long)row * p.K + k),
              __ldg(p.logit + (long long)row * p.K + k));
  if (lane < (-p.K & 3)) t.id[p.K + lane] = -1;  // read four at a time
  __syncwarp();
  constexpr int MOST = SD_MAX_DISTILL_K / 32;
  float z[MOST];  // on their way while the entries are normalised
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int k = lane + 32 * i;
    const int id = k < p.K ? t.id[k] : -1;
    z[i] = id >= lo && id < hi ? load_col(r, id) : 0.f;
  }
  normalise(p, row, t);
#pragma unroll
  for (int i = 0; i < MOST; ++i)
    if (lane + 32 * i < p.K) t.at[lane + 32 * i] = z[i];
}

// Whether entry k is the first of its id, and then the sum of p over all
// entries with that id: K x K comparisons a row, which the step hides up to
// about K = 64 (2048 rows of 128256 bf16: 198 us; 251 with K = 128, 470 with
// 256).
__device__ __forceinline__ bool first_of_id(const Teacher &t, int K, int k,
                                            float &sum) {
  const int id = t.id[k];
  bool first = true;
  sum = 0.f;
  for (int i = 0; i < K; i += 4) {
    const int4 v = *reinterpret_cast<const int4 *>(t.id + i);
    if (v.x != id && v.y != id && v.z != id && v.w != id) continue;
    const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (w[e] == id) {
        first = first && i + e >= k;
        sum += t.p[i + e];
      }
  }
  return first;
}

// The columns of the entries with ids in [lo, hi), over what the pass over
// the row wrote: the first entry of an id writes for all that repeat it.
template <int DT>
__device__ void store_entries(const DistillParams &p, const Teacher &t,
                              char *grad, int lo, int hi, float c, float P,
                              float nl2, int threads) {
  for (int k = threadIdx.x; k < p.K; k += threads) {
    const int id = t.id[k];
    float sum;
    if (id >= lo && id < hi && first_of_id(t, p.K, k, sum))
      store_elt<DT>(grad, id, c * (P * ex2(fmaf(t.at[k], p.k2, nl2)) - sum));
  }
}

// The forward call and the step: a cluster of CL CTAs per row, a contiguous
// run of its slots each, in batches of kRowThreads kBatch slots.
//
// The step goes over its run twice and keeps what it can of it in between:
// the first kKept slots in shared memory and the last batch in registers
// (each thread its own, so nothing is waited for), and it reads the rest,
// newest first, once more.  Two CTAs on an SM, each with a row, keep HBM
// busy through each other's reductions.  288 rows of 32000 fp32 forward:
// 10.0 us where reading them from HBM takes 5.5 (7.0 us out of L2).  The step
// takes this kernel where rows are few (100 such rows: 9.6 us) or too long
// for distill_step_kernel; many of the latter have a CTA each, which reads
// most of its row twice (2048 rows of 152064 fp32: 617 us, at HBM's rate 373).
constexpr int kRowThreads = 512;
constexpr int kKept = 6272;  // 98 KB a CTA

template <int DT, bool STEP>
__global__ void __launch_bounds__(kRowThreads, 2)
distill_row_kernel(const __grid_constant__ DistillParams p) {
  constexpr int VW = vec_width<DT>(), WARPS = kRowThreads / 32;
  constexpr int RUN = kRowThreads * kBatch;
  extern __shared__ __align__(16) char dyn[];
  __shared__ Teacher t;
  __shared__ MS part[WARPS], mine;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.CL > 1 ? (int)cluster.block_rank() : 0;
  const int row = blockIdx.x / p.CL;
  const SlotRow<DT> r(p.student, p.row_stride, row, p.V);
  const int s0 = (int)((long long)r.slots * rank / p.CL);
  const int s1 = (int)((long long)r.slots * (rank + 1) / p.CL);
  const float k2 = p.k2, nan = __int_as_float(0x7fc00000);
  uint4 *kept = reinterpret_cast<uint4 *>(dyn);
  const int batches = (s1 - s0 + RUN - 1) / RUN;
  Raw<DT, VW> x[kBatch];
  // before anything is written (the gradient may go to the student's rows)
  if (warp == WARPS - 1 && (rank == 0 || STEP))
    load_teacher(p, row, t, r, 0, p.V);
  MS st = ms_start(k2);
  float vmax;
  for (int b = 0; b < batches; ++b) {
    const int n = b * RUN + tid;
    if (s0 + b * RUN >= r.f0 && s0 + (b + 1) * RUN <= min(s1, r.f1)) {
      const uint4 *src = reinterpret_cast<const uint4 *>(r.base) + s0 + n;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) x[i].w = ld_v4(src + i * kRowThreads);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        ms_add_v<DT, VW>(st, x[i], k2, vmax);
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int s = s0 + n + i * kRowThreads;
        if (r.full(s) && s < s1) x[i].w = ld_v4(r.base + (long long)s * 16);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int s = s0 + n + i * kRowThreads;
        if (s >= s1) continue;
        if (!r.full(s)) x[i] = load_partial(r, s);
        ms_add_v<DT, VW>(st, x[i], k2, vmax);
      }
    }
    if (STEP && b + 1 < batches) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (n + i * kRowThreads < kKept) kept[n + i * kRowThreads] = x[i].w;
    }
  }
  st = warp_down_ms(st, k2);
  if (lane == 0) part[warp] = st;
  __syncthreads();
  if (p.CL == 1) {
    st = part[0];
    for (int i = 1; i < WARPS; ++i) st = ms_merge(st, part[i], k2);
  } else {
    if (tid == 0) {
      st = part[0];
      for (int i = 1; i < WARPS; ++i) st = ms_merge(st, part[i], k2);
      mine = st;
    }
    cluster.sync();
    st = ms_empty();
    for (int i = 0; i < p.CL; ++i)
      st = ms_merge(st, *cluster.map_shared_rank(&mine, i), k2);
  }
  const float ls = log2f(st.s);
  if (rank == 0 && warp == 0) {
    const bool ok = ms_valid(st) && t.P == t.P;
    float a = 0.f;
    for (int k = lane; k < p.K; k += 32)
      if (t.id[k] >= 0 && t.p[k] > 0.f)
        a += t.p[k] * (t.log2p[k] - ((t.at[k] - st.m) * k2 - ls));
    a = warp_down_sum(a);
    if (lane == 0) {
      p.loss[row] = ok ? a * kLn2 : nan;
      p.lse[row] = ok ? (st.m * k2 + ls) * kLn2 : nan;
      if (!ok) status_or(p.dev_status, SD_DEV_NONFINITE);
    }
  }
  if constexpr (STEP) {
    const float w = __ldg(p.grad_loss + row), P = t.P;
    const bool ok = ms_valid(st) && P == P;
    const float c = ok ? w * p.inv_T : nan, nl2 = -(st.m * k2 + ls);
    const GradRow<DT> grad(p.grad, p.grad_stride, row, r);
    for (int b = batches - 1; b >= 0; --b) {
      const int n = b * RUN + tid;
      if (b + 1 < batches) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int at = n + i * kRowThreads;
          if (at < kKept) x[i].w = kept[at];
          else if (s0 + at < s1) x[i] = load_slot(r, s0 + at);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int s = s0 + n + i * kRowThreads;
        if (s >= s1) continue;
        // a weight of 0: zeros, whatever the row holds
        const uint4 g = slot_grad<DT>(x[i], c * P, k2, nl2);
        grad.store(r, s, w == 0.f ? make_uint4(0, 0, 0, 0) : g);
      }
    }
    if (w != 0.f) {
      __syncthreads();
      store_entries<DT>(p, t, grad.row, max(0, r.first_col(s0)),
                        min(p.V, r.first_col(s1)), c, P, nl2, kRowThreads);
    }
  }
  if (p.CL > 1) cluster.sync();  // peers have read `mine`
}

// The step where there are rows enough to fill the GPU: clusters of CL CTAs,
// two CTAs an SM, take rows in turn, a contiguous run of a row's slots each.
// A row stays in shared memory from the pass that finds log sum exp to the
// pass that writes the gradient, so HBM sees each byte once.  A loading warp
// keeps a ring of 32 KB chunks full, across rows: while a row's sums are
// exchanged and its gradient is written, the next one arrives.  Two more
// warps have the teacher's entries of the next rows ready; eight do the two
// passes.  A wait that gives up (see role_wait) stops the loads; the passes
// run on over meaningless data, so that every barrier is reached.
//
// 2048 rows of 128256 bf16 (1.05 GB): 198 us, 0.79 of the measured copy rate,
// at 0.59 of the issue slots (two passes take some 60 instructions for eight
// logits).  One CTA an SM with 16 warps: 221 us; rows read twice instead,
// the second time partly out of L2: 246 us.
constexpr int kChunk = 2048;      // slots
constexpr int kRing = 3;          // chunks, 96 KB
constexpr int kMostChunks = 2;    // of a run: the rest of the ring runs ahead
constexpr int kStepWarps = 8;
constexpr int kStepThreads = 32 * (kStepWarps + 3);

struct StepShared {
  uint64_t full[kRing], empty[kRing];
  uint64_t t_full[2], t_empty[2], sum_full[2], row_full[2];
  volatile int abort;
  MS part[kStepWarps];
  alignas(8) MS sums[2][8];  // of the cluster's CTAs, two rows' worth
  alignas(8) MS row[2];      // of the whole row
  Teacher t[2];
  // a row's entries as its columns take them: the first of each id (others
  // and unused ones -1), and the sum of p over the id
  int col[2][SD_MAX_DISTILL_K];
  float sum[2][SD_MAX_DISTILL_K];
};

__device__ __forceinline__ void step_sync() {  // the warps of the passes
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kStepWarps) : "memory");
}

template <int DT>
__global__ void __launch_bounds__(kStepThreads, 2)
distill_step_kernel(const __grid_constant__ DistillParams p, int chunks) {
  constexpr int VW = vec_width<DT>();
  extern __shared__ __align__(16) char dyn[];
  uint4 *ring = reinterpret_cast<uint4 *>(dyn);
  StepShared &s =
      *reinterpret_cast<StepShared *>(dyn + kRing * kChunk * 16);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster.block_rank();
  const int clusters = gridDim.x / p.CL;
  const int first = blockIdx.x / p.CL;
  const float k2 = p.k2, nan = __int_as_float(0x7fc00000);
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kStepWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.t_full[i], 1);
      mbar_init(&s.t_empty[i], kStepWarps);
      mbar_init(&s.sum_full[i], 1);
      mbar_init(&s.row_full[i], 1);
    }
    s.abort = 0;
    fence_mbar_init();
  }
  cluster.sync();  // the peers' barriers are there
  bool fine = true;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    fine = __all_sync(~0u, fine && role_wait(bar, parity, &s.abort,
                                             p.dev_status));
  };

  if (warp == kStepWarps) {
    // ---- loads
    RingAt at(kRing);
    unsigned filled = 0;
    for (int row = first; row < p.N && fine; row += clusters) {
      const SlotRow<DT> r(p.student, p.row_stride, row, p.V);
      const int s0 = (int)((long long)r.slots * rank / p.CL);
      const int s1 = (int)((long long)r.slots * (rank + 1) / p.CL);
      for (int i = 0; i < chunks; ++i) {
        wait(&s.empty[at.slot], at.parity ^ 1);
        if (!fine) break;
        if (lane == 0) {
          const int a = max(s0 + i * kChunk, r.f0);
          const int b = min(min(s0 + (i + 1) * kChunk, s1), r.f1);
          const uint32_t bytes = b > a ? (uint32_t)(b - a) * 16 : 0;
          mbar_expect_tx(&s.full[at.slot], bytes);
          if (bytes)
            bulk_g2s_hint(ring + at.slot * kChunk + (a - s0 - i * kChunk),
                          r.base + (long long)a * 16, bytes,
                          &s.full[at.slot], l2_evict_first_policy());
        }
        at.next();
        ++filled;
      }
    }
    if (!fine)  // give up: let the copies in flight land first
      for (unsigned i = 0; i < kRing && i < filled; ++i) {
        const unsigned last = (filled - 1 - i) / kRing;
        for (unsigned it = 0; it < (1u << 20); ++it)
          if (mbar_try_wait(&s.full[i], last & 1)) break;
      }
  } else if (warp > kStepWarps) {
    // ---- the teacher's entries, and the student's logits at their ids:
    // before the row's sums leave this CTA, so before any CTA writes to the
    // row (the gradient may go to the student's own rows).  Off the other
    // warps' path, the loss.  A row's chain of loads takes longer than its
    // two passes: two warps, every other row each.
    const int me = warp - kStepWarps - 1;
    uint32_t parity = 0;
    Teacher &t = s.t[me];
    for (int row = first + me * clusters; row < p.N; row += 2 * clusters) {
      wait(&s.t_empty[me], parity ^ 1);
      if (!fine) break;
      const SlotRow<DT> r(p.student, p.row_stride, row, p.V);
      load_teacher(p, row, t, r, 0, p.V);
      __syncwarp();
      for (int k = lane; k < p.K; k += 32) {
        float sum = 0.f;
        const bool col = t.id[k] >= 0 && first_of_id(t, p.K, k, sum);
        s.col[me][k] = col ? t.id[k] : -1;
        s.sum[me][k] = sum;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.t_full[me]);
      wait(&s.row_full[me], parity);
      if (!fine) break;
      if (rank == 0) {
        const MS st = s.row[me];
        const float ls = log2f(st.s);
        const bool ok = ms_valid(st) && t.P == t.P;
        float a = 0.f;
        for (int k = lane; k < p.K; k += 32)
          if (t.id[k] >= 0 && t.p[k] > 0.f)
            a += t.p[k] * (t.log2p[k] - ((t.at[k] - st.m) * k2 - ls));
        a = warp_down_sum(a);
        if (lane == 0) {
          p.loss[row] = ok ? a * kLn2 : nan;
          p.lse[row] = ok ? (st.m * k2 + ls) * kLn2 : nan;
          if (!ok) status_or(p.dev_status, SD_DEV_NONFINITE);
        }
        __syncwarp();
      }
      parity ^= 1;
    }
  } else {
    RingAt read(kRing), write(kRing), two(2);
    for (int row = first; row < p.N; row += clusters) {
      const SlotRow<DT> r(p.student, p.row_stride, row, p.V);
      const int s0 = (int)((long long)r.slots * rank / p.CL);
      const int s1 = (int)((long long)r.slots * (rank + 1) / p.CL);
      const float w = __ldg(p.grad_loss + row);
      // ---- log sum exp
      MS st = ms_start(k2);
      float vmax;
      for (int i = 0; i < chunks; ++i) {
        wait(&s.full[read.slot], read.parity);
        const uint4 *src = ring + read.slot * kChunk + tid;
        const int lo = max(0, r.f0 - s0 - i * kChunk);
        const int hi = min(kChunk, min(s1, r.f1) - s0 - i * kChunk);
#pragma unroll
        for (int k = 0; k < kChunk; k += 32 * kStepWarps) {
          if (tid + k < lo || tid + k >= hi) continue;
          Raw<DT, VW> x;
          x.w = src[k];
          ms_add_v<DT, VW>(st, x, k2, vmax);
        }
        read.next();
      }
      // a row's partial slots: its first, and the one after the whole ones
      const int p0 = r.f0 > 0 && s0 == 0 && tid == 0 ? 0 : -1;
      const int p1 = r.f1 < r.slots && r.f1 >= s0 && r.f1 < s1 && tid == 32
                         ? r.f1 : -1;
      if (p0 >= 0) ms_add_v<DT, VW>(st, load_partial(r, p0), k2, vmax);
      if (p1 >= 0) ms_add_v<DT, VW>(st, load_partial(r, p1), k2, vmax);
      __syncwarp();
      st = warp_down_ms(st, k2);
      if (lane == 0) s.part[warp] = st;
      wait(&s.t_full[two.slot], two.parity);
      step_sync();
      if (warp == 0) {
        st = lane < kStepWarps ? s.part[lane] : ms_empty();
        st = warp_down_ms(st, k2);
        st.m = __shfl_sync(~0u, st.m, 0);
        st.s = __shfl_sync(~0u, st.s, 0);
        if (lane == 0) mbar_expect_tx(&s.sum_full[two.slot], 8 * p.CL);
        if (lane < p.CL)
          st_async_pair(&s.sums[two.slot][rank], &s.sum_full[two.slot], lane,
                        st.m, st.s);
        __syncwarp();
      }
      wait(&s.sum_full[two.slot], two.parity);
      st = ms_empty();
      for (int i = 0; i < p.CL; ++i)
        st = ms_merge(st, s.sums[two.slot][i], k2);
      const Teacher &t = s.t[two.slot];
      if (tid == 0) {
        s.row[two.slot] = st;
        mbar_arrive(&s.row_full[two.slot]);
      }
      const float P = t.P, ls = log2f(st.s);
      const bool ok = ms_valid(st) && P == P;
      // ---- the gradient; each chunk is handed back as soon as it is used
      const float c = ok ? w * p.inv_T : nan, nl2 = -(st.m * k2 + ls);
      const GradRow<DT> grad(p.grad, p.grad_stride, row, r);
      for (int i = 0; i < chunks; ++i) {
        const uint4 *src = ring + write.slot * kChunk + tid;
        const int lo = max(0, r.f0 - s0 - i * kChunk);
        const int hi = min(kChunk, min(s1, r.f1) - s0 - i * kChunk);
        uint4 *dst = reinterpret_cast<uint4 *>(grad.slots) + s0 +
                     i * kChunk + tid;
        if (w != 0.f && grad.like) {
#pragma unroll
          for (int k = 0; k < kChunk; k += 32 * kStepWarps) {
            if (tid + k < lo || tid + k >= hi) continue;
            Raw<DT, VW> x;
            x.w = src[k];
            dst[k] = slot_grad<DT>(x, c * P, k2, nl2);
          }
        } else {
          // zeros, whatever the row holds; or a gradient by the element
          for (int k = 0; k < kChunk; k += 32 * kStepWarps) {
            if (tid + k < lo || tid + k >= hi) continue;
            Raw<DT, VW> x;
            x.w = src[k];
            const uint4 g = slot_grad<DT>(x, c * P, k2, nl2);
            grad.store(r, s0 + i * kChunk + tid + k,
                       w == 0.f ? make_uint4(0, 0, 0, 0) : g);
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[write.slot]);
        write.next();
      }
      for (int part : {p0, p1})
        if (part >= 0) {
          const uint4 g =
              slot_grad<DT>(load_partial(r, part), c * P, k2, nl2);
          grad.store(r, part, w == 0.f ? make_uint4(0, 0, 0, 0) : g);
        }
      __syncwarp();
      step_sync();
      if (w != 0.f) {
        const int lo = max(0, r.first_col(s0));
        const int hi = min(p.V, r.first_col(s1));
        for (int k = tid; k < p.K; k += 32 * kStepWarps) {
          const int id = s.col[two.slot][k];
          if (id >= lo && id < hi)
            store_elt<DT>(grad.row, id,
                          c * (P * ex2(fmaf(t.at[k], k2, nl2)) -
                               s.sum[two.slot][k]));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.t_empty[two.slot]);
      two.next();
    }
  }
  __syncwarp();
  cluster.sync();  // nothing is on its way to a CTA that has ended
}

// The backward call: a CTA per row and span of up to `steps` runs of
// kBackRun slots, each run loaded while the one before it is stored.  The
// first is on its way before the teacher's chain of loads (ids, then the
// student's logits there), which every CTA of a row goes through: a span is
// as long as leaves CTAs enough to fill the GPU.  1021 rows of 152064 bf16
// (621 MB): 103 us, 0.90 of the measured copy rate; a CTA for each run of
// 2048 slots took 125 to 145 us, waiting for that chain.
constexpr int kBackBatch = 4;
constexpr int kBackRun = kThreads * kBackBatch;
constexpr int kBackSteps = 8;

template <int DT>
__global__ void __launch_bounds__(kThreads, 4)
distill_backward_kernel(const __grid_constant__ DistillParams p, int steps) {
  constexpr int VW = vec_width<DT>();
  __shared__ Teacher t;
  const int row = blockIdx.x, tid = threadIdx.x;
  const SlotRow<DT> r(p.student, p.row_stride, row, p.V);
  const int s0 = blockIdx.y * steps * kBackRun;
  const int s1 = min(s0 + steps * kBackRun, r.slots);
  if (s0 >= s1) return;
  const GradRow<DT> grad(p.grad, p.grad_stride, row, r);
  const float w = __ldg(p.grad_loss + row);
  if (w == 0.f) {  // the row is not read
    for (int s = s0 + tid; s < s1; s += kThreads)
      grad.store(r, s, make_uint4(0, 0, 0, 0));
    return;
  }
  Raw<DT, VW> x[kBackBatch], y[kBackBatch];
  // whole slots only; the others are read when they are written
  auto fetch = [&](Raw<DT, VW> *v, int s) {
#pragma unroll
    for (int i = 0; i < kBackBatch; ++i) {
      const int at = s + tid + i * kThreads;
      if (at < s1 && r.full(at)) v[i].w = ld_v4(r.base + (long long)at * 16);
    }
  };
  fetch(x, s0);
  const int lo = max(0, r.first_col(s0)), hi = min(p.V, r.first_col(s1));
  if (tid < 32) load_teacher(p, row, t, r, lo, hi);
  const float lse = __ldg(p.lse_in + row);
  __syncthreads();
  const float P = t.P;
  const bool ok = P == P && fabsf(lse) < kInf;
  if (!ok && tid == 0) status_or(p.dev_status, SD_DEV_NONFINITE);
  const float c = ok ? w * p.inv_T : __int_as_float(0x7fc00000);
  const float nl2 = -lse * (1.f / kLn2);
  auto store = [&](const Raw<DT, VW> *v, int s) {
#pragma unroll
    for (int i = 0; i < kBackBatch; ++i) {
      const int at = s + tid + i * kThreads;
      if (at < s1 && r.full(at) && grad.like)
        *reinterpret_cast<uint4 *>(grad.slots + (long long)at * 16) =
            slot_grad<DT>(v[i], c * P, p.k2, nl2);
    }
  };
  for (int s = s0; s < s1; s += 2 * kBackRun) {
    fetch(y, s + kBackRun);
    store(x, s);
    fetch(x, s + 2 * kBackRun);
    store(y, s + kBackRun);
  }
  // a row's partial slots, and all of one whose gradient lies differently
  if (!grad.like) {
    for (int s = s0 + tid; s < s1; s += kThreads)
      grad.store(r, s, slot_grad<DT>(load_slot(r, s), c * P, p.k2, nl2));
  } else if (tid < 2) {
    const int s = tid == 0 ? 0 : r.f1;
    if (s >= s0 && s < s1 && !r.full(s) && (tid == 1 || r.f0 > 0))
      grad.store(r, s, slot_grad<DT>(load_partial(r, s), c * P, p.k2, nl2));
  }
  __syncthreads();
  store_entries<DT>(p, t, grad.row, lo, hi, c, P, nl2, kThreads);
}

sd_status check_distill(const void *student, long long row_stride,
                        sd_dtype dt, const float *logit, const int32_t *id,
                        int N, int V, int K, float T) {
  SDV_REQUIRE(dt == SD_F32 || dt == SD_BF16, "bad dtype %d", (int)dt);
  SDV_REQUIRE(N >= 0, "N < 0");
  SDV_REQUIRE(V >= 1 && V <= SD_MAX_V, "V=%d outside [1, %d]", V, SD_MAX_V);
  SDV_REQUIRE(K >= 1 && K <= SD_MAX_DISTILL_K, "K=%d outside [1, %d]", K,
              SD_MAX_DISTILL_K);
  SDV_REQUIRE(T > 0.f && std::isfinite(T), "T must be finite and > 0");
  SDV_REQUIRE(row_stride >= V, "row_stride < V");
  SDV_REQUIRE(N == 0 || (student && logit && id), "null pointer");
  return SD_OK;
}

// Slots a row of V columns can take, wherever it starts.
int max_slots(int V, sd_dtype dt) {
  const int vw = dt == SD_F32 ? 4 : 8;
  return (V + 2 * vw - 2) / vw;
}

// The ring kernel, where a run fits and there are rows for every SM; *done
// says whether it took the call.
sd_status launch_step(DistillParams &p, sd_dtype dt, int sms, cudaStream_t s,
                      bool *done) {
  *done = false;
  const int slots = max_slots(p.V, dt);
  constexpr int run = kMostChunks * kChunk - 1;  // shares differ by one slot
  const int cl = (slots + run - 1) / run;
  if (cl > 8 || (long long)p.N * cl < sms) return SD_OK;
  int chunks = (slots / cl + 1 + kChunk - 1) / kChunk;
  const void *kernel = dt == SD_F32 ? (const void *)distill_step_kernel<0>
                                    : (const void *)distill_step_kernel<1>;
  const size_t smem = (size_t)kRing * kChunk * 16 + sizeof(StepShared);
  int resident = 0;
  const sd_status st =
      max_active_clusters(kernel, cl, smem, &resident, kStepThreads);
  if (st != SD_OK) return st;
  p.CL = cl;
  const int clusters = p.N < resident ? p.N : resident;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * cl), 1, 1);
  cfg.blockDim = dim3(kStepThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *args[] = {&p, &chunks};
  SDV_CUDA(cudaLaunchKernelExC(&cfg, kernel, args));
  *done = true;
  return SD_OK;
}

// In clusters of as many CTAs per row as it takes to fill the GPU, each with
// at least 512 slots.
template <bool STEP>
sd_status launch_rows(DistillParams &p, sd_dtype dt, int sms,
                      cudaStream_t s) {
  const int slots = max_slots(p.V, dt);
  int cl = 1;
  while (cl < 8 && (long long)p.N * cl <= sms && slots / (2 * cl) >= 512)
    cl *= 2;
  p.CL = cl;
  const void *kernel = dt == SD_F32 ? (const void *)distill_row_kernel<0, STEP>
                                    : (const void *)distill_row_kernel<1, STEP>;
  // a run of one batch stays in registers
  const int run = slots / cl + 1;
  const size_t smem =
      STEP && run > kRowThreads * kBatch ? kKept * 16 : 0;
  if (smem) {
    int dev = 0;
    SDV_CUDA(cudaGetDevice(&dev));
    static std::atomic<unsigned long long> ready[2];
    std::atomic<unsigned long long> &have = ready[dt == SD_F32 ? 0 : 1];
    if (dev >= 64 || !(have.load() >> dev & 1)) {
      SDV_CUDA(cudaFuncSetAttribute(
          kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
      if (dev < 64) have.fetch_or(1ull << dev);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.N * (unsigned)cl, 1, 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *args[] = {&p};
  SDV_CUDA(cudaLaunchKernelExC(&cfg, kernel, args));
  return SD_OK;
}

DistillParams distill_params(const void *student, long long row_stride,
                             const float *logit, const int32_t *id,
                             const float *teacher_lse, int N, int V, int K,
                             float T, int32_t *dev_status) {
  DistillParams p = {};
  p.student = student;
  p.row_stride = row_stride;
  p.logit = logit;
  p.id = id;
  p.teacher_lse = teacher_lse;
  p.N = N;
  p.V = V;
  p.K = K;
  p.k2 = (float)(1.4426950408889634 / (double)T);
  p.inv_T = (float)(1.0 / (double)T);
  p.dev_status = dev_status;
  return p;
}

}  // namespace
}  // namespace sdv

using namespace sdv;

extern "C" sd_status sd_distill_topk(
    const void *student, long long row_stride, sd_dtype dt,
    const float *teacher_logit, const int32_t *teacher_id,
    const float *teacher_lse, int N, int V, int K, float T, float *loss,
    float *lse, int32_t *dev_status, void *stream) {
  sd_status st = check_distill(student, row_stride, dt, teacher_logit,
                               teacher_id, N, V, K, T);
  if (st != SD_OK) return st;
  if (N == 0) return SD_OK;
  SDV_REQUIRE(loss && lse, "null pointer");
  int sms = 0;
  st = check_device(&sms);
  if (st != SD_OK) return st;
  DistillParams p =
      distill_params(student, row_stride, teacher_logit, teacher_id,
                     teacher_lse, N, V, K, T, dev_status);
  p.loss = loss;
  p.lse = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_rows<false>(p, dt, sms, s);
}

extern "C" sd_status sd_distill_topk_backward(
    const void *student, long long row_stride, sd_dtype dt, const float *lse,
    const float *teacher_logit, const int32_t *teacher_id,
    const float *teacher_lse, const float *grad_loss, int N, int V, int K,
    float T, void *grad, long long grad_stride, int32_t *dev_status,
    void *stream) {
  sd_status st = check_distill(student, row_stride, dt, teacher_logit,
                               teacher_id, N, V, K, T);
  if (st != SD_OK) return st;
  SDV_REQUIRE(grad_stride >= V, "grad_stride < V");
  if (N == 0) return SD_OK;
  SDV_REQUIRE(lse && grad_loss && grad, "null pointer");
  int sms = 0;
  st = check_device(&sms);
  if (st != SD_OK) return st;
  DistillParams p =
      distill_params(student, row_stride, teacher_logit, teacher_id,
                     teacher_lse, N, V, K, T, dev_status);
  p.lse_in = lse;
  p.grad_loss = grad_loss;
  p.grad = grad;
  p.grad_stride = grad_stride;
  const int runs = (max_slots(V, dt) + kBackRun - 1) / kBackRun;
  int steps = kBackSteps;
  while (steps > 1 && (long long)N * ((runs + steps - 1) / steps) < 10LL * sms)
    steps /= 2;
  const dim3 grid(N, (runs + steps - 1) / steps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == SD_F32)
    distill_backward_kernel<0><<<grid, kThreads, 0, s>>>(p, steps);
  else distill_backward_kernel<1><<<grid, kThreads, 0, s>>>(p, steps);
  SDV_CUDA(cudaGetLastError());
  return SD_OK;
}

extern "C" sd_status sd_distill_topk_step(
    const void *student, long long row_stride, sd_dtype dt,
    const float *teacher_logit, const int32_t *teacher_id,
    const float *teacher_lse, const float *grad_loss, int N, int V, int K,
    float T, float *loss, float *lse, void *grad, long long grad_stride,
    int32_t *dev_status, void *stream) {
  sd_status st = check_distill(student, row_stride, dt, teacher_logit,
                               teacher_id, N, V, K, T);
  if (st != SD_OK) return st;
  SDV_REQUIRE(grad_stride >= V, "grad_stride < V");
  if (N == 0) return SD_OK;
  SDV_REQUIRE(loss && lse && grad_loss && grad, "null pointer");
  int sms = 0;
  st = check_device(&sms);
  if (st != SD_OK) return st;
  DistillParams p =
      distill_params(student, row_stride, teacher_logit, teacher_id,
                     teacher_lse, N, V, K, T, dev_status);
  p.loss = loss;
  p.lse = lse;
  p.grad_loss = grad_loss;
  p.grad = grad;
  p.grad_stride = grad_stride;
  bool done = false;
  st = launch_step(p, dt, sms, static_cast<cudaStream_t>(stream), &done);
  if (st != SD_OK || done) return st;
  return launch_rows<true>(p, dt, sms, static_cast<cudaStream_t>(stream));
}
