// sdv_distill.cu -- sd_distill_topk and its gradient: distillation of a
// drafter from the target's top logits.
//
// With p the teacher's probabilities of its K entries, P their sum and q =
// softmax(z / T) of the student's row,
//   loss = sum_k p_k (log p_k - log q_k)
//   d loss / d z_j = (P q_j - sum_{k: id_k = j} p_k) / T.
//
// All three calls stream vocabulary rows and are bound by HBM: the forward
// call reads a row once, the backward call reads and writes it once, and so
// does the step, which keeps a row in the shared memory of a cluster between
// the pass that finds log sum exp and the pass that writes the gradient.
//
// A row is cut into 16-byte slots by address, whatever its own alignment:
// only its first and last slot can be partial, and those alone are read and
// written by the element.
#include "sdv_device.cuh"
#include "sdv_host.cuh"
#include "sdv_tma.cuh"

namespace sdv {
namespace {

constexpr float kLn2 = 0.693147180559945f;
constexpr int kSlotsPerCopy = 1024;  // 16 KB a bulk copy
constexpr int kMaxCopies = 5;        // a step's slice of a row
constexpr int kBatch = 8;            // slots a thread has in flight

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
// column j is element head + j.
template <int DT> struct SlotRow {
  static constexpr int VW = vec_width<DT>();
  const char *base;
  int head, V, slots;
  __device__ SlotRow(const void *rows, long long stride, int row, int V_)
      : V(V_) {
    const char *start =
        (const char *)rows + (long long)row * stride * elt_bytes<DT>();
    head = (int)(reinterpret_cast<uintptr_t>(start) & 15) / elt_bytes<DT>();
    base = start - head * elt_bytes<DT>();
    slots = (head + V + VW - 1) / VW;
  }
  __device__ bool full(int s) const {
    return (s > 0 || head == 0) && (s + 1) * VW <= head + V;
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
__device__ Raw<DT, vec_width<DT>()> load_partial(const SlotRow<DT> &r, int s) {
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

// Gradients of a slot: c 2^(z k2 + nl2) of its columns (c alone scales).
template <int DT>
__device__ __forceinline__ void store_slot(
    const SlotRow<DT> &r, char *grad, bool aligned, int s,
    const Raw<DT, vec_width<DT>()> &x, float c, float k2, float nl2) {
  float g[SlotRow<DT>::VW];
#pragma unroll
  for (int e = 0; e < r.VW; ++e)
    g[e] = c * ex2(fmaf(elt<DT, SlotRow<DT>::VW>(x, e), k2, nl2));
  const int c0 = r.first_col(s);
  if (aligned && r.full(s)) {
    uint4 w;
    if constexpr (DT == 0) {
      w = make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]),
                     __float_as_uint(g[2]), __float_as_uint(g[3]));
    } else {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
            : "=r"(u[e])
            : "f"(g[2 * e + 1]), "f"(g[2 * e]));
      w = make_uint4(u[0], u[1], u[2], u[3]);
    }
    *reinterpret_cast<uint4 *>(grad + (long long)c0 * elt_bytes<DT>()) = w;
  } else {
    for (int e = 0; e < r.VW; ++e)
      if (c0 + e >= 0 && c0 + e < r.V) store_elt<DT>(grad, c0 + e, g[e]);
  }
}

// The teacher's entries of one row, in shared memory: id (-1: padding or
// p = 0 by a logit of -inf), p, log2 p, and P (NaN: unusable entries).
struct Teacher {
  int id[SD_MAX_DISTILL_K];
  float p[SD_MAX_DISTILL_K];
  float log2p[SD_MAX_DISTILL_K];
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

// Read and normalise a row's entries (one warp).
__device__ void load_teacher(const DistillParams &p, int row, Teacher &t) {
  for (int k = threadIdx.x & 31; k < p.K; k += 32)
    put_entry(p, t, k, __ldg(p.id + (long long)row * p.K + k),
              __ldg(p.logit + (long long)row * p.K + k));
  __syncwarp();
  normalise(p, row, t);
}

// The columns of the entries with ids in [lo, hi), over what the pass over
// the row wrote: the first entry of an id writes for all that repeat it.
// at: the student's logits at the ids.
template <int DT>
__device__ void store_entries(const DistillParams &p, const Teacher &t,
                              char *grad, int lo, int hi, const float *at,
                              float c, float P, float nl2) {
  for (int k = threadIdx.x; k < p.K; k += kThreads) {
    const int id = t.id[k];
    if (id < lo || id >= hi) continue;
    float sum = 0.f;
    bool first = true;
    for (int i = 0; i < p.K; ++i)
      if (t.id[i] == id) {
        first = first && i >= k;
        sum += t.p[i];
      }
    if (first)
      store_elt<DT>(grad, id, c * (P * ex2(fmaf(at[k], p.k2, nl2)) - sum));
  }
}

// (max, sum) of a row's slots: this thread's part in, the cluster's out.
// Every CTA merges the parts in rank order.  A CTA that is a row ahead may
// not change what a peer still reads: rows alternate between the two `mine`.
struct RowReduce {
  MS part[kWarps], mine[2];
};
__device__ __forceinline__ MS reduce_row(MS st, float k2, int CL,
                                         RowReduce &red, int which,
                                         cg::cluster_group &cluster) {
  const int tid = threadIdx.x;
  st = warp_down_ms(st, k2);
  if ((tid & 31) == 0) red.part[tid >> 5] = st;
  __syncthreads();
  if (tid == 0) {
    st = red.part[0];
    for (int i = 1; i < kWarps; ++i) st = ms_merge(st, red.part[i], k2);
    red.mine[which] = st;
  }
  cluster.sync();
  st = ms_empty();
  for (int i = 0; i < CL; ++i)
    st = ms_merge(st, *cluster.map_shared_rank(&red.mine[which], i), k2);
  return st;
}

// The forward call: a cluster of CL CTAs per row, a contiguous run of its
// slots each.
template <int DT>
__global__ void __launch_bounds__(kThreads)
distill_forward_kernel(const __grid_constant__ DistillParams p) {
  constexpr int VW = vec_width<DT>();
  __shared__ Teacher t;
  __shared__ float at[SD_MAX_DISTILL_K];
  __shared__ RowReduce red;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster.block_rank();
  const int row = blockIdx.x / p.CL;
  const SlotRow<DT> r(p.student, p.row_stride, row, p.V);
  const int s0 = (int)((long long)r.slots * rank / p.CL);
  const int s1 = (int)((long long)r.slots * (rank + 1) / p.CL);
  const float k2 = p.k2;
  if (rank == 0 && warp == kWarps - 1) {
    load_teacher(p, row, t);
    __syncwarp();
    for (int k = lane; k < p.K; k += 32)
      at[k] = t.id[k] >= 0 ? load_col(r, t.id[k]) : 0.f;
  }
  MS st = ms_empty();
  float vmax;
  for (int s = s0 + tid; s < s1; s += kThreads * kBatch) {
    Raw<DT, VW> x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (s + i * kThreads < s1) x[i] = load_slot(r, s + i * kThreads);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (s + i * kThreads < s1) ms_add_v<DT, VW>(st, x[i], k2, vmax);
  }
  st = reduce_row(st, k2, p.CL, red, 0, cluster);
  if (rank == 0 && warp == 0) {
    const float ls = log2f(st.s), nan = __int_as_float(0x7fc00000);
    const bool ok = ms_valid(st) && t.P == t.P;
    float a = 0.f;
    for (int k = lane; k < p.K; k += 32)
      if (t.id[k] >= 0 && t.p[k] > 0.f)
        a += t.p[k] * (t.log2p[k] - ((at[k] - st.m) * k2 - ls));
    a = warp_down_sum(a);
    if (lane == 0) {
      p.loss[row] = ok ? a * kLn2 : nan;
      p.lse[row] = ok ? (st.m * k2 + ls) * kLn2 : nan;
      if (!ok) status_or(p.dev_status, SD_DEV_NONFINITE);
    }
  }
  cluster.sync();  // peers have read `red`
}

// The step: clusters of CL CTAs take rows in turn and keep a row in their
// shared memory (bulk copies of up to 16 KB, a barrier each) from the pass
// that finds log sum exp to the pass that writes the gradient.  The second
// pass hands a copy's space to the next row as soon as it has used it, so
// loads and stores overlap within a CTA as well as between the three on an
// SM; the next row's teacher entries are fetched a row ahead.
template <int DT>
__global__ void __launch_bounds__(kThreads)
distill_step_kernel(const __grid_constant__ DistillParams p) {
  constexpr int VW = vec_width<DT>();
  extern __shared__ __align__(16) char kept[];
  __shared__ Teacher t;
  __shared__ float at[SD_MAX_DISTILL_K], entry_loss[2];
  __shared__ RowReduce red;
  __shared__ uint64_t bar[kMaxCopies];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster.block_rank();
  const int clusters = gridDim.x / p.CL;
  const float k2 = p.k2, nan = __int_as_float(0x7fc00000);
  uint4 *slot = reinterpret_cast<uint4 *>(kept);
  // this CTA's run of a row's slots; [f0, f1) are whole
  struct Run {
    int s0, s1, f0, f1;
  };
  auto run_of = [&](const SlotRow<DT> &r) {
    Run u;
    u.s0 = (int)((long long)r.slots * rank / p.CL);
    u.s1 = (int)((long long)r.slots * (rank + 1) / p.CL);
    u.f0 = u.s0 + (u.s1 > u.s0 && !r.full(u.s0));
    u.f1 = u.s1 - (u.s1 > u.f0 && !r.full(u.s1 - 1));
    return u;
  };
  // copy i of a row (thread 0)
  auto fetch = [&](const SlotRow<DT> &r, const Run &u, int i) {
    const int a = max(u.s0 + i * kSlotsPerCopy, u.f0);
    const int b = min(u.s0 + (i + 1) * kSlotsPerCopy, u.f1);
    const uint32_t bytes = b > a ? (uint32_t)(b - a) * 16 : 0;
    mbar_expect_tx(&bar[i], bytes);
    if (bytes)
      bulk_g2s_hint(slot + (a - u.s0), r.base + (long long)a * 16, bytes,
                    &bar[i], l2_evict_first_policy());
  };
  if (tid == 0) {
    for (int i = 0; i < kMaxCopies; ++i) mbar_init(&bar[i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  int row = blockIdx.x / p.CL;
  SlotRow<DT> r(p.student, p.row_stride, row, p.V);
  Run u = run_of(r);
  if (tid == 0)
    for (int i = 0; i < kMaxCopies; ++i) fetch(r, u, i);
  auto entry_of = [&](int n, int &id, float &z) {
    id = -1;
    z = 0.f;
    if (n < p.N && tid < p.K) {
      id = __ldg(p.id + (long long)n * p.K + tid);
      z = __ldg(p.logit + (long long)n * p.K + tid);
    }
  };
  static_assert(SD_MAX_DISTILL_K <= kThreads, "an entry a thread");
  int id;
  float z;
  entry_of(row, id, z);
  uint32_t parity = 0;
  int last = -1;  // the row whose loss is being added up
  bool last_ok = false;
  // rank 0, after a cluster barrier: the loss of row `last`
  auto finish_loss = [&] {
    if (rank == 0 && warp == 0 && last >= 0) {
      float a = lane < p.CL
                    ? *cluster.map_shared_rank(&entry_loss[parity ^ 1], lane)
                    : 0.f;
      a = warp_down_sum(a);
      if (lane == 0) p.loss[last] = last_ok ? a * kLn2 : nan;
    }
  };
  for (; row < p.N; row += clusters) {
    const int n = u.s1 - u.s0;
    if (tid < p.K) put_entry(p, t, tid, id, z);
    entry_of(row + clusters, id, z);
    if (tid == 32 && u.f0 > u.s0) slot[0] = load_partial(r, u.s0).w;
    if (tid == 64 && u.f1 < u.s1) slot[n - 1] = load_partial(r, u.s1 - 1).w;
    __syncthreads();
    if (warp == kWarps - 1) normalise(p, row, t);
    MS st = ms_empty();
    float vmax;
    for (int i = 0; i < kMaxCopies; ++i) {
      mbar_wait(&bar[i], parity, p.dev_status);
      const int b = min((i + 1) * kSlotsPerCopy, n);
#pragma unroll 4
      for (int s = i * kSlotsPerCopy + tid; s < b; s += kThreads) {
        Raw<DT, VW> x;
        x.w = slot[s];
        ms_add_v<DT, VW>(st, x, k2, vmax);
      }
    }
    st = reduce_row(st, k2, p.CL, red, parity, cluster);
    finish_loss();
    const float P = t.P;
    const bool ok = ms_valid(st) && P == P;
    const float ls = log2f(st.s);
    const int lo = max(0, r.first_col(u.s0));
    const int hi = min(p.V, r.first_col(u.s1));
    // the entries in this run: their logits and their part of the loss
    float a = 0.f;
    if (tid < p.K && t.id[tid] >= lo && t.id[tid] < hi) {
      const int c = t.id[tid] - r.first_col(u.s0);
      const char *src = kept + (long long)c * elt_bytes<DT>();
      const float x =
          DT == 0 ? *reinterpret_cast<const float *>(src)
                  : __uint_as_float(
                        (uint32_t)*reinterpret_cast<const unsigned short *>(src)
                        << 16);
      at[tid] = x;
      if (t.p[tid] > 0.f)
        a = t.p[tid] * (t.log2p[tid] - ((x - st.m) * k2 - ls));
    }
    __shared__ float loss_part[kWarps];
    a = warp_down_sum(a);
    if (lane == 0) loss_part[warp] = a;
    if (rank == 0 && tid == 0) {
      p.lse[row] = ok ? (st.m * k2 + ls) * kLn2 : nan;
      if (!ok) status_or(p.dev_status, SD_DEV_NONFINITE);
    }
    last = row;
    last_ok = ok;
    // the gradient, and the next row into the space of the copies used up
    const float w = __ldg(p.grad_loss + row);
    const float c = w == 0.f ? 0.f : ok ? w * p.inv_T : nan;
    const float nl2 = -(st.m * k2 + ls);
    char *grad =
        (char *)p.grad + (long long)row * p.grad_stride * elt_bytes<DT>();
    const bool aligned = ((reinterpret_cast<uintptr_t>(grad) & 15) /
                          elt_bytes<DT>()) == (unsigned)r.head;
    const SlotRow<DT> next(p.student, p.row_stride,
                           min(row + clusters, p.N - 1), p.V);
    const Run nu = run_of(next);
    for (int i = 0; i < kMaxCopies; ++i) {
      const int b = min((i + 1) * kSlotsPerCopy, n);
#pragma unroll 4
      for (int s = i * kSlotsPerCopy + tid; s < b; s += kThreads) {
        Raw<DT, VW> x;
        // a weight of 0: zeros, whatever the row holds
        x.w = w == 0.f ? make_uint4(0, 0, 0, 0) : slot[s];
        store_slot<DT>(r, grad, aligned, u.s0 + s, x, w == 0.f ? 0.f : c * P,
                       w == 0.f ? 0.f : k2, w == 0.f ? 0.f : nl2);
      }
      fence_proxy_async();
      __syncthreads();
      if (tid == 0 && row + clusters < p.N) fetch(next, nu, i);
    }
    if (tid == 0) {
      float sum = 0.f;
      for (int i = 0; i < kWarps; ++i) sum += loss_part[i];
      entry_loss[parity] = sum;
    }
    if (w != 0.f) store_entries<DT>(p, t, grad, lo, hi, at, c, P, nl2);
    __syncthreads();  // t, at and the parts may change
    r = next;
    u = nu;
    parity ^= 1;
  }
  cluster.sync();
  finish_loss();
  cluster.sync();  // peers have read entry_loss
}

// The backward call: a CTA per row and run of kThreads kBatch slots.
template <int DT>
__global__ void __launch_bounds__(kThreads)
distill_backward_kernel(const __grid_constant__ DistillParams p) {
  constexpr int VW = vec_width<DT>();
  __shared__ Teacher t;
  __shared__ float at[SD_MAX_DISTILL_K];
  const int row = blockIdx.x, tid = threadIdx.x;
  const SlotRow<DT> r(p.student, p.row_stride, row, p.V);
  const int s0 = blockIdx.y * (kThreads * kBatch);
  const int s1 = min(s0 + kThreads * kBatch, r.slots);
  if (s0 >= s1) return;
  char *grad =
      (char *)p.grad + (long long)row * p.grad_stride * elt_bytes<DT>();
  const bool aligned = ((reinterpret_cast<uintptr_t>(grad) & 15) /
                        elt_bytes<DT>()) == (unsigned)r.head;
  const float w = __ldg(p.grad_loss + row);
  Raw<DT, VW> x[kBatch];
  if (w != 0.f) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (s0 + tid + i * kThreads < s1)
        x[i] = load_slot(r, s0 + tid + i * kThreads);
  }
  const int lo = max(0, r.first_col(s0)), hi = min(p.V, r.first_col(s1));
  float P = 0.f, c = 0.f, nl2 = 0.f;
  if (w != 0.f) {
    if (tid < 32) load_teacher(p, row, t);
    __syncthreads();
    P = t.P;
    const float lse = __ldg(p.lse_in + row);
    const bool ok = P == P && fabsf(lse) < kInf;
    if (!ok && tid == 0) status_or(p.dev_status, SD_DEV_NONFINITE);
    c = ok ? w * p.inv_T : __int_as_float(0x7fc00000);
    nl2 = -lse * (1.f / kLn2);
    // before any of this CTA's columns is written
    for (int k = tid; k < p.K; k += kThreads)
      if (t.id[k] >= lo && t.id[k] < hi)
        at[k] = load_col(r, t.id[k]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int s = s0 + tid + i * kThreads;
    if (s >= s1) continue;
    if (w == 0.f) x[i].w = make_uint4(0, 0, 0, 0);
    store_slot<DT>(r, grad, aligned, s, x[i], c * P, w == 0.f ? 0.f : p.k2,
                   nl2);
  }
  if (w == 0.f) return;
  __syncthreads();
  store_entries<DT>(p, t, grad, lo, hi, at, c, P, nl2);
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

// CTAs per row of the forward call: enough for some eight on every SM, each
// with at least 512 slots.
int forward_cluster(int N, int slots, int sms) {
  int cl = 1;
  while (cl < 8 && (long long)N * cl < 4LL * sms && slots / (2 * cl) >= 512)
    cl *= 2;
  return cl;
}

// CTAs per row of the step, 0 where a row does not fit their shared memory:
// slices of at most 70 KB (three CTAs on an SM: one loads while another
// writes), smaller ones while there are too few rows to fill the GPU.
int step_cluster(int N, int slots, int sms) {
  constexpr int kMost = 4480;
  int cl = (slots + kMost - 1) / kMost;
  if (cl > 16) return 0;
  if (cl > 8) return 16;
  while (cl <= 4 && (long long)N * cl < sms && slots / (2 * cl) >= 512) cl *= 2;
  return cl;
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
  const void *kernel = dt == SD_F32 ? (const void *)distill_forward_kernel<0>
                                    : (const void *)distill_forward_kernel<1>;
  p.CL = forward_cluster(N, max_slots(V, dt), sms);
  void *args[] = {&p};
  return launch_clusters(kernel, N, p.CL, 0, s, args);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int run = kThreads * kBatch;
  const dim3 grid(N, (max_slots(V, dt) + run - 1) / run);
  if (dt == SD_F32) distill_backward_kernel<0><<<grid, kThreads, 0, s>>>(p);
  else distill_backward_kernel<1><<<grid, kThreads, 0, s>>>(p);
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
  const int slots = max_slots(V, dt), cl = step_cluster(N, slots, sms);
  if (cl == 0) {  // rows too long to keep: read them twice
    st = sd_distill_topk(student, row_stride, dt, teacher_logit, teacher_id,
                         teacher_lse, N, V, K, T, loss, lse, dev_status,
                         stream);
    if (st != SD_OK) return st;
    return sd_distill_topk_backward(
        student, row_stride, dt, lse, teacher_logit, teacher_id, teacher_lse,
        grad_loss, N, V, K, T, grad, grad_stride, dev_status, stream);
  }
  DistillParams p =
      distill_params(student, row_stride, teacher_logit, teacher_id,
                     teacher_lse, N, V, K, T, dev_status);
  p.loss = loss;
  p.lse = lse;
  p.grad_loss = grad_loss;
  p.grad = grad;
  p.grad_stride = grad_stride;
  const void *kernel = dt == SD_F32 ? (const void *)distill_step_kernel<0>
                                    : (const void *)distill_step_kernel<1>;
  const size_t smem = (size_t)(slots / cl + 2) * 16;
  int resident = 0;
  st = max_active_clusters(kernel, cl, smem, &resident);
  if (st != SD_OK) return st;
  p.CL = cl;
  void *args[] = {&p};
  return launch_clusters(kernel, N < resident ? N : resident, cl, smem,
                         static_cast<cudaStream_t>(stream), args);
}
