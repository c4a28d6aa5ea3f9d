// sdv_distill.cu -- sd_distill_topk and its gradient: distillation of a
// drafter from the target's top logits.
//
// With p the teacher's probabilities of its K entries, P their sum and q =
// softmax(z / T) of the student's row,
//   loss = sum_k p_k (log p_k - log q_k)
//   d loss / d z_j = (P q_j - sum_{k: id_k = j} p_k) / T.
#include "sdv_device.cuh"
#include "sdv_host.cuh"

namespace sdv {
namespace {

constexpr float kLn2 = 0.693147180559945f;

struct DistillParams {
  const void *student;
  long long row_stride;
  const float *logit, *teacher_lse, *grad_loss;
  const int32_t *id;
  int N, V, K;
  float k2;     // log2(e) / T
  float inv_T;
  float *loss, *lse;
  const float *lse_in;
  void *grad;
  long long grad_stride;
  int32_t *dev_status;
};

// The teacher's entries of one row, in shared memory: id (-1: padding or
// p = 0 by a logit of -inf), p and log2 p.
struct Teacher {
  int id[SD_MAX_DISTILL_K];
  float p[SD_MAX_DISTILL_K];
  float log2p[SD_MAX_DISTILL_K];
};

// Reads a row's entries and normalises them (all threads of the CTA call
// it); returns P, NaN when the entries are unusable.
__device__ float load_teacher(const DistillParams &p, int row, Teacher &t,
                              float *scratch) {
  const int tid = threadIdx.x;
  int st = 0;
  float m = -kInf;
  bool bad = false;
  for (int k = tid; k < p.K; k += kThreads) {
    int id = p.id[(long long)row * p.K + k];
    const float z = p.logit[(long long)row * p.K + k];
    if (id >= p.V) {
      st |= SD_DEV_BAD_TOKEN;
      id = -1;
    }
    if (id >= 0) {
      if (z != z || z == kInf) bad = true;
      if (z == -kInf) id = -1;
    }
    t.id[k] = id < 0 ? -1 : id;
    t.log2p[k] = z;
    if (id >= 0) m = fmaxf(m, z);
  }
  status_or(p.dev_status, st);
  const bool any_bad = __syncthreads_or(bad);
  scratch[tid] = m;
  __syncthreads();
  for (int i = kThreads / 2; i; i >>= 1) {
    if (tid < i) scratch[tid] = fmaxf(scratch[tid], scratch[tid + i]);
    __syncthreads();
  }
  m = scratch[0];
  __syncthreads();
  // sum of 2^((z - m) k2) over the entries
  float s = 0.f;
  for (int k = tid; k < p.K; k += kThreads)
    if (t.id[k] >= 0) s += ex2((t.log2p[k] - m) * p.k2);
  scratch[tid] = s;
  __syncthreads();
  for (int i = kThreads / 2; i; i >>= 1) {
    if (tid < i) scratch[tid] += scratch[tid + i];
    __syncthreads();
  }
  s = scratch[0];
  __syncthreads();
  float tl = 0.f;
  bool tl_bad = false;
  if (p.teacher_lse) {
    tl = p.teacher_lse[row];
    tl_bad = !(fabsf(tl) < kInf);
  }
  const float ls = log2f(s);
  for (int k = tid; k < p.K; k += kThreads) {
    const float z = t.log2p[k];
    float l2 = p.teacher_lse ? (z * p.inv_T - tl) * (1.f / kLn2)
                             : (z - m) * p.k2 - ls;
    t.log2p[k] = l2;
    t.p[k] = t.id[k] >= 0 ? ex2(l2) : 0.f;
  }
  __syncthreads();
  float P = 1.f;
  if (m == -kInf) P = 0.f;  // no usable entry
  else if (p.teacher_lse) {
    P = 0.f;
    for (int k = 0; k < p.K; ++k) P += t.p[k];
  }
  return any_bad || tl_bad ? __int_as_float(0x7fc00000) : P;
}

// One CTA per row.
template <int DT>
__global__ void __launch_bounds__(kThreads)
distill_forward_kernel(const __grid_constant__ DistillParams p) {
  __shared__ Teacher t;
  __shared__ float scratch[kThreads];
  const int row = blockIdx.x, tid = threadIdx.x;
  const char *z = (const char *)p.student +
                  (long long)row * p.row_stride * elt_bytes<DT>();
  const float P = load_teacher(p, row, t, scratch);
  MS st = ms_empty();
  float vmax;
  for (int j = tid; j < p.V; j += kThreads)
    ms_add_v<DT, 1>(st, load_vec<DT, 1>(z, j), p.k2, vmax);
  __shared__ MS part[kThreads];
  part[tid] = st;
  __syncthreads();
  for (int i = kThreads / 2; i; i >>= 1) {
    if (tid < i) part[tid] = ms_merge(part[tid], part[tid + i], p.k2);
    __syncthreads();
  }
  st = part[0];
  const bool ok = ms_valid(st) && P == P;
  const float lse2 = st.m * p.k2 + log2f(st.s);
  float a = 0.f;
  if (ok)
    for (int k = tid; k < p.K; k += kThreads)
      if (t.id[k] >= 0 && t.p[k] > 0.f)
        a += t.p[k] *
             (t.log2p[k] - ((load_logit<DT>(z, t.id[k]) - st.m) * p.k2 -
                            log2f(st.s)));
  __syncthreads();
  scratch[tid] = a;
  __syncthreads();
  for (int i = kThreads / 2; i; i >>= 1) {
    if (tid < i) scratch[tid] += scratch[tid + i];
    __syncthreads();
  }
  if (tid == 0) {
    const float nan = __int_as_float(0x7fc00000);
    p.loss[row] = ok ? scratch[0] * kLn2 : nan;
    p.lse[row] = ok ? lse2 * kLn2 : nan;
    if (!ok) status_or(p.dev_status, SD_DEV_NONFINITE);
  }
}

template <int DT>
__device__ __forceinline__ void store_elt(void *row, int j, float x) {
  if constexpr (DT == 0) ((float *)row)[j] = x;
  else {
    uint32_t u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(u) : "f"(x));
    ((unsigned short *)row)[j] = (unsigned short)u;
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
distill_backward_kernel(const __grid_constant__ DistillParams p) {
  __shared__ Teacher t;
  __shared__ float scratch[kThreads];
  __shared__ float at[SD_MAX_DISTILL_K];
  const int row = blockIdx.x, tid = threadIdx.x;
  const char *z = (const char *)p.student +
                  (long long)row * p.row_stride * elt_bytes<DT>();
  char *g = (char *)p.grad + (long long)row * p.grad_stride * elt_bytes<DT>();
  const float w = p.grad_loss[row];
  if (w == 0.f) {
    for (int j = tid; j < p.V; j += kThreads) store_elt<DT>(g, j, 0.f);
    return;
  }
  const float P = load_teacher(p, row, t, scratch);
  const float lse = p.lse_in[row];
  const bool ok = P == P && fabsf(lse) < kInf;
  const float c = ok ? w * p.inv_T : __int_as_float(0x7fc00000);
  const float nl2 = -lse * (1.f / kLn2);
  if (!ok && tid == 0) status_or(p.dev_status, SD_DEV_NONFINITE);
  for (int k = tid; k < p.K; k += kThreads)
    at[k] = t.id[k] >= 0 ? load_logit<DT>(z, t.id[k]) : 0.f;
  __syncthreads();
  for (int j = tid; j < p.V; j += kThreads) {
    const float x = elt<DT, 1>(load_vec<DT, 1>(z, j), 0);
    store_elt<DT>(g, j, c * P * ex2(fmaf(x, p.k2, nl2)));
  }
  __syncthreads();
  // the entries' columns again, with the teacher's probabilities: the first
  // entry of an id writes for all that repeat it
  for (int k = tid; k < p.K; k += kThreads) {
    const int id = t.id[k];
    if (id < 0) continue;
    float sum = 0.f;
    bool first = true;
    for (int i = 0; i < p.K; ++i)
      if (t.id[i] == id) {
        first = first && i >= k;
        sum += t.p[i];
      }
    if (first)
      store_elt<DT>(g, id, c * (P * ex2(fmaf(at[k], p.k2, nl2)) - sum));
  }
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
  if (dt == SD_F32) distill_forward_kernel<0><<<N, kThreads, 0, s>>>(p);
  else distill_forward_kernel<1><<<N, kThreads, 0, s>>>(p);
  SDV_CUDA(cudaGetLastError());
  return SD_OK;
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
  if (dt == SD_F32) distill_backward_kernel<0><<<N, kThreads, 0, s>>>(p);
  else distill_backward_kernel<1><<<N, kThreads, 0, s>>>(p);
  SDV_CUDA(cudaGetLastError());
  return SD_OK;
}

extern "C" sd_status sd_distill_topk_step(
    const void *student, long long row_stride, sd_dtype dt,
    const float *teacher_logit, const int32_t *teacher_id,
    const float *teacher_lse, const float *grad_loss, int N, int V, int K,
    float T, float *loss, float *lse, void *grad, long long grad_stride,
    int32_t *dev_status, void *stream) {
  SDV_REQUIRE(N <= 0 || (grad_loss && grad), "null pointer");
  SDV_REQUIRE(grad_stride >= V, "grad_stride < V");
  sd_status st = sd_distill_topk(student, row_stride, dt, teacher_logit,
                                 teacher_id, teacher_lse, N, V, K, T, loss,
                                 lse, dev_status, stream);
  if (st != SD_OK) return st;
  return sd_distill_topk_backward(student, row_stride, dt, lse, teacher_logit,
                                  teacher_id, teacher_lse, grad_loss, N, V, K,
                                  T, grad, grad_stride, dev_status, stream);
}
