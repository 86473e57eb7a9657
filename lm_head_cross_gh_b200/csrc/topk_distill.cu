// Distillation from a teacher's top logits: the row loss and the logits
// gradient from K stored entries (id, value) per row.
//
// With z = x / T, p = softmax(z) of the student's row x and q_k the teacher's
// probabilities (softmax of value / T over the row's entries, or exp(value)
// where the values are log-probabilities), Q = sum_k q_k:
//     row loss = T^2 sum_k q_k (log q_k - log p_{id_k})        (0 log 0 = 0)
//     grad_j   = scale T (Q p_j - sum_{k: id_k = j} q_k)
// (the T^2 keeps the gradient's size as T grows).  An entry whose id is -1 or
// whose value is -inf is none; a row without entries has no loss and a zero
// gradient.
#include "ce.h"
#include "ce_device.cuh"
#include "common.cuh"
#include "profile.h"
#include "token_ops.h"

namespace gh {

namespace {

constexpr int kDistillThreads = 512;

__device__ __forceinline__ bool distill_entry(int64_t id, float v, int64_t V) {
  return id >= 0 && id < V && !(v == kNegInf);
}

// Rows with at least one entry; one warp per row, one CTA, no atomics.
__global__ void __launch_bounds__(1024) distill_count_kernel(const int64_t* __restrict__ ids,
                                                             const float* __restrict__ values, int64_t B, int K,
                                                             int64_t V, unsigned long long* count) {
  __shared__ unsigned long long part[32];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned long long n = 0;
  for (int64_t row = warp; row < B; row += 32) {
    bool any = false;
    for (int k = lane; k < K; k += 32) {
      const int64_t id = ids[row * K + k];
      any |= distill_entry(id, values[row * K + k], V);
    }
    n += __any_sync(0xffffffffu, any) ? 1 : 0;
  }
  if (lane == 0) part[warp] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned long long tot = 0;
    for (int w = 0; w < 32; ++w) tot += part[w];
    *count = tot;
  }
}

template <typename T>
__global__ void __launch_bounds__(kDistillThreads) distill_kernel(DistillArgs a) {
  constexpr int ES = Elem<T>::kBytes;
  __shared__ float red[2][kDistillThreads / 32];
  __shared__ float q_s[GH_MAX_TOP_K], fix_s[GH_MAX_TOP_K], tot_s[2];
  __shared__ int64_t id_s[GH_MAX_TOP_K];
  pdl_wait();
  pdl_trigger();
  const int tid = static_cast<int>(threadIdx.x);
  const unsigned long long nv = *a.n_valid;
  const float scale = a.mean ? 1.0f / static_cast<float>(nv > 0 ? nv : 1ull) : 1.0f;
  for (int64_t row = blockIdx.x; row < a.B; row += gridDim.x) {
    const uint8_t* src = static_cast<const uint8_t*>(a.logits) + row * a.ld * ES;
    uint8_t* dst = static_cast<uint8_t*>(a.grad) + row * a.ld_grad * ES;
    __syncthreads();
    // the entries; thread 0 computes q (K is at most 128)
    if (tid < a.K) {
      const int64_t id = a.ids[row * a.K + tid];
      const float v = a.values[row * a.K + tid];
      if (id < -1 || id >= a.V) record_status(GH_ERR_TARGET_RANGE);
      id_s[tid] = distill_entry(id, v, a.V) ? id : -1;
      q_s[tid] = v;
    }
    __syncthreads();
    if (tid == 0) {
      float vm = kNegInf, sum = 0.0f;
      int n = 0;
      for (int k = 0; k < a.K; ++k)
        if (id_s[k] >= 0) {
          ++n;
          vm = fmaxf(vm, q_s[k]);
        }
      if (a.renormalize)
        for (int k = 0; k < a.K; ++k)
          if (id_s[k] >= 0) sum += expf((q_s[k] - vm) / a.temperature);
      float Q = 0.0f;
      for (int k = 0; k < a.K; ++k) {
        const float lq = a.renormalize ? (q_s[k] - vm) / a.temperature - logf(sum) : q_s[k];
        q_s[k] = lq;  // log q
        if (id_s[k] >= 0) Q += expf(lq);
      }
      tot_s[0] = n ? Q : -1.0f;
    }
    __syncthreads();
    const float Q = tot_s[0];
    if (Q == -1.0f) {
      if (tid == 0) a.row_loss[row] = 0.0f;
      if (a.grad)
        for (int64_t j = tid; j < a.V; j += kDistillThreads) Elem<T>::store(dst + j * ES, 0.0f);
      continue;
    }
    float m = kNegInf;
    for (int64_t j = tid; j < a.V; j += kDistillThreads) m = fmaxf(m, Elem<T>::load(src + j * ES));
    m = block_max<kDistillThreads>(m, red[0]);
    float s = 0.0f;
    for (int64_t j = tid; j < a.V; j += kDistillThreads) s += ex2((Elem<T>::load(src + j * ES) - m) * a.c);
    s = block_sum<kDistillThreads>(s, red[1]);
    const float l2s = log2f(s);
    const float ct = scale * a.temperature;
    if (tid < a.K && id_s[tid] >= 0) {
      // every entry with this id writes the same value: p Q less the q of all of them
      const float y = (Elem<T>::load(src + id_s[tid] * ES) - m) * a.c;
      float qs = 0.0f;
      for (int k = 0; k < a.K; ++k)
        if (id_s[k] == id_s[tid]) qs += expf(q_s[k]);
      fix_s[tid] = ct * (Q * ex2(y) / s - qs);
    }
    if (tid == 0) {
      float loss = 0.0f;
      for (int k = 0; k < a.K; ++k) {
        if (id_s[k] < 0) continue;
        const float q = expf(q_s[k]);
        const float y = (Elem<T>::load(src + id_s[k] * ES) - m) * a.c;
        if (!(q == 0.0f)) loss += q * (q_s[k] - kLn2 * (y - l2s));
      }
      a.row_loss[row] = a.temperature * a.temperature * loss;
    }
    if (!a.grad) continue;
    __syncthreads();  // in place: the entries' logits are read before they are overwritten
    const float coef = ct * Q / s;
    for (int64_t j = tid; j < a.V; j += kDistillThreads)
      Elem<T>::store(dst + j * ES, coef * ex2((Elem<T>::load(src + j * ES) - m) * a.c));
    __syncthreads();
    if (tid < a.K && id_s[tid] >= 0) Elem<T>::store(dst + id_s[tid] * ES, fix_s[tid]);
  }
}

}  // namespace

gh_status_t distill_count_launch(const int64_t* ids, const float* values, int64_t B, int K, int64_t V,
                                 unsigned long long* count, cudaStream_t stream) {
  note_launch();
  return launch_pdl(distill_count_kernel, dim3(1), dim3(1024), 0, stream, 1, ids, values, B, K, V, count) ==
                 cudaSuccess
             ? GH_OK
             : GH_ERR_CUDA;
}

gh_status_t distill_launch(const DistillArgs& a, gh_dtype_t dtype, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(tmin<int64_t>(a.B, 148 * 4));
  ProfileScope prof(GH_KERNEL_DISTILL, stream);
  note_launch();
  const cudaError_t e =
      dtype == GH_F32 ? launch_pdl(distill_kernel<float>, dim3(grid), dim3(kDistillThreads), 0, stream, 1, a)
                      : launch_pdl(distill_kernel<uint16_t>, dim3(grid), dim3(kDistillThreads), 0, stream, 1, a);
  return e == cudaSuccess ? GH_OK : GH_ERR_CUDA;
}

}  // namespace gh
