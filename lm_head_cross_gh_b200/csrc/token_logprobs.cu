// Log-probabilities of given tokens with the row's entropy, log-sum-exp and
// most probable alternatives, and their gradient.
//
// For a row x of V logits, temperature T and c = log2(e) / T, with M = max x,
//     y_j = (x_j - M) c,   s = sum_j 2^y_j,   t = sum_j 2^y_j y_j,
//     log p_j = ln 2 (y_j - log2 s),   lse = M / T + ln s,
//     entropy = ln 2 (log2 s - t / s)
// (a term with 2^y = 0 adds nothing to t, so -inf logits are 0 log 0 = 0).
// The alternatives are the top_k logits by (value descending, index
// ascending); the temperature does not change their order.
#include "ce_device.cuh"
#include "common.cuh"
#include "profile.h"
#include "token_ops.h"

namespace gh {

namespace {

constexpr int kLpThreads = 512;

// Order-preserving key of a logit that is not NaN (-0 and +0 alike); 0 is
// below every logit's key.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// Key of (value descending, index ascending): larger is earlier.
__device__ __forceinline__ uint64_t rank_key(float x, int64_t j) {
  return (static_cast<uint64_t>(order_key(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(j));
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t k = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ int64_t key_index(uint64_t key) {
  return static_cast<int64_t>(0xffffffffu - static_cast<uint32_t>(key));
}

constexpr float kNaN = __builtin_nanf("");

__device__ __forceinline__ bool index_in(int64_t t, int64_t V) { return t >= 0 && t < V; }

template <int kThreads>
__device__ __forceinline__ uint64_t block_max_u64(uint64_t v, uint64_t* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u > v ? u : v;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  uint64_t r = 0;
  for (int w = 0; w < kThreads / 32; ++w) r = scratch[w] > r ? scratch[w] : r;
  return r;
}

// One CTA per row, three sweeps of the row (max, sums, one sweep per
// alternative).
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(LogprobArgs a) {
  constexpr int ES = Elem<T>::kBytes;
  __shared__ float red[3][kLpThreads / 32];
  __shared__ uint64_t red64[kLpThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = static_cast<int>(threadIdx.x);
  for (int64_t row = blockIdx.x; row < a.B; row += gridDim.x) {
    const int64_t ti = a.index[row];
    const bool ignored = ti == a.ignore_index, bad = !ignored && !index_in(ti, a.V);
    if (ignored || bad) {
      const float v = bad ? kNaN : 0.0f;
      if (tid == 0) {
        a.logprob[row] = a.entropy[row] = a.lse[row] = v;
        if (bad) record_status(GH_ERR_TARGET_RANGE);
      }
      for (int k = tid; k < a.top_k; k += kLpThreads) {
        a.top_logprob[row * a.top_k + k] = bad ? kNaN : kNegInf;
        a.top_index[row * a.top_k + k] = -1;
      }
      continue;
    }
    const uint8_t* src = static_cast<const uint8_t*>(a.logits) + row * a.ld * ES;
    float m = kNegInf;
    for (int64_t j = tid; j < a.V; j += kLpThreads) m = fmaxf(m, Elem<T>::load(src + j * ES));
    __syncthreads();
    m = block_max<kLpThreads>(m, red[0]);
    float s = 0.0f, t = 0.0f;
    for (int64_t j = tid; j < a.V; j += kLpThreads) {
      const float y = (Elem<T>::load(src + j * ES) - m) * a.c;
      const float e = ex2(y);
      s += e;
      if (e > 0.0f) t = fmaf(e, y, t);
    }
    s = block_sum<kLpThreads>(s, red[1]);
    t = block_sum<kLpThreads>(t, red[2]);
    const bool none = !(s > 0.0f && s < -kNegInf);
    const float l2s = log2f(s);
    if (tid == 0) {
      const float y = (Elem<T>::load(src + ti * ES) - m) * a.c;
      a.logprob[row] = none ? kNaN : kLn2 * (y - l2s);
      a.entropy[row] = none ? kNaN : kLn2 * (l2s - t / s);
      a.lse[row] = none ? kNaN : fmaf(m, a.c * kLn2, kLn2 * l2s);
    }
    uint64_t prev = ~0ull;
    for (int k = 0; k < a.top_k; ++k) {
      uint64_t best = 0;
      if (!none) {
        for (int64_t j = tid; j < a.V; j += kLpThreads) {
          const uint64_t key = rank_key(Elem<T>::load(src + j * ES), j);
          if (key < prev && key > best) best = key;
        }
        best = block_max_u64<kLpThreads>(best, red64);
      }
      if (tid == 0) {
        a.top_logprob[row * a.top_k + k] = none ? kNaN : kLn2 * ((key_value(best) - m) * a.c - l2s);
        a.top_index[row * a.top_k + k] = none ? -1 : key_index(best);
      }
      prev = best;
    }
  }
}

// Beyond this |lse| its fp32 rounding (2^-14 here) would show in exp(x / T -
// lse): rows whose logits all lie far from 0, such as fully masked ones.
constexpr float kFarLse = 1024.0f;

// Gradient of the row's log-probability and entropy:
//     grad_j = (1/T) (g_l [j == t] - p_j (g_l + g_H (log p_j + H))).
// With y = x c - lse log2(e) (the logits below X0 give p = 0 in fp32, and are
// read as X0 so that p (log p) stays 0 there),
//     grad_j = 2^y (a + b y) + [j == t] g_l / T,
//     a = -(g_l + g_H H) / T,  b = -g_H ln 2 / T.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_vjp_kernel(LogprobVjpArgs a) {
  constexpr int ES = Elem<T>::kBytes;
  __shared__ float red[2][kLpThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = static_cast<int>(threadIdx.x);
  for (int64_t row = blockIdx.x; row < a.B; row += gridDim.x) {
    const int64_t ti = a.index[row];
    const bool counts = ti != a.ignore_index && index_in(ti, a.V);
    const uint8_t* src = static_cast<const uint8_t*>(a.logits) + row * a.ld * ES;
    uint8_t* dst = static_cast<uint8_t*>(a.grad) + row * a.ld_grad * ES;
    if (!counts) {
      if (tid == 0 && ti != a.ignore_index) record_status(GH_ERR_TARGET_RANGE);
      for (int64_t j = tid; j < a.V; j += kLpThreads) Elem<T>::store(dst + j * ES, 0.0f);
      continue;
    }
    const float lse = a.lse[row];
    float sub = 0.0f, lse2 = lse * kLog2e;  // y = (x - sub) c - lse2
    if (fabsf(lse) > kFarLse) {
      // fp32 does not hold this lse finely enough: max and sum again
      float m = kNegInf, s = 0.0f;
      for (int64_t j = tid; j < a.V; j += kLpThreads) m = fmaxf(m, Elem<T>::load(src + j * ES));
      __syncthreads();
      m = block_max<kLpThreads>(m, red[0]);
      for (int64_t j = tid; j < a.V; j += kLpThreads) s += ex2((Elem<T>::load(src + j * ES) - m) * a.c);
      sub = m;
      lse2 = log2f(block_sum<kLpThreads>(s, red[1]));
    }
    const float gl = a.g_logprob[row], gH = a.g_entropy ? a.g_entropy[row] : 0.0f;
    const float ca = -(gl + gH * a.entropy[row]) * a.inv_t, cb = -gH * kLn2 * a.inv_t;
    for (int64_t j = tid; j < a.V; j += kLpThreads) {
      const float y = fmaf(Elem<T>::load(src + j * ES) - sub, a.c, -lse2);
      const float e = ex2(y);
      float g = e == 0.0f ? 0.0f : e * fmaf(cb, y, ca);
      if (j == ti) g += gl * a.inv_t;
      Elem<T>::store(dst + j * ES, g);
    }
  }
}

}  // namespace

gh_status_t logprobs_launch(const LogprobArgs& a, gh_dtype_t dtype, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(tmin<int64_t>(a.B, 148 * 4));
  ProfileScope prof(GH_KERNEL_LOGPROBS, stream);
  note_launch();
  const cudaError_t e = dtype == GH_F32
                            ? launch_pdl(logprobs_kernel<float>, dim3(grid), dim3(kLpThreads), 0, stream, 1, a)
                            : launch_pdl(logprobs_kernel<uint16_t>, dim3(grid), dim3(kLpThreads), 0, stream, 1, a);
  return e == cudaSuccess ? GH_OK : GH_ERR_CUDA;
}

gh_status_t logprobs_vjp_launch(const LogprobVjpArgs& a, gh_dtype_t dtype, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(tmin<int64_t>(a.B, 148 * 4));
  ProfileScope prof(GH_KERNEL_LOGPROBS_VJP, stream);
  note_launch();
  const cudaError_t e = dtype == GH_F32
                            ? launch_pdl(logprobs_vjp_kernel<float>, dim3(grid), dim3(kLpThreads), 0, stream, 1, a)
                            : launch_pdl(logprobs_vjp_kernel<uint16_t>, dim3(grid), dim3(kLpThreads), 0, stream, 1, a);
  return e == cudaSuccess ? GH_OK : GH_ERR_CUDA;
}

}  // namespace gh
