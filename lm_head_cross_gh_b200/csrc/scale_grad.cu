// A stored gradient times the scalar upstream gradient g (an fp32 device scalar):
//     out_j = round(grad_j g),
// the product in fp32 and rounded once.  (g rounded to bf16 beforehand would scale
// the whole gradient wrongly, by up to 2^-8.)
//
// Bound by HBM, one read and one write of every element: CTAs of four warps take
// parts of about 32 KiB of a row, or of a dense tensor as one row, as the
// log-probabilities' gradient does, four 16-byte loads of a thread in flight:
// [8192, 50257] bf16 in 249 us and fp32 in 496, both at the copy rate.  (torch's
// broadcast product with the same rounding takes 1481 us in bf16, and 852 with g
// rounded first.)
#include "profile.h"
#include "token_device.cuh"
#include "token_ops.h"

namespace gh {

namespace {

constexpr int kScaleThreads = 128;
constexpr int kScaleAhead = 4;
constexpr int64_t kScalePartBytes = 32 * 1024;

template <typename T>
__device__ __forceinline__ void scale_chunk(const uint4& q, float g, uint8_t* dst, bool congruent) {
  constexpr int ES = Elem<T>::kBytes, EPC = 16 / ES;
  float v[EPC];
  unpack16<T>(q, v);
#pragma unroll
  for (int j = 0; j < EPC; ++j) v[j] *= g;
  if (congruent) {
    __stcs(reinterpret_cast<uint4*>(dst), pack16<T>(v));
  } else {
#pragma unroll
    for (int j = 0; j < EPC; ++j) Elem<T>::store(dst + j * ES, v[j]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kScaleThreads) scale_grad_kernel(ScaleArgs a) {
  constexpr int ES = Elem<T>::kBytes;
  pdl_wait();
  pdl_trigger();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const int64_t row = blockIdx.x / a.parts;
  const int part = static_cast<int>(blockIdx.x - row * a.parts);
  const RowGeo r = row_geo<ES>(a.grad, row, a.ld, a.V);
  const int64_t from = tmin(r.c_hi, r.c_lo + part * a.part_chunks);
  const int64_t nc = (part == a.parts - 1 ? r.c_hi : tmin(r.c_hi, from + a.part_chunks)) - from;
  const uint4* const chunks = reinterpret_cast<const uint4*>(r.base) + from;
  uint8_t* const dst = static_cast<uint8_t*>(a.out) + row * a.ld_out * ES;
  uint8_t* const obase = dst - r.lead + 16 * from;  // this part's chunk c goes to obase + 16 c
  const bool congruent = ((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(r.src)) & 15) == 0;
  const float g = *a.g;
  for (int64_t c0 = tid; c0 < nc; c0 += kScaleAhead * kScaleThreads) {
    uint4 q[kScaleAhead];
#pragma unroll
    for (int i = 0; i < kScaleAhead; ++i)
      if (c0 + i * kScaleThreads < nc) q[i] = __ldcs(chunks + c0 + i * kScaleThreads);
#pragma unroll
    for (int i = 0; i < kScaleAhead; ++i)
      if (c0 + i * kScaleThreads < nc) scale_chunk<T>(q[i], g, obase + 16 * (c0 + i * kScaleThreads), congruent);
  }
  const int64_t e = part == 0 && tid < 32 ? edge_element(r, a.V, lane) : -1;
  if (e >= 0) Elem<T>::store(dst + e * ES, Elem<T>::load(r.src + e * ES) * g);
}

}  // namespace

gh_status_t scale_grad_launch(const ScaleArgs& args, gh_dtype_t dtype, cudaStream_t stream) {
  ScaleArgs a = args;
  if (a.ld == a.V && a.ld_out == a.V) {  // dense: one row
    a.V *= a.B;
    a.ld = a.ld_out = a.V;
    a.B = 1;
  }
  const int64_t bytes = a.V * (dtype == GH_F32 ? 4 : 2);
  // parts of about kScalePartBytes; smaller ones, down to 8 KiB, while they are fewer than are resident
  const int64_t resident = static_cast<int64_t>(token_sm_count()) * 8;
  int64_t parts = (bytes + kScalePartBytes - 1) / kScalePartBytes;
  while (a.B * parts < resident && bytes / (2 * parts) >= 8 * 1024) parts *= 2;
  if (parts > INT32_MAX || a.B > INT32_MAX / parts) return GH_ERR_UNSUPPORTED;
  a.parts = static_cast<int>(parts);
  a.part_chunks = (bytes / 16 + parts - 1) / parts;
  note_launch();
  const auto kern = dtype == GH_F32 ? scale_grad_kernel<float> : scale_grad_kernel<uint16_t>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(a.B * parts)), dim3(kScaleThreads), 0, stream, 1, a) == cudaSuccess
             ? GH_OK
             : GH_ERR_CUDA;
}

}  // namespace gh
