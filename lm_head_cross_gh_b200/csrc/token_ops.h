// Internal interface of the token log-probability kernels (token_logprobs.cu),
// the top-logits distillation kernels (topk_distill.cu) and the stored gradients'
// scaling (scale_grad.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/gh.h"

namespace gh {

struct LogprobArgs {
  const void* logits;    // [B, V], row stride ld elements
  const int64_t* index;  // [B]
  int64_t B, V, ld;
  int64_t ignore_index;
  float temperature;
  float c;               // log2(e) / temperature
  int top_k;
  float* logprob;        // [B]
  float* entropy;        // [B]
  float* lse;            // [B], of the scaled logits
  float* top_logprob;    // [B, top_k]
  int64_t* top_index;    // [B, top_k]
  // set by logprobs_launch
  uint32_t low;          // lowest logit whose x c is finite (packed bf16, or fp32 bits)
  int slices;            // CTAs per row
  int64_t slice_chunks;  // 16-byte chunks per CTA of a row
  int seg_kind;          // what a segment is
};

struct LogprobVjpArgs {
  const void* logits;  // [B, V], row stride ld
  void* grad;          // [B, V], row stride ld_grad (may be logits with the same stride)
  const int64_t* index;
  int64_t B, V, ld, ld_grad;
  int64_t ignore_index;
  float c, c_lo;  // log2(e) / temperature as a sum of two floats
  float inv_t;    // 1 / temperature
  const float *lse, *entropy, *g_logprob, *g_entropy;  // [B] (g_entropy may be null)
  // set by logprobs_vjp_launch
  int parts;            // CTAs per row
  int64_t part_chunks;  // 16-byte chunks each
};

struct DistillArgs {
  const void* logits;
  void* grad;  // null: loss only
  int64_t B, V, ld, ld_grad;
  const int64_t* ids;   // [B, K] teacher entries
  const float* values;  // [B, K]
  int K;
  float temperature;
  float c;       // log2(e) / temperature
  int renormalize;
  int mean;
  const unsigned long long* n_valid;  // rows with an entry, of the whole batch (null: counted here)
  float* row_loss;                    // [B] (null: scratch)
  // set by distill_launch
  unsigned int* parts;        // counts of rows with an entry, to be added (null: counted by each CTA)
  int nparts;
  int8_t* flags;              // [B] 1: the row has an entry (null: looked up)
  int cluster;                // CTAs per row
  int64_t slice_chunks;       // 16-byte chunks per CTA of a row
};

struct ScaleArgs {
  const void* grad;  // [B, V], row stride ld
  void* out;         // [B, V], row stride ld_out (may be grad with the same stride)
  const float* g;    // device scalar
  int64_t B, V, ld, ld_out;
  // set by scale_grad_launch
  int parts;            // CTAs per row
  int64_t part_chunks;  // 16-byte chunks each
};

gh_status_t logprobs_launch(const LogprobArgs& a, gh_dtype_t dtype, cudaStream_t stream);
gh_status_t logprobs_vjp_launch(const LogprobVjpArgs& a, gh_dtype_t dtype, cudaStream_t stream);
// Counts the rows with an entry into *count (written, not added to).
gh_status_t distill_count_launch(const int64_t* ids, const float* values, int64_t B, int K, int64_t V,
                                 unsigned long long* count, cudaStream_t stream);
// Writes the scalar loss, the row losses and, with a.grad, the gradient.
gh_status_t distill_launch(const DistillArgs& a, gh_dtype_t dtype, float* loss, cudaStream_t stream);
gh_status_t scale_grad_launch(const ScaleArgs& a, gh_dtype_t dtype, cudaStream_t stream);

}  // namespace gh
