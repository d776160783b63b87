// layer_ops.cuh — internal interface of the rest of a layer of grouped heads: products
// with a weight (linear.cu), the heads' norm and rotation (head_rope.cu) and what a
// sampler reads off the logits (token_scores.cu).  include/dllm.h is the public ABI.
#pragma once

#include "kernels.cuh"

namespace dllm {

// ---- products with a weight
constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3;  // DLLM_ACT_*
struct LinearArgs {
  const void* x;         // bf16 [rows][K] at x_stride
  int64_t x_stride;
  const void* gain;      // bf16 [K], nullable
  const void* w;         // bf16 [wide][K]
  const void* bias;      // bf16 [wide], nullable
  const void* residual;  // bf16 [rows][N] at r_stride, nullable; may be y
  int64_t r_stride;
  void* y;               // bf16 [rows][N] at y_stride
  int64_t y_stride;
  void* xhat;            // workspace: bf16 [rows][K], where there is a gain
  int32_t* err;
  int32_t rows, k, n, wide;  // wide: rows of w (N, or 2 N gate and up units side by side)
  int32_t act;
  bool gated;
  float rms_eps;
};
cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream);

// ---- the heads' norm and rotation
struct HeadRows {
  const void* in;
  int64_t in_row, in_head;
  void* out;
  int64_t out_row, out_head;
  const void* gain;  // nullable
  int32_t n_heads;
};
struct HeadRopeArgs {
  HeadRows q, k;  // k.n_heads == 0: none
  const int32_t* row_pos;
  const float* table;
  int32_t* err;
  int32_t rows, head_dim, max_pos, rotary_dim;
  bool neighbours;
  float eps;
};
cudaError_t launch_head_rope(const HeadRopeArgs& a, int num_sms, cudaStream_t stream);

// ---- token scores
constexpr int kMaxTop = 32;
struct ScoreArgs {
  const void* logits;
  int64_t stride;
  const int32_t* tokens;  // nullable, as logp, lse, entropy
  float* logp;
  float* lse;
  float* entropy;
  int32_t* top_ids;
  float* top_logp;
  int32_t* err;
  int32_t rows, vocab, top;
  float scale;
  bool fp32;
};
cudaError_t launch_token_scores(const ScoreArgs& a, int num_sms, cudaStream_t stream);

}  // namespace dllm
