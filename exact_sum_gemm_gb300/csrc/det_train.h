// Internal launch interface of the training operators beside the linear
// layers: layer norm, attention and token log probabilities.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "det_kernels.h"

namespace det {

// A row-wise operand: row r starts r * ld elements after the pointer.
struct LayerNormArgs {
  const void* x;
  int64_t ldx;
  const void* weight;      // [width] or null (1)
  const void* bias;        // [width] or null (0)
  void* y;
  int64_t ldy;
  float* mean;             // [rows]
  float* rstd;             // [rows]
  int64_t rows, width;
  float eps;
  int bf16, weight_bf16;
};

struct LayerNormGradArgs {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const float* mean;
  const float* rstd;
  const void* weight;      // or null (1)
  void* dx;                // or null: not wanted
  int64_t lddx;
  void* dweight;           // [width] in the weight's type, or null
  void* dbias;             // likewise
  float* partial;          // set by the launcher
  int64_t rows, width;
  int bf16, weight_bf16;
};

cudaError_t launch_layer_norm_forward(const LayerNormArgs& a, cudaStream_t stream);
cudaError_t launch_layer_norm_backward(const LayerNormGradArgs& a, cudaStream_t stream);

// Most alternatives of one row.
constexpr int kMaxTop = 32;

struct LogprobsArgs {
  const void* logits;
  int64_t ld;
  const int64_t* tokens;   // [rows]; negative: no token
  int64_t rows, vocab;
  int top;
  float* logprobs;         // [rows]
  float* entropy;          // [rows]
  float* stats;            // [rows][2]: maximum, sum of exp(x - maximum)
  float* top_logprobs;     // [rows][top]
  int64_t* top_tokens;     // [rows][top]
  int bf16;
};

struct LogprobsGradArgs {
  const float* dlogprobs;  // [rows] or null (0)
  const float* dentropy;   // [rows] or null (0)
  const void* logits;
  int64_t ld;
  const int64_t* tokens;
  const float* entropy;
  const float* stats;
  void* dlogits;
  int64_t ldd;
  int64_t rows, vocab;
  int bf16;
};

cudaError_t launch_logprobs_forward(const LogprobsArgs& a, cudaStream_t stream);
cudaError_t launch_logprobs_backward(const LogprobsGradArgs& a, cudaStream_t stream);

// A [batch, length, heads, dim] tensor with unit stride over dim.
struct Heads {
  void* p;
  int64_t sb, sl, sh;      // strides in elements
};

struct AttentionArgs {
  Heads q, k, v, o;
  Heads dout, dq, dk, dv;      // backward; dq.p / dk.p null: not wanted
  float* lse;              // [batch, hq, lq]: written by forward, read by backward
  // Scratch of backward, [batch, hq, stat_stride] with stat_stride = lq rounded
  // up to 128, as the kernels copy whole steps of up to 128 rows: sum_d do o (0
  // past lq), and lse log2(e) (+inf for a query without a key and past lq: its
  // probabilities are then 0).
  float* delta;
  float* lse2;
  int64_t stat_stride;
  const int32_t* k_lengths;  // [batch] or null
  int32_t batch, lq, lk, hq, hkv, dim;
  float scale;
  int causal;
  int bf16;
  // bf16: set by the tensor-core kernels per owned tile ([batch][tiles][heads]
  // of flag_rows rows) where a tile that the causal diagonal crosses held a
  // non-finite value.  f32: set by the split per block where any value was one;
  // flag_rows is then 0 and every tile counts as flagged.
  int* flags;
  int flag_rows;
  int64_t dq_flags;        // backward: where the query tiles' flags start
  // f32 on the tensor cores: three bf16 planes of q, k, v and dO,
  // [plane][batch][heads][length][64] each (head dimensions above 64: 128).
  void* planes[4];
  int halves;              // tensor-core forward: 128-row halves of a block, 1 or 2
};

constexpr int kMaxHeadDim = 128;
// The largest magnitude that is split: its first plane does not round to inf.
constexpr float kMostSplit = 3.38e38f;

// On the tensor cores (f32: after the split); the flagged tiles' affected rows
// are left to the CUDA-core kernels.  A forward block owns attention_halves x
// 128 rows (set in the arguments), a backward block kTcBackwardRows.
constexpr int kTcBackwardRows = 128;
int attention_halves(const AttentionArgs& a);
int64_t attention_split_blocks(const AttentionArgs& a);    // flags per tensor
cudaError_t launch_attention_split(const AttentionArgs& a, int tensors, cudaStream_t stream);
cudaError_t launch_attention_wide_forward(const AttentionArgs& a, cudaStream_t stream);
cudaError_t launch_attention_wide_backward(const AttentionArgs& a, cudaStream_t stream);
cudaError_t launch_attention_tc_forward(const AttentionArgs& a, cudaStream_t stream);
// (dq.p / dk.p null: not wanted)
cudaError_t launch_attention_tc_backward(const AttentionArgs& a, cudaStream_t stream);

cudaError_t launch_attention_forward(const AttentionArgs& a, cudaStream_t stream);
cudaError_t launch_attention_backward(const AttentionArgs& a, cudaStream_t stream);

}  // namespace det
