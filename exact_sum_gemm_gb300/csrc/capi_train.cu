// C ABI of the training operators (declared in include/det_gemm.h): argument
// checks on the host, then the launch on the caller's stream.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "det_gemm.h"
#include "det_train.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
det_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DET_OK : DET_ERR_CUDA; }
bool dtype_ok(det_dtype t) { return t == DET_F32 || t == DET_BF16; }
uintptr_t size_of(det_dtype t) { return t == DET_F32 ? 4 : 2; }

// One block per row, and byte offsets that stay within 63 bits: no axis reaches
// over more than 2^58 elements.
constexpr int64_t kMaxRows = 0x7FFFFFFFll;
constexpr int64_t kMaxWidth = 0x7FFFFFFFll - 0xFFFF;
constexpr int64_t kMaxStride = int64_t(1) << 40;
bool reaches_too_far(int64_t n, int64_t stride) { return n > 1 && stride > (int64_t(1) << 58) / n; }

det_status check_rows(det_dtype dtype, int64_t rows, int64_t width) {
  if (!dtype_ok(dtype)) return DET_ERR_DTYPE;
  if (rows < 0 || width < 0 || rows > kMaxRows || width > kMaxWidth) return DET_ERR_SHAPE;
  return DET_OK;
}

// A row-wise operand that is read or written.
det_status check_operand(const void* p, int64_t rows, int64_t ld, int64_t width, uintptr_t size) {
  if (p == nullptr || ld < width || ld > kMaxStride || reaches_too_far(rows, ld)) return DET_ERR_INVALID_ARG;
  return aligned(p, size) ? DET_OK : DET_ERR_ALIGNMENT;
}
det_status check_vector(const void* p, uintptr_t size) {
  if (p == nullptr) return DET_ERR_INVALID_ARG;
  return aligned(p, size) ? DET_OK : DET_ERR_ALIGNMENT;
}

#define DET_CHECK(expr)                    \
  do {                                     \
    const det_status status_ = (expr);     \
    if (status_ != DET_OK) return status_; \
  } while (0)

det_status check_norm_types(det_dtype dtype, det_dtype weight_dtype) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return DET_ERR_DTYPE;
  return weight_dtype == DET_BF16 && dtype != DET_BF16 ? DET_ERR_DTYPE : DET_OK;
}

det_status check_shape(det_dtype dtype, const det_attention_shape* s) {
  if (!dtype_ok(dtype)) return DET_ERR_DTYPE;
  if (s == nullptr) return DET_ERR_INVALID_ARG;
  constexpr int64_t kMax = int64_t(1) << 30;
  if (s->batch < 0 || s->lq < 0 || s->lk < 0 || s->hq < 1 || s->hkv < 1 || s->dim < 1) return DET_ERR_SHAPE;
  if (s->batch > kMax || s->lq > kMax || s->lk > kMax || s->hq > 65535 || s->hkv > s->hq) return DET_ERR_SHAPE;
  if (s->hq % s->hkv != 0 || s->dim > DET_MAX_HEAD_DIM) return DET_ERR_SHAPE;
  // blocks of a launch, for each head of each entry: one per 64 rows, or per 16 (the f32 split), at most
  const int64_t tiles = (s->lq > s->lk ? s->lq : s->lk) / 8 + 1;
  if (s->batch > 0 && tiles > kMaxRows / (s->batch * s->hq)) return DET_ERR_SHAPE;
  if ((s->causal != 0 && s->causal != 1) || !isfinite(s->scale)) return DET_ERR_INVALID_ARG;
  if (s->k_lengths != nullptr && !aligned(s->k_lengths, 4)) return DET_ERR_ALIGNMENT;
  return DET_OK;
}

// Of a shape that check_shape passes.  Backward has a block per 64 queries (dq)
// and per 64 keys (dk and dv) in one launch, and, bf16, one per 16 queries, of
// which a head has whole 128s.
det_status check_backward_blocks(det_dtype dtype, const det_attention_shape* s, bool dq, bool dkv) {
  int64_t tiles = 0;
  if (dq) tiles += s->batch * s->hq * ((s->lq + 63) / 64);
  if (dkv) tiles += s->batch * s->hkv * ((s->lk + 63) / 64);
  const int64_t statistics = dtype == DET_BF16 ? s->batch * s->hq * ((s->lq + 127) / 128 * 8) : 0;
  return tiles > kMaxRows || statistics > kMaxRows ? DET_ERR_SHAPE : DET_OK;
}

// A tensor of `length` rows of `heads` heads; an empty one is never touched.
det_status check_heads(const det_heads& h, det_dtype dtype, int64_t batch, int64_t length, int64_t heads) {
  if (batch == 0 || length == 0) return DET_OK;
  if (h.ptr == nullptr) return DET_ERR_INVALID_ARG;
  for (int64_t s : {h.stride_batch, h.stride_length, h.stride_head})
    if (s < 0 || s > kMaxStride) return DET_ERR_INVALID_ARG;
  if (reaches_too_far(batch, h.stride_batch) || reaches_too_far(length, h.stride_length) ||
      reaches_too_far(heads, h.stride_head))
    return DET_ERR_INVALID_ARG;
  return aligned(h.ptr, size_of(dtype)) ? DET_OK : DET_ERR_ALIGNMENT;
}

det::Heads heads(const det_heads& h) { return {h.ptr, h.stride_batch, h.stride_length, h.stride_head}; }

det::AttentionArgs attention_args(det_dtype dtype, const det_attention_shape* s, const det_heads& q,
                                  const det_heads& k, const det_heads& v, const det_heads& o) {
  det::AttentionArgs a{};
  a.q = heads(q);
  a.k = heads(k);
  a.v = heads(v);
  a.o = heads(o);
  a.k_lengths = s->k_lengths;
  a.batch = static_cast<int32_t>(s->batch);
  a.lq = static_cast<int32_t>(s->lq);
  a.lk = static_cast<int32_t>(s->lk);
  a.hq = static_cast<int32_t>(s->hq);
  a.hkv = static_cast<int32_t>(s->hkv);
  a.dim = static_cast<int32_t>(s->dim);
  a.scale = s->scale;
  a.causal = s->causal;
  a.bf16 = dtype == DET_BF16;
  return a;
}

}  // namespace

extern "C" {

det_status det_layer_norm_forward(det_dtype dtype, det_dtype weight_dtype, int64_t rows,
                                  int64_t width, const void* x, int64_t ldx, const void* weight,
                                  const void* bias, float eps, void* y, int64_t ldy, float* mean,
                                  float* rstd, void* stream) {
  DET_CHECK(check_norm_types(dtype, weight_dtype));
  DET_CHECK(check_rows(dtype, rows, width));
  if (!(eps >= 0.f) || !isfinite(eps)) return DET_ERR_INVALID_ARG;
  if (rows == 0 || width == 0) return DET_OK;
  DET_CHECK(check_operand(x, rows, ldx, width, size_of(dtype)));
  DET_CHECK(check_operand(y, rows, ldy, width, size_of(dtype)));
  DET_CHECK(check_vector(mean, 4));
  DET_CHECK(check_vector(rstd, 4));
  if (!aligned(weight, size_of(weight_dtype)) || !aligned(bias, size_of(weight_dtype))) return DET_ERR_ALIGNMENT;
  det::LayerNormArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.width = width;
  a.eps = eps;
  a.bf16 = dtype == DET_BF16;
  a.weight_bf16 = weight_dtype == DET_BF16;
  return from_cuda(det::launch_layer_norm_forward(a, static_cast<cudaStream_t>(stream)));
}

det_status det_layer_norm_backward(det_dtype dtype, det_dtype weight_dtype, int64_t rows,
                                   int64_t width, const void* dy, int64_t lddy, const void* x,
                                   int64_t ldx, const float* mean, const float* rstd,
                                   const void* weight, void* dx, int64_t lddx, void* dweight,
                                   void* dbias, void* stream) {
  DET_CHECK(check_norm_types(dtype, weight_dtype));
  DET_CHECK(check_rows(dtype, rows, width));
  for (const void* p : {weight, static_cast<const void*>(dweight), static_cast<const void*>(dbias)})
    if (!aligned(p, size_of(weight_dtype))) return DET_ERR_ALIGNMENT;
  if (width == 0) return DET_OK;
  if (rows > 0) {
    DET_CHECK(check_operand(dy, rows, lddy, width, size_of(dtype)));
    DET_CHECK(check_operand(x, rows, ldx, width, size_of(dtype)));
    if (dx != nullptr) DET_CHECK(check_operand(dx, rows, lddx, width, size_of(dtype)));
    DET_CHECK(check_vector(mean, 4));
    DET_CHECK(check_vector(rstd, 4));
  }
  det::LayerNormGradArgs a{};
  a.dy = dy;
  a.lddy = lddy;
  a.x = x;
  a.ldx = ldx;
  a.mean = mean;
  a.rstd = rstd;
  a.weight = weight;
  a.dx = dx;
  a.lddx = lddx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.rows = rows;
  a.width = width;
  a.bf16 = dtype == DET_BF16;
  a.weight_bf16 = weight_dtype == DET_BF16;
  return from_cuda(det::launch_layer_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

det_status det_attention_forward(det_dtype dtype, const det_attention_shape* shape, det_heads q,
                                 det_heads k, det_heads v, det_heads o, float* lse, void* stream) {
  DET_CHECK(check_shape(dtype, shape));
  const auto check_queries = [&](const det_heads& h) { return check_heads(h, dtype, shape->batch, shape->lq, shape->hq); };
  const auto check_keys = [&](const det_heads& h) { return check_heads(h, dtype, shape->batch, shape->lk, shape->hkv); };
  DET_CHECK(check_queries(q));
  DET_CHECK(check_keys(k));
  DET_CHECK(check_keys(v));
  DET_CHECK(check_queries(o));
  if (shape->batch == 0 || shape->lq == 0) return DET_OK;
  DET_CHECK(check_vector(lse, 4));
  det::AttentionArgs a = attention_args(dtype, shape, q, k, v, o);
  a.lse = lse;
  return from_cuda(det::launch_attention_forward(a, static_cast<cudaStream_t>(stream)));
}

det_status det_attention_backward(det_dtype dtype, const det_attention_shape* shape, det_heads dout,
                                  det_heads q, det_heads k, det_heads v, det_heads o,
                                  const float* lse, det_heads dq, det_heads dk, det_heads dv,
                                  void* stream) {
  DET_CHECK(check_shape(dtype, shape));
  DET_CHECK(check_backward_blocks(dtype, shape, dq.ptr != nullptr, dk.ptr != nullptr));
  const auto check_queries = [&](const det_heads& h) { return check_heads(h, dtype, shape->batch, shape->lq, shape->hq); };
  const auto check_keys = [&](const det_heads& h) { return check_heads(h, dtype, shape->batch, shape->lk, shape->hkv); };
  DET_CHECK(check_queries(dout));
  DET_CHECK(check_queries(q));
  DET_CHECK(check_keys(k));
  DET_CHECK(check_keys(v));
  DET_CHECK(check_queries(o));
  if (shape->batch > 0 && shape->lq > 0) DET_CHECK(check_vector(lse, 4));
  if (dq.ptr != nullptr) DET_CHECK(check_queries(dq));
  if ((dk.ptr == nullptr) != (dv.ptr == nullptr)) return DET_ERR_INVALID_ARG;
  if (dk.ptr != nullptr) {
    DET_CHECK(check_keys(dk));
    DET_CHECK(check_keys(dv));
  }
  det::AttentionArgs a = attention_args(dtype, shape, q, k, v, o);
  a.dout = heads(dout);
  a.dq = heads(dq);
  a.dk = heads(dk);
  a.dv = heads(dv);
  a.lse = const_cast<float*>(lse);
  return from_cuda(det::launch_attention_backward(a, static_cast<cudaStream_t>(stream)));
}

det_status det_token_logprobs_forward(det_dtype dtype, int64_t rows, int64_t vocab,
                                      const void* logits, int64_t ld, const int64_t* tokens,
                                      int top, float* logprobs, float* entropy, float* stats,
                                      float* top_logprobs, int64_t* top_tokens, void* stream) {
  DET_CHECK(check_rows(dtype, rows, vocab));
  if (vocab < 1 || top < 0 || top > DET_MAX_TOP || top > vocab) return DET_ERR_SHAPE;
  if (rows == 0) return DET_OK;
  DET_CHECK(check_operand(logits, rows, ld, vocab, size_of(dtype)));
  DET_CHECK(check_vector(tokens, 8));
  DET_CHECK(check_vector(logprobs, 4));
  DET_CHECK(check_vector(entropy, 4));
  DET_CHECK(check_vector(stats, 4));
  if (top > 0) {
    DET_CHECK(check_vector(top_logprobs, 4));
    DET_CHECK(check_vector(top_tokens, 8));
  }
  det::LogprobsArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.tokens = tokens;
  a.rows = rows;
  a.vocab = vocab;
  a.top = top;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.stats = stats;
  a.top_logprobs = top_logprobs;
  a.top_tokens = top_tokens;
  a.bf16 = dtype == DET_BF16;
  return from_cuda(det::launch_logprobs_forward(a, static_cast<cudaStream_t>(stream)));
}

det_status det_token_logprobs_backward(det_dtype dtype, int64_t rows, int64_t vocab,
                                       const float* dlogprobs, const float* dentropy,
                                       const void* logits, int64_t ld, const int64_t* tokens,
                                       const float* entropy, const float* stats, void* dlogits,
                                       int64_t ldd, void* stream) {
  DET_CHECK(check_rows(dtype, rows, vocab));
  if (vocab < 1) return DET_ERR_SHAPE;
  if (rows == 0) return DET_OK;
  DET_CHECK(check_operand(logits, rows, ld, vocab, size_of(dtype)));
  DET_CHECK(check_operand(dlogits, rows, ldd, vocab, size_of(dtype)));
  DET_CHECK(check_vector(tokens, 8));
  DET_CHECK(check_vector(entropy, 4));
  DET_CHECK(check_vector(stats, 4));
  if (!aligned(dlogprobs, 4) || !aligned(dentropy, 4)) return DET_ERR_ALIGNMENT;
  det::LogprobsGradArgs a{};
  a.dlogprobs = dlogprobs;
  a.dentropy = dentropy;
  a.logits = logits;
  a.ld = ld;
  a.tokens = tokens;
  a.entropy = entropy;
  a.stats = stats;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.rows = rows;
  a.vocab = vocab;
  a.bf16 = dtype == DET_BF16;
  return from_cuda(det::launch_logprobs_backward(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
