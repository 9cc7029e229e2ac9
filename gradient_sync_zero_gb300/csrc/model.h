// The operators at the ends of a training step: what the C ABI entries
// (model_api.cu) hand to the kernel launchers (kernels_embedding.cu,
// kernels_dropout.cu, kernels_token.cu).  Arguments are checked before.
#pragma once

#include <cstdint>

#include "internal.h"

namespace dps {

// A checked dp_rows: strides of extents of one are 0.
struct Mat {
  uint8_t* p = nullptr;
  int64_t rs = 0, ws = 0;   // rank and row stride, elements
  int32_t dtype = 0;        // DP_BF16 / DP_F32
};

inline int esize(int32_t dtype) { return dtype == DP_BF16 ? 2 : 4; }

// A checked dropout: words up to `last` are dropped, so that the whole range can be.
// inv is 1 / (1 - p), and 1 where nothing is dropped.
struct DropArgs {
  uint64_t seed = 0;
  const uint64_t* dev = nullptr;
  uint32_t offset = 0;
  uint32_t rank0 = 0;
  uint32_t last = 0;
  float inv = 1.0f;
  int32_t on = 0;
};

struct TokenArgs {
  const void* p = nullptr;
  int32_t wide = 0;   // int64 tokens
};

struct PolicyArgs {
  const float* old_logp = nullptr;
  const float* ref_logp = nullptr;
  const float* adv = nullptr;
  const float* weight = nullptr;
  float lo = 0, hi = 0, beta = 0;   // clamp bounds 1 - clip_low, 1 + clip_high
};

// CTAs per rank of the largest grid, at most (a grid takes 2^31 - 1).
int64_t dropout_ctas(int64_t T, int64_t D);
int64_t embedding_backward_ctas(int P, int64_t T, int64_t V, int64_t D);

// Each returns a cudaError_t value (0 = success); an empty problem launches nothing.
int launch_dropout(const Mat& x, const Mat& res, const Mat& out, int P, int64_t T, int64_t D,
                   const DropArgs& d, void* stream);
int launch_embedding_forward(const Mat& table, int64_t V, int64_t D, const TokenArgs& tok, int P,
                             int64_t T, float scale, const DropArgs& d, const Mat& out,
                             void* stream);
int64_t embedding_workspace_bytes(int P, int64_t T, int64_t V, int64_t D);
int launch_embedding_backward(const Mat& dout, const TokenArgs& tok, int P, int64_t T, float scale,
                              const DropArgs& d, const Mat& grad, int64_t V, int64_t D,
                              bool accumulate, uint8_t* ws, void* stream);
int launch_token_logprob(const Mat& logits, int P, int64_t T, int64_t V, const TokenArgs& tok,
                         float scale, float* logp, float* lse, void* stream);
int launch_token_logprob_backward(const Mat& logits, int P, int64_t T, int64_t V,
                                  const TokenArgs& tok, float scale, const float* lse,
                                  const float* dlogp, const Mat& dlogits, void* stream);
int launch_policy_loss(const Mat& logits, int P, int64_t T, int64_t V, const TokenArgs& tok,
                       float scale, const PolicyArgs& a, float* logp, float* stats,
                       const Mat& dlogits, void* stream);

}  // namespace dps
