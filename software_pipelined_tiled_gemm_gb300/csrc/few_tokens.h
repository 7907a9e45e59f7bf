// few_tokens.h -- the gated block's products for a few tokens (few_tokens.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "ops_internal.h"

namespace spgemm {

constexpr int kFewTokens = 32;

struct FewTokens {
  Matrix x;            // rows: the tokens; cols: K
  Matrix w;            // weights, rows of K
  int64_t rows;        // outputs of a token (gated: rows of either half of w)
  bool gated, bf16;
  bool weights_ready;  // the launch before this one is another of these, and does not write w
  uint16_t* out;
  int64_t ldo;
  float* pre;          // gated: kept projections (block_params.h), or nullptr
  int act;
};

// m tokens, `rows` rows of weights w (gated: of both halves).
bool few_tokens_fits(const gemm_ops* ops, int64_t m, int64_t rows, const Matrix& w);
cudaError_t few_tokens_init(const gemm_ops* ops);
cudaError_t few_tokens_launch(const gemm_ops* ops, const FewTokens& f, cudaStream_t stream);

}  // namespace spgemm
