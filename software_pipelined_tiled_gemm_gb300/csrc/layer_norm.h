// layer_norm.h -- what the layer norm's argument checks (layer_norm.cu) and its
// kernels (layer_norm.cuh, one file for each type of rows) share.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "ops_internal.h"

namespace spgemm {

constexpr int kLayerNormMaxCols = 32768;     // above it rows are read again from memory
constexpr size_t kLayerNormStatic = 1024;    // shared memory, at least what the kernels declare

struct LayerNormJob {
  const void* x;
  int64_t ldx;
  const void* dy;
  int64_t lddy;
  const void* weight;
  const void* bias;
  void* out;            // y or dx, dense
  float* stats;         // 3 x rows
  float* partial;       // backward: blocks x 2 x cols, or nullptr
  int64_t rows;
  int cols;
  float inv;            // 1 / cols
  float eps;
  int ahead;            // rows of a group on their way or in work
  int weight_bytes;     // of the weights in shared memory
};

#define SPGEMM_DECLARE_LAYER_NORM(NAME)                                                                      \
  cudaError_t layer_norm_set_smem_##NAME(size_t smem);                                                       \
  cudaError_t layer_norm_forward_##NAME(const gemm_ops* ops, const LayerNormJob& p, bool vec, bool wide,     \
                                        cudaStream_t stream);                                                \
  cudaError_t layer_norm_backward_##NAME(const gemm_ops* ops, const LayerNormJob& p, bool vec, bool wide,    \
                                         void* dweight, void* dbias, cudaStream_t stream);
SPGEMM_DECLARE_LAYER_NORM(f16)
SPGEMM_DECLARE_LAYER_NORM(bf16)
SPGEMM_DECLARE_LAYER_NORM(f32)
#undef SPGEMM_DECLARE_LAYER_NORM

// Blocks of a backward pass at most, each of which leaves a partial.
int layer_norm_backward_blocks(const gemm_ops* ops, int64_t rows, int64_t cols);

}  // namespace spgemm
