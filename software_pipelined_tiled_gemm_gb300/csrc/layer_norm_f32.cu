// Layer norm of rows of fp32 (see layer_norm.cuh).
#include "layer_norm.cuh"
SPGEMM_DEFINE_LAYER_NORM(f32, float)

namespace spgemm {
// The most that any type of rows takes (16384 columns and more may be read from memory again).
int layer_norm_backward_blocks(const gemm_ops* ops, int64_t rows, int64_t cols) {
  return std::max(cols > kLayerNormMaxCols / 2 ? long_grid(ops, rows) : 0, backward_grid<__half, true>(ops, rows, cols));
}
}  // namespace spgemm
