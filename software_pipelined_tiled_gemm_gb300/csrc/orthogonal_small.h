// orthogonal_small.h -- launch parameters and plan of the on-chip
// Newton-Schulz kernel (orthogonal_small.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernel_params.h"

struct gemm_ops;

namespace spgemm {

// 64-column panels of the iterate that a CTA can hold: beside the s x s
// matrix in shared memory, and their products in TMEM's 512 columns.
constexpr int small_newton_panels(int rows) { return rows == 1 ? 8 : 3; }

struct SmallNewton {
  Params base;         // status, timeout_ns, inject_fault
  const void* g;
  int64_t ld, g_batch;
  int type;            // gemm_in_t
  int tall;            // rows of G run along the long side
  int aligned;         // vectors of 8 elements of a row may be loaded whole
  int s, l;            // short and long side
  int batch, steps, cluster;
  float a, b, c, eps;
  uint16_t* out;       // batch x m x n
  // Per cluster, where it has more than one CTA: a sum of squares from each,
  // each one's fp32 partial of A, and A.
  double* norms;
  float* parts;
  uint16_t* gram;
};

struct SmallPlan {
  int rows = 0;        // blocks of 128 rows of the short side; 0: not for this kernel
  int cluster = 1, slots = 1;  // CTAs of a cluster; clusters
  size_t norm_bytes = 0, part_bytes = 0, gram_bytes = 0;
};

cudaError_t small_newton_init(gemm_ops* ops);  // once per handle
SmallPlan small_newton_plan(const gemm_ops* ops, int64_t m, int64_t n, int64_t batch);
cudaError_t small_newton_launch(const gemm_ops* ops, const SmallPlan& plan, SmallNewton& p,
                                cudaStream_t stream);

}  // namespace spgemm
