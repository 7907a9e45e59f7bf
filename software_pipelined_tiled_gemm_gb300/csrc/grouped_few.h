// grouped_few.h -- the products grouped by expert for a few rows a group (grouped_few.cu).
#pragma once

#include <cuda_runtime.h>

#include "ops_internal.h"

namespace spgemm {

bool grouped_few_fits(const gemm_ops* ops, const gemm_grouped_args_t* args);  // forward pass
cudaError_t grouped_few_init(const gemm_ops* ops);
cudaError_t grouped_few_launch(const gemm_ops* ops, const gemm_grouped_args_t* args, cudaStream_t stream);

}  // namespace spgemm
