// Layer norm of rows of bf16 (see layer_norm.cuh).
#include "layer_norm.cuh"
SPGEMM_DEFINE_LAYER_NORM(bf16, __nv_bfloat16)
