// Layer norm of rows of fp16 (see layer_norm.cuh).
#include "layer_norm.cuh"
SPGEMM_DEFINE_LAYER_NORM(f16, __half)
