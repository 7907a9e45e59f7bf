// Layer norm of rows of fp32 (see layer_norm.cuh).
#include "layer_norm.cuh"
SPGEMM_DEFINE_LAYER_NORM(f32, float)
