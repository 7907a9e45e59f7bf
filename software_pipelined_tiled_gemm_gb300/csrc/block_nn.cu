// Instances of the block product "nn" (see block_params.h).
#include "block_kernel.cuh"
SPGEMM_DEFINE_BLOCK(nn, false, true, kEpiLinear)
