// Instances of the block product "tn" (see block_params.h).
#include "block_kernel.cuh"
SPGEMM_DEFINE_BLOCK(tn, true, true, kEpiLinear)
