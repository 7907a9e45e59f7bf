// Instances of the block product "gated" (see block_params.h).
#include "block_kernel.cuh"
SPGEMM_DEFINE_BLOCK(gated, false, false, kEpiGated)
