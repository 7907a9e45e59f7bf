// Instances of the block product "gated_bwd" (see block_params.h).
#include "block_kernel.cuh"
SPGEMM_DEFINE_BLOCK(gated_bwd, false, true, kEpiGatedBwd)
