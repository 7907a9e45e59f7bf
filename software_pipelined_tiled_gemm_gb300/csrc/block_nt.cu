// Instances of the block product "nt" (see block_params.h).
#include "block_kernel.cuh"
SPGEMM_DEFINE_BLOCK(nt, false, false, kEpiLinear)
