// Instances of the block product "diag_out" (see block_params.h).
#include "block_kernel.cuh"
SPGEMM_DEFINE_BLOCK(diag_out, false, false, kEpiDiagOut)
