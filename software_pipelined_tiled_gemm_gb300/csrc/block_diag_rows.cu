// Instances of the block product "diag_rows" (see block_params.h).
#include "block_kernel.cuh"
SPGEMM_DEFINE_BLOCK(diag_rows, false, true, kEpiDiagRows)
