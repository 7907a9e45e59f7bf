// Instances of the block product "diag_cols" (see block_params.h).
#include "block_kernel.cuh"
SPGEMM_DEFINE_BLOCK(diag_cols, false, false, kEpiDiagCols)
