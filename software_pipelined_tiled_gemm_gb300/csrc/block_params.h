// block_params.h -- launch parameters of the block products (block_kernel.cuh)
// shared by the host planner (ops_api.cu) and the device kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernel_params.h"

namespace spgemm {

// What the epilogue does with a tile's fp32 accumulator.
constexpr int kEpiLinear = 0;     // C = alpha acc, optionally mirrored across the diagonal
constexpr int kEpiGated = 1;      // H = act(gate) * up, the tile holding both; keeps both in fp32
constexpr int kEpiGatedBwd = 2;   // acc = dH: writes dGate and dUp from the kept gate and up

// C = alpha acc + beta D, with a diagonal in fp32 beside a 16-bit matrix: C's is
// moved there and 0 left in its place; or alpha diag[row] D or alpha
// diag[column] D is added.
constexpr int kEpiDiagOut = 3, kEpiDiagRows = 4, kEpiDiagCols = 5;

// Activation of the gated block (gemm_act_t).
constexpr int kActSilu = 0, kActGelu = 1, kActRelu = 2;

// One 16-bit (or, for a linear product, the same in another type) output of
// a product: a batch of row-major matrices.
struct BlockOut {
  void* ptr;
  int64_t ld;        // row pitch, elements
  int64_t batch;     // matrix pitch, elements
  int tma;           // 1: base and pitch 16-byte aligned, bulk tensor stores
};

// Params (kernel_params.h) carries the extents, tiling, ring and status
// fields; of its scheduling fields the block products use raster_group,
// dp_tiles, sk_tiles, sk_ws, sk_flags, a_box_rows, b_stream and
// l2_prefetch_first.
struct BlockParams : Params {
  int tiles_per;       // tiles of one matrix of the batch
  int batch;
  int walkers;         // CTAs, or CTA pairs
  int epi;             // epilogue warps per TMEM lane quarter, 1 or 2
  int splits;          // > 1: each tile's K is split over a cluster of this many single CTAs
  int zero_flags;      // > 0: this launch needs no flags and zeroes so many for the next ones
  int symmetric;       // 1: only tiles on and above the diagonal run; each off-diagonal one is
                       // also written transposed (square output)
  int out_bf16;        // type of the 16-bit output(s)
  int act;
  int gate_rows;       // gated: rows of the gate half of w_in (the up half follows)
  float alpha, beta;
  float* diag;         // kEpiDiagOut, kEpiDiagRows, kEpiDiagCols
  int64_t diag_batch;  // of one matrix, elements
  BlockOut out0, out1;  // C or H or dGate; dUp
  // Gated: gate and up in fp32, [half][row block of 32][column][row in block],
  // so that an epilogue warp (lane = row) moves one 128-byte line a column;
  // nullptr: not kept.
  float* pre;
  int64_t pre_half;    // elements of one half
};

struct BlockMaps {
  CUtensorMap a, b, c0, c1, d;
};

// Tile shapes: CTA pairs computing 256 x 256 with two 64-wide K slices per
// ring slot, or single CTAs computing 128 x 128 with one.
constexpr int kPairBN = 256, kSoloBN = 128;
__host__ __device__ constexpr int block_bn(int cg) { return cg == 2 ? kPairBN : kSoloBN; }
__host__ __device__ constexpr int block_sub(int cg) { return cg == 2 ? 2 : 1; }

// fp32 partial of one CTA's tile in the stream-K workspace.
__host__ __device__ constexpr size_t block_partial_bytes(int cg) {
  return static_cast<size_t>(kBM) * block_bn(cg) * 4;
}

// A split tile's fp32 partial, staged in the CTA's idle ring.
constexpr uint32_t kSplitBytes = kBM * kSoloBN * 4u;
constexpr int kMaxSplits = 4;

// Launchers, one per operand layout (block_*.cu): A K-major or MN-major
// ("t": stored K x M), B likewise ("n": stored K x N).
#define SPGEMM_DECLARE_BLOCK(NAME)                                                          \
  cudaError_t block_set_smem_##NAME(size_t smem);                                           \
  cudaError_t block_launch_##NAME(const BlockMaps& m, const BlockParams& p, int cg, int grid, \
                                  size_t smem, cudaStream_t stream);
SPGEMM_DECLARE_BLOCK(nt)         // linear, A M x K, B N x K
SPGEMM_DECLARE_BLOCK(nn)         // linear, A M x K, B K x N
SPGEMM_DECLARE_BLOCK(tn)         // linear, A K x M, B K x N
SPGEMM_DECLARE_BLOCK(diag_out)   // kEpiDiagOut,  A M x K, B N x K
SPGEMM_DECLARE_BLOCK(diag_rows)  // kEpiDiagRows, A M x K, B K x N
SPGEMM_DECLARE_BLOCK(diag_cols)  // kEpiDiagCols, A M x K, B N x K
SPGEMM_DECLARE_BLOCK(gated)      // gated,          A M x K, B 2N x K
SPGEMM_DECLARE_BLOCK(gated_bwd)  // gated backward, A M x K, B K x N
#undef SPGEMM_DECLARE_BLOCK

}  // namespace spgemm
