// grouped_params.h -- launch parameters of the products grouped by expert
// (grouped_kernel.cuh) shared by the host code (grouped.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernel_params.h"

namespace spgemm {

// Which product.  In each the tile's lanes (the MMA's M side) run along an
// output row and its columns over output rows:
//   kForward   lanes: features n, columns: tokens of a group,  sum over k
//   kInput     lanes: features k, columns: tokens of a group,  sum over n
//   kWeight    lanes: features k, columns: rows n of dW_e,     sum over tokens
constexpr int kGroupedForward = 0, kGroupedInput = 1, kGroupedWeight = 2;

constexpr int kGroupedLanes = 256;    // of a CTA pair
constexpr int kGroupedUnit = 32;      // a tile's columns are a multiple of this (16 a CTA)
constexpr int kGroupedCols = 256;     // and at most this
constexpr int kGroupedTail = 16;      // tokens of one MMA step
constexpr int kGroupedStages = 7;     // ring slots at most
constexpr uint32_t kGroupedSlot = 2u * kStageA;  // A and B: 128 rows (or columns) x 64 each
constexpr int kGroupedThreads = 64 + 128 * 2;

struct GroupedParams : Params {  // of Params: stages, bf16, status, timeout_ns, inject_fault
  const int64_t* offsets;
  int groups;
  int rows;            // of x
  int reduce;          // length of the sum (kForward: k, kInput: n)
  int lanes;           // extent along the lanes
  int cols;            // kWeight: rows n of dW_e
  int tiles_lane;      // tiles along the lanes
  int cap;             // columns of a tile at most
  int zero_rest;
  int pairs;           // CTA pairs of the launch
  uint16_t* out;
  int64_t ldo;         // row pitch of the output; kWeight: of dW_e
  int64_t out_group;   // kWeight: elements of one dW_e
  int wide;            // output words of two elements (rows 4-byte aligned)
};

struct GroupedMaps {
  CUtensorMap a;       // kForward, kInput: w; kWeight: x
  CUtensorMap b[4];    // kForward, kInput: rows of x or dy, boxes of 16, 32, 64 and 128 rows;
                       // kWeight: dy, then the tails of x and dy
};

// Shared memory beside the ring: the groups' offsets and first tile rows.
inline size_t grouped_table_bytes(int groups) { return 2u * sizeof(int) * static_cast<size_t>(groups + 1); }
inline size_t grouped_smem_bytes(int stages, int groups) {
  return kAlignSlack + static_cast<size_t>(stages) * kGroupedSlot + 8u * (2 * kGroupedStages + 5) + 16u +
         grouped_table_bytes(groups);
}

cudaError_t grouped_set_smem(size_t smem);
cudaError_t grouped_launch(int kind, const GroupedMaps& m, const GroupedParams& p, size_t smem,
                           cudaStream_t stream);

}  // namespace spgemm
