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
constexpr int kGroupedStages = 3;     // ring slots
constexpr int kGroupedSlices = 2;     // of 64 of the sum, in a slot
constexpr int kGroupedK = kGroupedSlices * kBK;
constexpr uint32_t kGroupedOperand = kGroupedSlices * kStageA;  // 128 rows (or columns) of A or B
constexpr uint32_t kGroupedSlot = 2u * kGroupedOperand;
constexpr int kGroupedThreads = 64 + 128 * 2 + 64;
constexpr int kGroupedAhead = 4;      // tiles that a CTA's scheduler describes ahead

// What a tile costs, in clocks of a CTA pair.  A slot: 128 a
// unit of 32 columns for the tensor cores, or what its copies take at the 64
// bytes a clock that an SM receives: 32 KiB of one operand and boxes of 16 to
// 128 rows of the other.  So a tile of 224 columns costs one of 256, and one of
// 32 more than half of that; a group's rows make full tiles and one for the
// rest.  A tile's start and end: 1500.
__host__ __device__ constexpr int grouped_box(int width) { return width <= 32 ? 0 : width <= 64 ? 1 : width <= 128 ? 2 : 3; }
__host__ __device__ constexpr float grouped_tile_clocks(int width, int slots) {
  const int math = 4 * width, copies = 512 + (64 << grouped_box(width));
  return static_cast<float>(slots) * static_cast<float>(math > copies ? math : copies) + 1500.0f;
}
// Widths of full tiles to choose from.
constexpr int kGroupedCaps = 4;
__host__ __device__ constexpr int grouped_cap(int i) { return kGroupedCols >> i; }
// Tiles of a strip of `extent` columns, and their clocks.
__host__ __device__ constexpr int grouped_tiles(int extent, int cap) { return (extent + cap - 1) / cap; }
__host__ __device__ constexpr float grouped_strip_clocks(int extent, int cap, int slots) {
  const int full = extent / cap, rest = extent - full * cap;
  return static_cast<float>(full) * grouped_tile_clocks(cap, slots) + (rest > 0 ? grouped_tile_clocks(rest, slots) : 0.0f);
}
// Clocks of `tiles` tiles that take `clocks` in all on `pairs` walkers: an even
// share, and what the last round leaves idle.
__host__ __device__ constexpr float grouped_clocks(float clocks, int tiles, int cap, int slots, int pairs) {
  const int idle = (tiles + pairs - 1) / pairs * pairs - tiles;
  return (clocks + static_cast<float>(idle) * grouped_tile_clocks(cap, slots)) / static_cast<float>(pairs);
}

struct GroupedParams : Params {  // of Params: stages, bf16, status, timeout_ns, inject_fault
  const int64_t* offsets;
  int groups;
  int rows;            // of x
  int reduce;          // length of the sum (kForward: k, kInput: n)
  int lanes;           // extent along the lanes
  int cols;            // kWeight: rows n of dW_e
  int tiles_lane;      // tiles along the lanes
  int cap;             // kWeight: columns of a tile at most (the other kinds choose on the device)
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
  return kAlignSlack + static_cast<size_t>(stages) * kGroupedSlot + 8u * (2 * kGroupedStages + 5 + 2 * kGroupedAhead) + 16u + 48u * kGroupedAhead + 16u +
         grouped_table_bytes(groups);
}

cudaError_t grouped_set_smem(size_t smem);
cudaError_t grouped_launch(int kind, const GroupedMaps& m, const GroupedParams& p, size_t smem,
                           cudaStream_t stream);

}  // namespace spgemm
