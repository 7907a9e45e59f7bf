// pack.cu -- copies of operands whose rows the copy engine cannot read where
// they lie (row pitch or base address not 16-byte aligned) into rows padded
// to a multiple of 8 elements.  The matrices of a call go in one launch.
//
// Memory-bound: a warp copies a row at a time, kPackVecs 16-byte vectors per
// lane with their loads issued before the first store.  The source words of a
// vector come from the two aligned 16-byte words around it; words that reach
// over the ends of the array are put together from single elements.
#include <cuda_runtime.h>

#include <cstdint>

#include "byte_shift.cuh"
#include "ops_internal.h"

namespace spgemm {

namespace {

constexpr int kPackThreads = 256;
constexpr int kPackVecs = 4;

// The aligned 16-byte word at `addr`, with 0 for elements outside [first, end).
__device__ __forceinline__ uint4 load_word(uintptr_t addr, uintptr_t first, uintptr_t end) {
  if (addr >= first && addr + 16 <= end) return __ldg(reinterpret_cast<const uint4*>(addr));
  uint32_t wd[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uintptr_t at = addr + 2 * e;
    if (at >= first && at + 2 <= end)
      wd[e >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(at))) << ((e & 1) * 16);
  }
  return make_uint4(wd[0], wd[1], wd[2], wd[3]);
}

__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackJobs jobs, int64_t rows) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kPackThreads / 32);
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x) / 32; r < rows; r += warps) {
    int64_t row = r;
    int n = 0;
    while (row >= jobs.job[n].rows) row -= jobs.job[n++].rows;
    const PackJob& j = jobs.job[n];
    const uintptr_t first = reinterpret_cast<uintptr_t>(j.src);
    const uintptr_t end = reinterpret_cast<uintptr_t>(j.src + (j.rows - 1) * j.ld + j.cols);
    const uintptr_t start = reinterpret_cast<uintptr_t>(j.src + row * j.ld);
    const uint32_t shift = static_cast<uint32_t>(start & 15u);
    const uintptr_t base = start - shift;
    uint4* dst = reinterpret_cast<uint4*>(j.dst + row * j.ldp);
    const int64_t per = j.ldp / 8;
    for (int64_t v0 = lane; v0 < per; v0 += 32 * kPackVecs) {
      uint4 lo[kPackVecs], hi[kPackVecs];
#pragma unroll
      for (int i = 0; i < kPackVecs; ++i) {
        const int64_t v = v0 + 32 * i;
        lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
        if (v < per) {
          lo[i] = load_word(base + 16 * v, first, end);
          if (shift != 0) hi[i] = load_word(base + 16 * v + 16, first, end);
        }
      }
#pragma unroll
      for (int i = 0; i < kPackVecs; ++i) {
        const int64_t v = v0 + 32 * i;
        if (v >= per) break;
        const uint4 out = shift_window(lo[i], hi[i], shift);
        uint32_t wd[4] = {out.x, out.y, out.z, out.w};
        const int64_t valid = j.cols - 8 * v;  // elements of the vector inside the row
        if (valid < 8) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e >= valid) wd[e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
        }
        dst[v] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_pack(const PackJobs& jobs, int sm_count, cudaStream_t stream) {
  int64_t rows = 0;
  for (int i = 0; i < jobs.count; ++i) rows += jobs.job[i].rows;
  if (rows == 0) return cudaSuccess;
  const int64_t blocks = ceil_div(rows, kPackThreads / 32);
  const int64_t most = static_cast<int64_t>(sm_count) * 8;
  pack_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), kPackThreads, 0, stream>>>(jobs, rows);
  return cudaGetLastError();
}

}  // namespace spgemm
