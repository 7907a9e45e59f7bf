// pack.cu -- copies of operands whose rows the copy engine cannot read where
// they lie (row pitch or base address not 16-byte aligned) into rows padded
// to a multiple of 8 elements.  The matrices of a call go in one launch.
//
// Memory-bound: a thread writes 16 bytes per row for kPackRows rows, its
// loads all issued before the first store; the source words come from the
// two aligned 16-byte words around them, or, at the ends of the array, one
// element at a time.
#include <cuda_runtime.h>

#include <cstdint>

#include "byte_shift.cuh"
#include "ops_internal.h"

namespace spgemm {

namespace {

constexpr int kPackThreads = 256;
constexpr int kPackRows = 4;

__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackJobs jobs) {
  const PackJob& j = jobs.job[blockIdx.z];
  const int64_t v = static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x;
  const int64_t c0 = v * 8;
  if (c0 >= j.ldp) return;
  const int64_t valid = j.cols - c0 < 8 ? (j.cols > c0 ? j.cols - c0 : 0) : 8;
  const uintptr_t first = reinterpret_cast<uintptr_t>(j.src);
  const uintptr_t end = reinterpret_cast<uintptr_t>(j.src + (j.rows - 1) * j.ld + j.cols);
  for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * kPackRows; row0 < j.rows;
       row0 += static_cast<int64_t>(gridDim.y) * kPackRows) {
    uint4 lo[kPackRows], hi[kPackRows];
    uint32_t shift[kPackRows];
    bool fast[kPackRows];
#pragma unroll
    for (int i = 0; i < kPackRows; ++i) {
      fast[i] = false;
      shift[i] = 0u;
      lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row0 + i < j.rows && valid > 0) {
        const uintptr_t addr = reinterpret_cast<uintptr_t>(j.src + (row0 + i) * j.ld + c0);
        const uintptr_t base = addr & ~static_cast<uintptr_t>(15);
        if (base >= first && base + 32 <= end) {
          lo[i] = __ldg(reinterpret_cast<const uint4*>(base));
          hi[i] = __ldg(reinterpret_cast<const uint4*>(base + 16));
          shift[i] = static_cast<uint32_t>(addr - base);
          fast[i] = true;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kPackRows; ++i) {
      if (row0 + i >= j.rows) break;
      uint4 out = make_uint4(0u, 0u, 0u, 0u);
      if (fast[i]) out = shift_window(lo[i], hi[i], shift[i]);
      uint32_t wd[4] = {out.x, out.y, out.z, out.w};
      const uint16_t* sp = j.src + (row0 + i) * j.ld + c0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= valid)
          wd[e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
        else if (!fast[i])
          wd[e >> 1] |= static_cast<uint32_t>(__ldg(sp + e)) << ((e & 1) * 16);
      }
      *reinterpret_cast<uint4*>(j.dst + (row0 + i) * j.ldp + c0) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
    }
  }
}

}  // namespace

cudaError_t launch_pack(const PackJobs& jobs, cudaStream_t stream) {
  int64_t vecs = 0, groups = 0;
  for (int i = 0; i < jobs.count; ++i) {
    vecs = vecs > jobs.job[i].ldp / 8 ? vecs : jobs.job[i].ldp / 8;
    const int64_t g = ceil_div(jobs.job[i].rows, kPackRows);
    groups = groups > g ? groups : g;
  }
  if (vecs == 0 || groups == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(ceil_div(vecs, kPackThreads)),
                  static_cast<unsigned>(groups < 65535 ? groups : 65535),
                  static_cast<unsigned>(jobs.count));
  pack_kernel<<<grid, kPackThreads, 0, stream>>>(jobs);
  return cudaGetLastError();
}

}  // namespace spgemm
