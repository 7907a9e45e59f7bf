// pack.cu -- copies of operands whose rows the copy engine cannot read where
// they lie (row pitch or base address not 16-byte aligned) into rows padded
// to a multiple of 8 elements.  The matrices of a call go in one launch.
//
// Memory-bound: the 16-byte vectors of all padded copies form one range that
// the grid's threads stride over, kPackVecs at a time with their loads issued
// before the first store; the source words come from the two aligned 16-byte
// words around them, or, at the ends of the array, one element at a time.
// (One block per 256 vectors of a row group instead, most of them short: 23 us
// for the 37 MB of a 1531-wide block's weights, against 12 us.)
#include <cuda_runtime.h>

#include <cstdint>

#include "byte_shift.cuh"
#include "ops_internal.h"

namespace spgemm {

namespace {

constexpr int kPackThreads = 256;
constexpr int kPackVecs = 4;

__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackJobs jobs, int64_t total) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kPackThreads;
  for (int64_t v0 = static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x; v0 < total;
       v0 += kPackVecs * stride) {
    uint4 lo[kPackVecs], hi[kPackVecs];
    uint32_t shift[kPackVecs];
    const uint16_t* sp[kPackVecs];  // the vector's first element
    uint16_t* dp[kPackVecs];        // nullptr: past the end
    int valid[kPackVecs];           // elements inside the row
    bool fast[kPackVecs];
#pragma unroll
    for (int i = 0; i < kPackVecs; ++i) {
      int64_t v = v0 + i * stride;
      dp[i] = nullptr;
      fast[i] = false;
      shift[i] = 0u;
      valid[i] = 0;
      lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
      if (v >= total) continue;
      int n = 0;
      while (v >= jobs.job[n].vectors) v -= jobs.job[n++].vectors;
      const PackJob& j = jobs.job[n];
      const int64_t per = j.ldp / 8;
      const int64_t row = v < (int64_t{1} << 31) ? static_cast<uint32_t>(v) / static_cast<uint32_t>(per) : v / per;
      const int64_t c = (v - row * per) * 8;
      sp[i] = j.src + row * j.ld + c;
      dp[i] = j.dst + row * j.ldp + c;
      valid[i] = static_cast<int>(j.cols - c < 8 ? j.cols - c : 8);  // ldp < cols + 8, so at least 1
      const uintptr_t addr = reinterpret_cast<uintptr_t>(sp[i]);
      const uintptr_t base = addr & ~static_cast<uintptr_t>(15);
      if (base >= reinterpret_cast<uintptr_t>(j.src) &&
          base + 32 <= reinterpret_cast<uintptr_t>(j.src + (j.rows - 1) * j.ld + j.cols)) {
        lo[i] = __ldg(reinterpret_cast<const uint4*>(base));
        hi[i] = __ldg(reinterpret_cast<const uint4*>(base + 16));
        shift[i] = static_cast<uint32_t>(addr - base);
        fast[i] = true;
      }
    }
#pragma unroll
    for (int i = 0; i < kPackVecs; ++i) {
      if (dp[i] == nullptr) continue;
      uint4 out = make_uint4(0u, 0u, 0u, 0u);
      if (fast[i]) out = shift_window(lo[i], hi[i], shift[i]);
      uint32_t wd[4] = {out.x, out.y, out.z, out.w};
      if (!fast[i] || valid[i] < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (e >= valid[i])
            wd[e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
          else if (!fast[i])
            wd[e >> 1] |= static_cast<uint32_t>(__ldg(sp[i] + e)) << ((e & 1) * 16);
        }
      }
      *reinterpret_cast<uint4*>(dp[i]) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
    }
  }
}

}  // namespace

cudaError_t launch_pack(PackJobs jobs, int sm_count, cudaStream_t stream) {
  int64_t total = 0;
  for (int i = 0; i < jobs.count; ++i) {
    jobs.job[i].vectors = jobs.job[i].rows * (jobs.job[i].ldp / 8);
    total += jobs.job[i].vectors;
  }
  if (total == 0) return cudaSuccess;
  const int64_t blocks = ceil_div(total, kPackThreads * kPackVecs);
  const int64_t most = static_cast<int64_t>(sm_count) * 6;
  pack_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), kPackThreads, 0, stream>>>(jobs, total);
  return cudaGetLastError();
}

}  // namespace spgemm
