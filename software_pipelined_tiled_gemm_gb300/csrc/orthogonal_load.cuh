// orthogonal_load.cuh -- reading a gradient eight elements at a time and
// summing its squares, for the kernels of the orthogonalised update.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

namespace spgemm {

// Iterates are kept times this: a normalised matrix's elements (1 / sqrt(m n)
// in the mean) lie in fp16's normal range then.
constexpr float kIterateScale = 256.0f;

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Elements [c, c + 8) of a row (0 at and past n).
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t c, int64_t n, bool aligned, float (&v)[8]) {
  if (aligned && c + 8 <= n) {
    constexpr int kWords = sizeof(T) * 8 / 16;
    uint4 w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(row + c) + i);
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float<T>(e[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c + i < n ? to_float<T>(row[c + i]) : 0.0f;
}

// A sum of squares right for any fp32 elements: those below 2^-40 and above
// 2^40 are squared at another scale.  Ten instructions an element: only where
// the plain sum may have lost something (plain_sum_holds).
//
// The threads of a warp are summed in fp32 and only the warps in fp64: an SM
// does two fp64 operations a cycle, and sums, roots and quotients in every
// thread of a block took 3 to 8 us.
struct SquareSum {
  float mid = 0.0f, small = 0.0f, large = 0.0f;  // small x 2^80, large x 2^-70
  template <typename T>
  __device__ __forceinline__ void add(float x) {
    if (std::is_same<T, __half>::value) {  // within range
      mid = fmaf(x, x, mid);
      return;
    }
    const float size = fabsf(x);
    const float lo = size < 0x1p-40f ? x * 0x1p80f : 0.0f, hi = size > 0x1p40f ? x * 0x1p-70f : 0.0f;
    const float m = size < 0x1p-40f || size > 0x1p40f ? 0.0f : x;  // NaN is here
    small = fmaf(lo, lo, small);
    mid = fmaf(m, m, mid);
    large = fmaf(hi, hi, large);
  }
  // The sum over the block's threads, in thread 0 (shared: one per warp).
  template <int kThreads>
  __device__ __forceinline__ double block_total(double* shared) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mid += __shfl_xor_sync(0xffffffffu, mid, o);
      small += __shfl_xor_sync(0xffffffffu, small, o);
      large += __shfl_xor_sync(0xffffffffu, large, o);
    }
    if ((threadIdx.x & 31) == 0)
      shared[threadIdx.x >> 5] = static_cast<double>(mid) + static_cast<double>(small) * 0x1p-160 +
                                 static_cast<double>(large) * 0x1p140;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
      for (int i = 0; i < kThreads / 32; ++i) s += shared[i];
    return s;
  }
};

// A plain fp32 sum of squares in this range has neither overflowed nor lost
// more to underflow than 2^-60 of itself in 2^30 elements.
__device__ __forceinline__ bool plain_sum_holds(double sum) { return sum > 0x1p-60 && sum < 0x1p100; }

// The square root of kIterateScale / max(|G|, eps): the scale in two equal
// factors, each within fp32's range.  The fourth root of the squares' sum is
// taken in fp32 of a mantissa in [1, 16), within 2^-22 of exact.
__device__ __forceinline__ float half_scale(double squares, float eps) {
  const double least = static_cast<double>(eps) * eps;
  if (squares < least) squares = least;
  if (!(squares <= 1e300)) return squares != squares ? __int_as_float(0x7fffffff) : 0.0f;
  const int k = (((__double2hiint(squares) >> 20) & 0x7ff) - 1023) >> 2;  // squares = m 16^k
  const float m = static_cast<float>(squares * __hiloint2double((1023 - 4 * k) << 20, 0));
  static_assert(kIterateScale == 256.0f, "its root");
  return 16.0f / sqrtf(sqrtf(m)) * __int_as_float((127 - k) << 23);
}

}  // namespace spgemm
