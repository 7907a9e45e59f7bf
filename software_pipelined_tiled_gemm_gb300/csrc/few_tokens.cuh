// few_tokens.cuh -- what the passes over weights for a few tokens share
// (few_tokens.cu, grouped_few.cu): the layout of tokens in shared memory, the
// instruction, and vectors of rows that are not 16-byte aligned.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "byte_shift.cuh"

namespace spgemm {

// 16-byte words of a token's row in shared memory: an odd multiple of 64 bytes,
// so that the rows of an instruction's tokens lie in different banks.
__host__ __device__ constexpr int token_pitch(int k) { return (k + 63) / 64 * 8 + 4; }

template <bool kBf16>
__device__ __forceinline__ uint16_t round16(float v) {
  if constexpr (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}

// c += rows (16 x 16) times tokens (16 x 8).
template <bool kBf16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  if constexpr (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The eight elements from p on (`end`: past the array's last), as the aligned
// words around them.  The second is read only if it holds an element of the
// array; each has one, so both lie in its allocation.
struct Window {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const uint16_t* p, const uint16_t* end, bool in) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), base = at & ~uintptr_t{15};
    lo = hi = make_uint4(0u, 0u, 0u, 0u);
    if (in) lo = __ldcg(reinterpret_cast<const uint4*>(base));
    if (in && at != base && base + 16 < reinterpret_cast<uintptr_t>(end))
      hi = __ldcg(reinterpret_cast<const uint4*>(base + 16));
  }
  // The first `count` of them, 0 after those.
  __device__ __forceinline__ uint4 get(const uint16_t* p, int count) const {
    const uint4 v = shift_window(lo, hi, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u));
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (count < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= count) w[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

}  // namespace spgemm
