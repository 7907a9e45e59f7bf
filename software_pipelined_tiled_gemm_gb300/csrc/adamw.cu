// adamw.cu -- the AdamW step of many tensors, with states in fp32 or in 8 bits.
//
// Bound by memory: parameter and states are read and written, the gradient
// read and the copy written, each once.  All tensors go in one launch (of up
// to kMostTensors): their table travels with the kernel's arguments, so
// nothing is copied to the device before it and a captured call keeps it.
//
// The states of 256 neighbouring elements are a block; a warp takes a block at
// a time, a lane eight elements, so a block's largest magnitude takes one
// reduction instruction.  A thread block has a chunk of one tensor, whose
// addresses are found once; its warps fetch their next blocks to shared memory
// while they compute.  Tensors whose addresses allow no 16-byte vectors, and a
// tensor's last block, are read element by element (67 M elements, bf16 gradients and
// copies: 273 us with 32-bit states and 196 with 8-bit ones, 664 and 556 from odd addresses).
//
// With 8-bit states the arithmetic (some 400 instructions a lane and block,
// a fifth of them for square roots in full precision) takes about as long as
// the memory, so it is done on pairs of values where it can be.
//
// 8 bits: e4m3 times the block's scale, the average's and the second moment's
// root's.  The root (not v) halves the range of exponents that the format has
// to hold: 2^-9 .. 448 covers ratios of 2^36 in v.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "ops_internal.h"
#include "packed_f32.cuh"
#include "ptx.cuh"

using namespace spgemm;

namespace {

constexpr int kBlock = GEMM_ADAMW_BLOCK;
constexpr int kEach = 8;                 // elements of a lane: 32 lanes, one block
constexpr int kPairs = kEach / 2;
constexpr int kThreads = 256, kWarps = kThreads / 32;
// Blocks of a warp on their way or in work, thread blocks of an SM that the
// registers are shared out for (of four with 32-bit states, 64 KiB of ring
// each, three fit its shared memory), and blocks of a warp in a chunk at most.
// Measured, in us (252 M elements with 8-bit states; 106 M with 32-bit ones):
//   8 bits    3, 3 and 1 / 3 / 4 / 5 / 8:  816 / 612 / 605 / 704 / 697;  2, 4 and 4: 632;  4, 2 and 16: 642
//   32 bits   2, 4 and 2: 429;  2, 3 and 2 / 3 / 4: 430 / 435 / 440;  1, 4 and 2 / 4: 437 / 450;  3, 2 and 4: 433
constexpr int kSlots8 = 3, kOcc8 = 3, kMostEach8 = 4;
constexpr int kSlots32 = 2, kOcc32 = 4, kMostEach32 = 2;
// Types of an entry: parameter, gradient, copy (3: none), two bits each, and
// whether its addresses allow vectors.
constexpr uint32_t kNoCopy = 3u, kVectors = 1u << 6;

struct Entry {
  void* param;
  const void* grad;
  void* copy;
  int64_t numel;
  int64_t state;         // first element of the states
  uint32_t first_chunk;  // of this launch
  uint32_t kinds;
  float decay;           // weight decay
};

// Tables of two sizes: a launch's arguments cost the host time (a call of 32 tensors
// takes it 4.6 us, one of 33, with the larger table, 5.9).
constexpr int kFewTensors = 32, kMostTensors = 512;
template <int kTensors>
struct Job {
  Entry entry[kTensors];
  int count;
  uint32_t chunk;         // blocks of a thread block, all of one tensor
  void* exp_avg;
  void* exp_avg_sq;
  float* scales;          // of exp_avg, then (scale_step later) of exp_avg_sq
  int64_t scale_step;
  const int64_t* step;
  const float* lr_device;
  const float* scale;
  float lr, beta1, beta2, one_less1, one_less2, ln_beta1, ln_beta2, eps, one;
};

// Eight fp32 values, in pairs, from fp16, bf16 or fp32 at p.
__device__ __forceinline__ void load8(const void* p, uint32_t kind, F32x2 (&v)[kPairs]) {
  if (kind == GEMM_IN_F32) {
    const ulonglong2 a = static_cast<const ulonglong2*>(p)[0], b = static_cast<const ulonglong2*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    return;
  }
  const uint4 raw = *static_cast<const uint4*>(p);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    if (kind == GEMM_IN_BF16) {  // a bf16 is the upper half of its fp32
      v[i] = pack_f32(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[i] = pack_f32(f.x, f.y);
    }
  }
}

__device__ __forceinline__ void store8(void* p, uint32_t kind, const F32x2 (&v)[kPairs]) {
  if (kind == GEMM_IN_F32) {
    __stcs(static_cast<ulonglong2*>(p), make_ulonglong2(v[0], v[1]));
    __stcs(static_cast<ulonglong2*>(p) + 1, make_ulonglong2(v[2], v[3]));
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const float2 f = unpack_f32(v[i]);
    if (kind == GEMM_IN_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      memcpy(&w[i], &h, 4);
    } else {
      const __half2 h = __floats2half2_rn(f.x, f.y);
      memcpy(&w[i], &h, 4);
    }
  }
  __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

__device__ __forceinline__ float load1(const void* p, uint32_t kind, int64_t i) {
  if (kind == GEMM_IN_F32) return static_cast<const float*>(p)[i];
  if (kind == GEMM_IN_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ void store1(void* p, uint32_t kind, int64_t i, float v) {
  if (kind == GEMM_IN_F32)
    static_cast<float*>(p)[i] = v;
  else if (kind == GEMM_IN_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// e4m3 codes of two values a half-word; |x| is at most 448 (1 + 2^-22).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  return __half22float2(__half2(h));
}

// The largest magnitude of three values, NaN if one is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) { return fminf(fminf(a, b), c); }

// 1 / x to one unit in the last place; x is 0, normal or infinite (a sum of an eps
// that is not subnormal and a square root of an fp32 number).
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Four e4m3 codes of y rounded down after adding u 2^-20 steps, from s = the
// bits of 2^-120 y as fp32, plus u.  With that factor fp32's exponent is
// e4m3's, and the fp32 numbers below its normal range are e4m3's below its
// own: in both a step of the code is 2^20 units of the bits, so the sum's
// upper bits are the code.  (Only the largest, 448 plus rounding, can carry
// into the code of NaN, from which it is taken back.)
__device__ __forceinline__ uint32_t dithered_codes(uint32_t s0, uint32_t s1, uint32_t s2, uint32_t s3) {
  const uint32_t w = (s0 >> 20) | (s1 >> 20) << 8 | (s2 >> 20) << 16 | (s3 >> 20) << 24;
  return w - (((w + 0x01010101u) & 0x80808080u) >> 7);
}

// Entry of chunk c: the last whose first chunk is not after it.
template <typename J>
__device__ __forceinline__ int find_entry(const J& job, uint32_t c) {
  int lo = 0, hi = job.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (job.entry[mid].first_chunk <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void copy_async16(uint32_t smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t smem, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem), "l"(src) : "memory");
}

// A warp's ring: the blocks that it works on next are on their way while it
// works on one.  Of a block: parameters and gradients (1 KiB each where they
// are fp32), the two states, their scales.
template <int kBits>
struct Ring {
  static constexpr uint32_t kState = kBlock * kBits / 8;
  static constexpr uint32_t kGrad = 1024u, kM = 2048u, kV = kM + kState, kScales = kV + kState;
  static constexpr uint32_t kSlot = kScales + (kBits == 8 ? 16u : 0u);
  static constexpr int kSlots = kBits == 8 ? kSlots8 : kSlots32;
  static constexpr size_t kBytes = static_cast<size_t>(kWarps) * kSlots * kSlot;
};

template <int kBits, int kTensors>
__global__ void __launch_bounds__(kThreads, kBits == 8 ? kOcc8 : kOcc32) adamw_kernel(const __grid_constant__ Job<kTensors> job) {
  using R = Ring<kBits>;
  extern __shared__ __align__(16) uint8_t ring[];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Entry& e = job.entry[find_entry(job, blockIdx.x)];
  const uint32_t kp = e.kinds & 3u, kg = (e.kinds >> 2) & 3u, kc = (e.kinds >> 4) & 3u;
  const int psize = kp == GEMM_IN_F32 ? 4 : 2, gsize = kg == GEMM_IN_F32 ? 4 : 2;
  // This warp's blocks: every eighth of the chunk.
  const int64_t first = static_cast<int64_t>(blockIdx.x - e.first_chunk) * job.chunk + warp;
  const int64_t blocks = (e.numel + kBlock - 1) / kBlock;  // of the tensor
  const int count = static_cast<int>(min(static_cast<int64_t>(job.chunk - warp + kWarps - 1), blocks - first + kWarps - 1)) / kWarps;
  // Of those, the ones that are all the tensor's and whose addresses allow vectors.
  const int whole = (e.kinds & kVectors) == 0 ? 0 : first + static_cast<int64_t>(count - 1) * kWarps < e.numel / kBlock ? count : count - 1;
  uint8_t* mine = ring + warp * (R::kSlots * R::kSlot);

  const int64_t at0 = first * kBlock, state0 = e.state + at0;
  const uint8_t* from_p = static_cast<const uint8_t*>(e.param) + at0 * psize + lane * 16;
  const uint8_t* from_g = static_cast<const uint8_t*>(e.grad) + at0 * gsize + lane * 16;
  const uint8_t* from_m = static_cast<const uint8_t*>(job.exp_avg) + state0 * (kBits / 8) + lane * 16;
  const uint8_t* from_v = static_cast<const uint8_t*>(job.exp_avg_sq) + state0 * (kBits / 8) + lane * 16;
  if (kBits == 8 && lane >= 16) from_m = from_v - 256;
  const float* from_s = kBits == 8 ? job.scales + (lane & 1) * job.scale_step + state0 / kBlock : nullptr;
  auto fetch = [&](int i, int slot) {
    if (i < whole) {
      const uint32_t to = ptx::smem_addr(mine + slot * R::kSlot) + lane * 16;
      const int64_t skip = static_cast<int64_t>(i) * (kWarps * kBlock);
      copy_async16(to, from_p + skip * psize);
      if (kp == GEMM_IN_F32) copy_async16(to + 512, from_p + skip * 4 + 512);
      copy_async16(to + R::kGrad, from_g + skip * gsize);
      if (kg == GEMM_IN_F32) copy_async16(to + R::kGrad + 512, from_g + skip * 4 + 512);
      if constexpr (kBits == 32) {
        copy_async16(to + R::kM, from_m + skip * 4);
        copy_async16(to + R::kM + 512, from_m + skip * 4 + 512);
        copy_async16(to + R::kV, from_v + skip * 4);
        copy_async16(to + R::kV + 512, from_v + skip * 4 + 512);
      } else {
        copy_async16(to + R::kM, from_m + skip);  // m, and v by the upper lanes
        if (lane < 2) copy_async4(to + R::kScales - lane * 12, from_s + i * kWarps);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < R::kSlots - 1; ++i) fetch(i, i);

  // 1 - beta^t = -expm1(t ln beta), which keeps its bits where beta^t is near 1.
  const uint32_t t = static_cast<uint32_t>(*job.step) + 1u;
  const float lr = job.lr_device ? *job.lr_device : job.lr;
  const float factor = job.scale ? *job.scale : 1.0f;
  const float rate = lr / -expm1f(static_cast<float>(t) * job.ln_beta1);
  const float unbias = rsqrtf(-expm1f(static_cast<float>(t) * job.ln_beta2));
  const F32x2 keep = both_f32(-lr * e.decay), step_size = both_f32(-rate), unbiases = both_f32(unbias);
  const F32x2 factors = both_f32(factor), beta1 = both_f32(job.beta1), beta2 = both_f32(job.beta2);
  const F32x2 less1 = both_f32(job.one_less1), less2 = both_f32(job.one_less2), eps = both_f32(job.eps);
  // A sum below is the product with a one that the assembler does not know, plus the rest:
  // it merges a packed product and the packed sum that follows into one rounding.
  const F32x2 one = both_f32(job.one);
  int slot = 0;
  for (int n = 0; n < count; ++n) {
    fetch(n + R::kSlots - 1, slot == 0 ? R::kSlots - 1 : slot - 1);
    const int64_t at = at0 + static_cast<int64_t>(n) * (kWarps * kBlock) + lane * kEach;  // in the tensor
    const int64_t state = e.state + at;
    F32x2 p[kPairs], g[kPairs], m[kPairs], v[kPairs];
    uint2 cm, cv;
    float sm_old, sv_old;
    int left = kEach;  // elements that exist
    if (n < whole) {
      asm volatile("cp.async.wait_group %0;" ::"n"(R::kSlots - 1) : "memory");
      __syncwarp();  // lanes read what others copied
      const uint8_t* from = mine + slot * R::kSlot;
      load8(from + lane * kEach * psize, kp, p);
      load8(from + R::kGrad + lane * kEach * gsize, kg, g);
      if constexpr (kBits == 32) {
        load8(from + R::kM + lane * 32, GEMM_IN_F32, m);
        load8(from + R::kV + lane * 32, GEMM_IN_F32, v);
      } else {
        cm = *reinterpret_cast<const uint2*>(from + R::kM + lane * 8);
        cv = *reinterpret_cast<const uint2*>(from + R::kV + lane * 8);
        const float2 s = *reinterpret_cast<const float2*>(from + R::kScales);
        sm_old = s.x;
        sv_old = s.y;
      }
      __syncwarp();  // before the slot is filled again
    } else {
      // A tensor's last block may end inside: elements that do not exist count as zeros, and
      // so do their states, which are written all the same (they are the buffer's own).
      left = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(kEach), e.numel - at)));
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int j = 2 * i;
        p[i] = pack_f32(j < left ? load1(e.param, kp, at + j) : 0.0f, j + 1 < left ? load1(e.param, kp, at + j + 1) : 0.0f);
        g[i] = pack_f32(j < left ? load1(e.grad, kg, at + j) : 0.0f, j + 1 < left ? load1(e.grad, kg, at + j + 1) : 0.0f);
      }
      if constexpr (kBits == 32) {
        load8(static_cast<const float*>(job.exp_avg) + state, GEMM_IN_F32, m);
        load8(static_cast<const float*>(job.exp_avg_sq) + state, GEMM_IN_F32, v);
      } else {
        cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(job.exp_avg) + state);
        cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(job.exp_avg_sq) + state);
        sm_old = job.scales[state / kBlock];
        sv_old = job.scales[job.scale_step + state / kBlock];
      }
    }
    slot = slot == R::kSlots - 1 ? 0 : slot + 1;
    if constexpr (kBits == 8) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 fm = from_e4m3x2((i < 2 ? cm.x : cm.y) >> (16 * (i & 1)));
        const float2 fv = from_e4m3x2((i < 2 ? cv.x : cv.y) >> (16 * (i & 1)));
        m[i] = mul_f32x2(pack_f32(fm.x, fm.y), both_f32(sm_old));
        const F32x2 r = mul_f32x2(pack_f32(fv.x, fv.y), both_f32(sv_old));
        v[i] = mul_f32x2(r, r);
      }
    }
    // Each operation on the states is rounded by itself (no fused multiply-add):
    // whoever evaluates the formulas in fp32 step by step gets the same bits,
    // and in 8 bits, where a last bit can decide a code, the same codes.
    float r[kEach];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      g[i] = mul_f32x2(g[i], factors);
      m[i] = fma_f32x2(mul_f32x2(beta1, m[i]), one, mul_f32x2(less1, g[i]));
      v[i] = fma_f32x2(mul_f32x2(beta2, v[i]), one, mul_f32x2(less2, mul_f32x2(g[i], g[i])));
      const float2 vi = unpack_f32(v[i]);
      r[2 * i] = __fsqrt_rn(vi.x);
      r[2 * i + 1] = __fsqrt_rn(vi.y);
      const float2 d = unpack_f32(fma_f32x2(pack_f32(r[2 * i], r[2 * i + 1]), unbiases, eps));
      // (The quotient is within 2 units of its last place, and p is larger.)
      const F32x2 q = mul_f32x2(m[i], pack_f32(reciprocal(d.x), reciprocal(d.y)));
      p[i] = fma_f32x2(step_size, q, fma_f32x2(keep, p[i], p[i]));
    }
    if (n < whole) {
      store8(static_cast<uint8_t*>(e.param) + at * psize, kp, p);
      if (kc != kNoCopy) store8(static_cast<uint16_t*>(e.copy) + at, kc, p);
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float2 pi = unpack_f32(p[i / 2]);
        if (i < left) {
          store1(e.param, kp, at + i, i % 2 ? pi.y : pi.x);
          if (kc != kNoCopy) store1(e.copy, kc, at + i, i % 2 ? pi.y : pi.x);
        } else {
          float2 mi = unpack_f32(m[i / 2]), vi = unpack_f32(v[i / 2]);
          (i % 2 ? mi.y : mi.x) = 0.0f;
          (i % 2 ? vi.y : vi.x) = 0.0f;
          m[i / 2] = pack_f32(mi.x, mi.y);
          v[i / 2] = pack_f32(vi.x, vi.y);
          r[i] = 0.0f;
        }
      }
    }
    if constexpr (kBits == 32) {
      store8(static_cast<float*>(job.exp_avg) + state, GEMM_IN_F32, m);
      store8(static_cast<float*>(job.exp_avg_sq) + state, GEMM_IN_F32, v);
    } else {
      float top_m = 0.0f, top_r = 0.0f, least_r = r[0];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 mi = unpack_f32(m[i]);
        top_m = max3_abs(top_m, mi.x, mi.y);
        top_r = max3_abs(top_r, r[2 * i], r[2 * i + 1]);
        least_r = min3(least_r, r[2 * i], r[2 * i + 1]);
      }
      // Magnitudes order as their bits, NaN above all.
      const uint32_t bm = __reduce_max_sync(0xffffffffu, __float_as_uint(top_m) & 0x7fffffffu);
      const uint32_t br = __reduce_max_sync(0xffffffffu, __float_as_uint(top_r) & 0x7fffffffu);
      constexpr float kLeast = 7.52316384526264e-37f;  // 2^-120
      const float sm = bm <= 0x7f800000u ? fmaxf(__fmul_rn(__uint_as_float(bm), 1.0f / 448.0f), kLeast) : __uint_as_float(bm);
      const float sv = br <= 0x7f800000u ? fmaxf(__fmul_rn(__uint_as_float(br), 1.0f / 448.0f), kLeast) : __uint_as_float(br);
      const float im = __frcp_rn(sm), iv = __frcp_rn(sv);
      const F32x2 ims = both_f32(im), ivs = both_f32(iv), down = both_f32(kLeast);
      const uint32_t dither = static_cast<uint32_t>(state) * 0xC13FA9A9u + t * 0x91E10DA5u;
      uint32_t wm[2] = {0u, 0u}, s[kEach];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 y = unpack_f32(mul_f32x2(mul_f32x2(pack_f32(r[2 * i], r[2 * i + 1]), ivs), down));
        s[2 * i] = __float_as_uint(y.x) + ((dither + static_cast<uint32_t>(2 * i) * 0xC13FA9A9u) >> 12);
        s[2 * i + 1] = __float_as_uint(y.y) + ((dither + static_cast<uint32_t>(2 * i + 1) * 0xC13FA9A9u) >> 12);
        const float2 mi = unpack_f32(mul_f32x2(m[i], ims));
        wm[i >> 1] |= e4m3x2(mi.x, mi.y) << (16 * (i & 1));
      }
      // Nothing but 0 becomes 0: a root below a step of the smallest codes, 2^-9 sv.
      if (least_r * iv < 0.001953125f) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) s[i] = r[i] > 0.0f ? max(s[i], 1u << 20) : 0u;
      }
      uint32_t wv[2] = {dithered_codes(s[0], s[1], s[2], s[3]), dithered_codes(s[4], s[5], s[6], s[7])};
      if (!(sv <= 3.4028235e38f)) wv[0] = wv[1] = 0x7f7f7f7fu;  // an infinite or NaN root: all of the block NaN
      __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(job.exp_avg) + state), make_uint2(wm[0], wm[1]));
      __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(job.exp_avg_sq) + state), make_uint2(wv[0], wv[1]));
      if (lane == 0) {
        __stcs(job.scales + state / kBlock, sm);
        __stcs(job.scales + job.scale_step + state / kBlock, sv);
      }
    }
  }
}

// Counts the step once the call's last kernel has ended, so that nothing reads it while it
// changes.  (Counted by the last of the thread blocks to have read it, which takes an atomic
// addition of each and a barrier: 608 us in place of 600 for 252 M elements with 8-bit states,
// and 615 where the reads that run beside those additions are relaxed loads.)
__global__ void count_kernel(int64_t* step) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  *step += 1;
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), unsigned blocks, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int64_t padded(int64_t n) { return (n + kBlock - 1) / kBlock * kBlock; }

gemm_status_t check(const gemm_adamw_args_t* a) {
  if (!a) return ops_fail(GEMM_ERR_INVALID_ARG, "args is NULL");
  if (a->count < 0 || (a->count > 0 && !a->tensors)) return ops_fail(GEMM_ERR_INVALID_ARG, "tensors is NULL or count < 0");
  if (a->bits != 32 && a->bits != 8) return ops_fail(GEMM_ERR_INVALID_ARG, "bits %d not in {8, 32}", a->bits);
  if (!(a->beta1 >= 0.0 && a->beta1 < 1.0 && a->beta2 >= 0.0 && a->beta2 < 1.0))
    return ops_fail(GEMM_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
  // As fp32, 0 or where the reciprocal of a sum with it is a normal number (0 / 1e-40 would be 0 times infinity).
  const float eps = static_cast<float>(a->eps);
  if (!(a->eps == 0.0 || (eps >= 1.1754943508222875e-38f && eps <= 8.507059173023462e+37f)))
    return ops_fail(GEMM_ERR_INVALID_ARG, "eps must be 0 or between 2^-126 and 2^126");
  if (!a->step) return ops_fail(GEMM_ERR_INVALID_ARG, "step is NULL");
  int64_t total = 0;
  for (int64_t i = 0; i < a->count; ++i) {
    const gemm_adamw_tensor_t& t = a->tensors[i];
    const long long at = i;
    if (t.numel < 0 || t.numel > (int64_t{1} << 40)) return ops_fail(GEMM_ERR_INVALID_ARG, "tensor %lld: numel out of range", at);
    total += padded(t.numel);
    if (t.param_type < GEMM_IN_F16 || t.param_type > GEMM_IN_F32 || t.grad_type < GEMM_IN_F16 || t.grad_type > GEMM_IN_F32)
      return ops_fail(GEMM_ERR_INVALID_ARG, "tensor %lld: type out of range", at);
    if (t.copy && t.copy_type != GEMM_IN_F16 && t.copy_type != GEMM_IN_BF16)
      return ops_fail(GEMM_ERR_INVALID_ARG, "tensor %lld: copy_type must be fp16 or bf16", at);
    if (t.numel > 0 && (!t.param || !t.grad)) return ops_fail(GEMM_ERR_INVALID_ARG, "tensor %lld: param or grad is NULL", at);
    if ((reinterpret_cast<uintptr_t>(t.param) & (t.param_type == GEMM_IN_F32 ? 3 : 1)) ||
        (reinterpret_cast<uintptr_t>(t.grad) & (t.grad_type == GEMM_IN_F32 ? 3 : 1)) ||
        (reinterpret_cast<uintptr_t>(t.copy) & 1))
      return ops_fail(GEMM_ERR_INVALID_ARG, "tensor %lld is not aligned to its elements", at);
  }
  if (total > kBlock * kOpsMaxDim) return ops_fail(GEMM_ERR_INVALID_ARG, "more than 2^39 elements");
  if (a->state_elements != total)
    return ops_fail(GEMM_ERR_INVALID_ARG, "state buffers of %lld elements, %lld needed", (long long)a->state_elements,
                    (long long)total);
  if (total > 0) {
    if (!a->exp_avg || !a->exp_avg_sq || (a->bits == 8 && !a->scales)) return ops_fail(GEMM_ERR_INVALID_ARG, "a state is NULL");
    if ((reinterpret_cast<uintptr_t>(a->exp_avg) | reinterpret_cast<uintptr_t>(a->exp_avg_sq)) & 15u)
      return ops_fail(GEMM_ERR_INVALID_ARG, "the states must be 16-byte aligned");
  }
  if ((reinterpret_cast<uintptr_t>(a->step) & 7u) || (reinterpret_cast<uintptr_t>(a->scales) & 3u) ||
      (reinterpret_cast<uintptr_t>(a->lr_device) & 3u) || (reinterpret_cast<uintptr_t>(a->scale) & 3u))
    return ops_fail(GEMM_ERR_INVALID_ARG, "step, scales, lr_device or scale is not aligned to its elements");
  return GEMM_OK;
}

// What is written may be nothing else that is read or written: sorted by
// address, a written range ends before the next one begins.
gemm_status_t check_overlap(const gemm_adamw_args_t* a) {
  struct Range {
    uintptr_t first, end;
    bool written;
  };
  std::vector<Range> ranges;
  ranges.reserve(static_cast<size_t>(3 * a->count + 6));
  auto add = [&](const void* p, size_t bytes, bool written) {
    if (p && bytes) ranges.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, written});
  };
  int64_t total = 0;
  for (int64_t i = 0; i < a->count; ++i) {
    const gemm_adamw_tensor_t& t = a->tensors[i];
    const size_t n = static_cast<size_t>(t.numel);
    add(t.param, n * (t.param_type == GEMM_IN_F32 ? 4 : 2), true);
    add(t.grad, n * (t.grad_type == GEMM_IN_F32 ? 4 : 2), false);
    add(t.copy, n * 2, true);
    total += padded(t.numel);
  }
  const size_t n = static_cast<size_t>(total);
  add(a->exp_avg, n * (a->bits == 32 ? 4 : 1), true);
  add(a->exp_avg_sq, n * (a->bits == 32 ? 4 : 1), true);
  add(a->bits == 8 ? a->scales : nullptr, n / kBlock * 8, true);
  add(a->step, 8, true);
  add(a->lr_device, 4, false);
  add(a->scale, 4, false);
  std::sort(ranges.begin(), ranges.end(), [](const Range& x, const Range& y) { return x.first < y.first; });
  uintptr_t read_end = 0, write_end = 0;
  for (const Range& r : ranges) {
    if (r.first < write_end || (r.written && r.first < read_end))
      return ops_fail(GEMM_ERR_INVALID_ARG, "a parameter, copy or state overlaps another tensor of the call");
    uintptr_t& end = r.written ? write_end : read_end;
    end = std::max(end, r.end);
  }
  return GEMM_OK;
}

template <int kBits, int kTensors>
cudaError_t run(const gemm_ops* ops, const gemm_adamw_args_t* a, int64_t first, int64_t count, int64_t state, int64_t total,
                cudaStream_t stream) {
  Job<kTensors> job;
  job.count = 0;
  // Chunks of eight blocks (one a warp), longer ones where there are many: a
  // chunk's first loads are waited for.
  uint64_t blocks = 0, chunks = 0;
  for (int64_t i = first; i < first + count; ++i) blocks += static_cast<uint64_t>(padded(a->tensors[i].numel) / kBlock);
  const uint64_t side_by_side = static_cast<uint64_t>(ops->sm_count) * (kBits == 8 ? kOcc8 : kOcc32);
  job.chunk = static_cast<uint32_t>(kWarps * std::max<uint64_t>(1, std::min<uint64_t>(kBits == 8 ? kMostEach8 : kMostEach32, blocks / (kWarps * 4 * side_by_side))));
  for (int64_t i = first; i < first + count; ++i) {
    const gemm_adamw_tensor_t& t = a->tensors[i];
    if (t.numel == 0) continue;
    Entry& e = job.entry[job.count++];
    e.param = t.param;
    e.grad = t.grad;
    e.copy = t.copy;
    e.numel = t.numel;
    e.state = state;
    e.first_chunk = static_cast<uint32_t>(chunks);
    e.kinds = static_cast<uint32_t>(t.param_type) | static_cast<uint32_t>(t.grad_type) << 2 |
              (t.copy ? static_cast<uint32_t>(t.copy_type) : kNoCopy) << 4;
    if (((reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad) | reinterpret_cast<uintptr_t>(t.copy)) & 15u) == 0)
      e.kinds |= kVectors;
    e.decay = t.weight_decay;
    state += padded(t.numel);
    chunks += (static_cast<uint64_t>(padded(t.numel) / kBlock) + job.chunk - 1) / job.chunk;
  }
  if (job.count == 0) return cudaSuccess;
  job.exp_avg = a->exp_avg;
  job.exp_avg_sq = a->exp_avg_sq;
  job.scales = a->scales;
  job.scale_step = total / kBlock;
  job.step = a->step;
  job.lr_device = a->lr_device;
  job.scale = a->scale;
  job.lr = static_cast<float>(a->lr);
  job.beta1 = static_cast<float>(a->beta1);
  job.beta2 = static_cast<float>(a->beta2);
  job.one_less1 = static_cast<float>(1.0 - a->beta1);
  job.one_less2 = static_cast<float>(1.0 - a->beta2);
  job.ln_beta1 = static_cast<float>(std::log(a->beta1));  // beta 0: -inf, and beta^t = 0
  job.ln_beta2 = static_cast<float>(std::log(a->beta2));
  job.eps = static_cast<float>(a->eps);
  job.one = 1.0f;
  return launch(adamw_kernel<kBits, kTensors>, static_cast<unsigned>(chunks), kThreads, Ring<kBits>::kBytes, stream, job);
}

}  // namespace

namespace spgemm {

cudaError_t adamw_set_smem() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel, size_t bytes) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  };
  set(adamw_kernel<32, kFewTensors>, Ring<32>::kBytes);
  set(adamw_kernel<32, kMostTensors>, Ring<32>::kBytes);
  set(adamw_kernel<8, kFewTensors>, Ring<8>::kBytes);
  set(adamw_kernel<8, kMostTensors>, Ring<8>::kBytes);
  return e;
}

}  // namespace spgemm

extern "C" {

int64_t gemm_adamw_state_elements(const gemm_adamw_tensor_t* tensors, int64_t count) {
  int64_t n = 0;
  for (int64_t i = 0; tensors && i < count; ++i)
    if (tensors[i].numel > 0) n += padded(tensors[i].numel);
  return n;
}

gemm_status_t gemm_adamw(gemm_ops_t* ops, const gemm_adamw_args_t* args, void* stream_handle) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops) return ops_fail(GEMM_ERR_INVALID_ARG, "ops is NULL");
  gemm_status_t st = check(args);
  if (st != GEMM_OK) return st;
  try {
    st = check_overlap(args);
  } catch (...) {  // the sorted list's memory
    return ops_fail(GEMM_ERR_INVALID_ARG, "out of host memory");
  }
  if (st != GEMM_OK) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  const int64_t total = gemm_adamw_state_elements(args->tensors, args->count);
  int64_t state = 0, done = 0;
  cudaError_t e = cudaSuccess;
  for (int64_t first = 0; first < args->count && done < total && e == cudaSuccess; first += kMostTensors) {
    const int64_t count = std::min<int64_t>(kMostTensors, args->count - first);
    const bool few = count <= kFewTensors;
    done += gemm_adamw_state_elements(args->tensors + first, count);
    if (args->bits == 32)
      e = few ? run<32, kFewTensors>(ops, args, first, count, state, total, stream)
              : run<32, kMostTensors>(ops, args, first, count, state, total, stream);
    else
      e = few ? run<8, kFewTensors>(ops, args, first, count, state, total, stream)
              : run<8, kMostTensors>(ops, args, first, count, state, total, stream);
    state = done;
  }
  if (e != cudaSuccess) return ops_cuda_fail(e, "AdamW launch");
  e = launch(count_kernel, 1, 1, 0, stream, args->step);
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "AdamW step count launch");
}

}  // extern "C"
