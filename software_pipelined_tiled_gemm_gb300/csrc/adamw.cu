// adamw.cu -- the AdamW step of many tensors, with states in fp32 or in 8 bits.
//
// Bound by memory: parameter and states are read and written, the gradient
// read and the copy written, each once.  All tensors go in one launch (of up
// to kMostTensors): their table travels with the kernel's arguments, so
// nothing is copied to the device before it and a captured call keeps it.
//
// The states of 256 neighbouring elements are a block; a warp takes a block at
// a time, a lane eight elements, so a block's largest magnitude takes one
// reduction instruction and no shared memory.  The elements of a lane lie
// side by side where the tensor's addresses allow 16-byte vectors, and are
// read one by one elsewhere and in a tensor's last block.
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
#include "ptx.cuh"

using namespace spgemm;

namespace {

constexpr int kBlock = GEMM_ADAMW_BLOCK;
constexpr int kEach = 8;                 // elements of a lane: 32 lanes, one block
constexpr int kThreads = 256, kWarps = kThreads / 32;
// Types of an entry: parameter, gradient, copy (3: none), two bits each, and
// whether its addresses allow vectors.
constexpr uint32_t kNoCopy = 3u, kVectors = 1u << 6;

struct Entry {
  void* param;
  const void* grad;
  void* copy;
  int64_t numel;
  int64_t state;         // first element of the states
  uint32_t first_block;  // of this launch
  uint32_t kinds;
  float decay;           // weight decay
};

// Tables of two sizes: a launch's arguments cost time to send (a table of 512
// entries 3 us more than one of 32).
constexpr int kFewTensors = 32, kMostTensors = 512;
template <int kTensors>
struct Job {
  Entry entry[kTensors];
  int count;
  uint32_t blocks;
  void* exp_avg;
  void* exp_avg_sq;
  float* scales;          // of exp_avg, then (scale_step later) of exp_avg_sq
  int64_t scale_step;
  const int64_t* step;
  const float* lr_device;
  const float* scale;
  float lr, beta1, beta2, one_less1, one_less2, ln_beta1, ln_beta2, eps;
};

// Eight fp32 values from fp16, bf16 or fp32 at p.
__device__ __forceinline__ void load8(const void* p, uint32_t kind, float (&v)[kEach]) {
  if (kind == GEMM_IN_F32) {
    const float4 a = __ldcs(static_cast<const float4*>(p)), b = __ldcs(static_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
  const uint4 raw = __ldcs(static_cast<const uint4*>(p));
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = kind == GEMM_IN_BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]))
                                          : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void store8(void* p, uint32_t kind, const float (&v)[kEach]) {
  if (kind == GEMM_IN_F32) {
    __stcs(static_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(static_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kind == GEMM_IN_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      memcpy(&w[i], &h, 4);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
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

// The e4m3 code of y in [0, 448] rounded down after adding u 2^-20 steps.  A
// normal value's step is 2^20 units of its fp32 bits, so the sum of the bits
// and u carries into the next code by itself; below 2^-6 the step is 2^-9.
__device__ __forceinline__ uint32_t e4m3_dithered(float y, uint32_t u) {
  if (y < 0.015625f) return static_cast<uint32_t>(fmaf(y, 512.0f, static_cast<float>(u) * 9.5367431640625e-07f));
  return ((__float_as_uint(y) + u) >> 20) - 960u;
}

// Largest of non-negative floats over the warp, NaN above all: their order is that of their bits.
__device__ __forceinline__ float warp_max(float v) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v))); }

// Entry of block b: the last whose first block is not after it.
template <typename J>
__device__ __forceinline__ int find_entry(const J& job, uint32_t b) {
  int lo = 0, hi = job.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (job.entry[mid].first_block <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int kBits, int kTensors>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Job<kTensors> job) {
  const int lane = threadIdx.x & 31;
  const uint32_t b = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (b >= job.blocks) return;
  const Entry& e = job.entry[find_entry(job, b)];
  const int64_t at = static_cast<int64_t>(b - e.first_block) * kBlock + lane * kEach;  // in the tensor
  const int64_t state = e.state + at;
  const uint32_t kp = e.kinds & 3u, kg = (e.kinds >> 2) & 3u, kc = (e.kinds >> 4) & 3u;
  const int left = static_cast<int>(min(static_cast<int64_t>(kEach), e.numel - at));  // may be negative
  // A tensor's last block may end inside: elements that do not exist count as zeros, and
  // so do their states, which are written all the same (they are the buffer's own).
  const bool whole = (e.kinds & kVectors) != 0 && left == kEach;
  const int psize = kp == GEMM_IN_F32 ? 4 : 2, gsize = kg == GEMM_IN_F32 ? 4 : 2;

  float p[kEach], g[kEach], m[kEach], v[kEach];
  if (whole) {
    load8(static_cast<const uint8_t*>(e.param) + at * psize, kp, p);
    load8(static_cast<const uint8_t*>(e.grad) + at * gsize, kg, g);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      p[i] = i < left ? load1(e.param, kp, at + i) : 0.0f;
      g[i] = i < left ? load1(e.grad, kg, at + i) : 0.0f;
    }
  }
  const int64_t scale_at = state / kBlock;
  if constexpr (kBits == 32) {
    load8(static_cast<const float*>(job.exp_avg) + state, GEMM_IN_F32, m);
    load8(static_cast<const float*>(job.exp_avg_sq) + state, GEMM_IN_F32, v);
  } else {
    const uint2 cm = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(job.exp_avg) + state));
    const uint2 cv = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(job.exp_avg_sq) + state));
    const float sm = job.scales[scale_at], sv = job.scales[job.scale_step + scale_at];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t wm = i < 2 ? cm.x : cm.y, wv = i < 2 ? cv.x : cv.y;
      const float2 fm = from_e4m3x2((wm >> (16 * (i & 1))) & 0xffffu), fv = from_e4m3x2((wv >> (16 * (i & 1))) & 0xffffu);
      m[2 * i] = fm.x * sm;
      m[2 * i + 1] = fm.y * sm;
      v[2 * i] = (fv.x * sv) * (fv.x * sv);
      v[2 * i + 1] = (fv.y * sv) * (fv.y * sv);
    }
  }
  // 1 - beta^t = -expm1(t ln beta), which keeps its bits where beta^t is near 1.
  const int64_t t = *job.step + 1;
  const float lr = job.lr_device ? *job.lr_device : job.lr;
  const float factor = job.scale ? *job.scale : 1.0f;
  const float rate = lr / -expm1f(static_cast<float>(t) * job.ln_beta1);
  const float unbias = rsqrtf(-expm1f(static_cast<float>(t) * job.ln_beta2));
  const float decay = lr * e.decay;
  float r[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    g[i] *= factor;
    m[i] = fmaf(job.beta1, m[i], job.one_less1 * g[i]);
    v[i] = fmaf(job.beta2, v[i], job.one_less2 * (g[i] * g[i]));
    r[i] = __fsqrt_rn(v[i]);
    // (The quotient is within 2 units of its last place, and p is larger.)
    p[i] = (p[i] - decay * p[i]) - rate * __fdividef(m[i], fmaf(r[i], unbias, job.eps));
  }
  if (whole) {
    store8(static_cast<uint8_t*>(e.param) + at * psize, kp, p);
    if (kc != kNoCopy) store8(static_cast<uint16_t*>(e.copy) + at, kc, p);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < left) {
        store1(e.param, kp, at + i, p[i]);
        if (kc != kNoCopy) store1(e.copy, kc, at + i, p[i]);
      } else {
        m[i] = v[i] = r[i] = 0.0f;
      }
  }
  if constexpr (kBits == 32) {
    store8(static_cast<float*>(job.exp_avg) + state, GEMM_IN_F32, m);
    store8(static_cast<float*>(job.exp_avg_sq) + state, GEMM_IN_F32, v);
  } else {
    float top_m = 0.0f, top_r = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      top_m = __uint_as_float(max(__float_as_uint(top_m), __float_as_uint(fabsf(m[i]))));
      top_r = __uint_as_float(max(__float_as_uint(top_r), __float_as_uint(r[i])));
    }
    top_m = warp_max(top_m);
    top_r = warp_max(top_r);
    // (A NaN stays one: it is larger than 2^-120 as bits.)
    const uint32_t least = 0x03800000u;  // 2^-120
    const float sm = __uint_as_float(max(__float_as_uint(__fdiv_rn(top_m, 448.0f)), least));
    const float sv = __uint_as_float(max(__float_as_uint(__fdiv_rn(top_r, 448.0f)), least));
    const float im = __frcp_rn(sm), iv = __frcp_rn(sv);
    const uint32_t lost = sv <= 3.4028235e38f ? 0u : 0x7fu;  // an infinite or NaN root: all of the block NaN
    uint32_t wm[2] = {0u, 0u}, wv[2] = {0u, 0u};
    const uint32_t dither = static_cast<uint32_t>(state) * 0xC13FA9A9u + static_cast<uint32_t>(t) * 0x91E10DA5u;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const float y = fminf(r[i] * iv, 448.0f);
      uint32_t code = e4m3_dithered(y, (dither + static_cast<uint32_t>(i) * 0xC13FA9A9u) >> 12);
      if (r[i] > 0.0f) code = max(code, 1u);
      wv[i >> 2] |= (code | lost) << (8 * (i & 3));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) wm[i >> 1] |= e4m3x2(m[2 * i] * im, m[2 * i + 1] * im) << (16 * (i & 1));
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(job.exp_avg) + state), make_uint2(wm[0], wm[1]));
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(job.exp_avg_sq) + state), make_uint2(wv[0], wv[1]));
    if (lane == 0) {
      job.scales[scale_at] = sm;
      job.scales[job.scale_step + scale_at] = sv;
    }
  }
}

__global__ void count_kernel(int64_t* step) { *step += 1; }

int64_t padded(int64_t n) { return (n + kBlock - 1) / kBlock * kBlock; }

gemm_status_t check(const gemm_adamw_args_t* a) {
  if (!a) return ops_fail(GEMM_ERR_INVALID_ARG, "args is NULL");
  if (a->count < 0 || (a->count > 0 && !a->tensors)) return ops_fail(GEMM_ERR_INVALID_ARG, "tensors is NULL or count < 0");
  if (a->bits != 32 && a->bits != 8) return ops_fail(GEMM_ERR_INVALID_ARG, "bits %d not in {8, 32}", a->bits);
  if (!(a->beta1 >= 0.0 && a->beta1 < 1.0 && a->beta2 >= 0.0 && a->beta2 < 1.0))
    return ops_fail(GEMM_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
  if (!(a->eps >= 0.0)) return ops_fail(GEMM_ERR_INVALID_ARG, "eps must be at least 0");
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
cudaError_t run(const gemm_adamw_args_t* a, int64_t first, int64_t count, int64_t state, int64_t total, cudaStream_t stream) {
  Job<kTensors> job;
  job.count = 0;
  uint64_t blocks = 0;
  for (int64_t i = first; i < first + count; ++i) {
    const gemm_adamw_tensor_t& t = a->tensors[i];
    if (t.numel == 0) continue;
    Entry& e = job.entry[job.count++];
    e.param = t.param;
    e.grad = t.grad;
    e.copy = t.copy;
    e.numel = t.numel;
    e.state = state;
    e.first_block = static_cast<uint32_t>(blocks);
    e.kinds = static_cast<uint32_t>(t.param_type) | static_cast<uint32_t>(t.grad_type) << 2 |
              (t.copy ? static_cast<uint32_t>(t.copy_type) : kNoCopy) << 4;
    if (((reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad) | reinterpret_cast<uintptr_t>(t.copy)) & 15u) == 0)
      e.kinds |= kVectors;
    e.decay = t.weight_decay;
    state += padded(t.numel);
    blocks += static_cast<uint64_t>(padded(t.numel) / kBlock);
  }
  if (job.count == 0) return cudaSuccess;
  job.blocks = static_cast<uint32_t>(blocks);
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
  adamw_kernel<kBits, kTensors><<<static_cast<unsigned>((blocks + kWarps - 1) / kWarps), kThreads, 0, stream>>>(job);
  return cudaGetLastError();
}

}  // namespace

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
  int64_t state = 0;
  cudaError_t e = cudaSuccess;
  for (int64_t first = 0; first < args->count && e == cudaSuccess; first += kMostTensors) {
    const int64_t count = std::min<int64_t>(kMostTensors, args->count - first);
    const bool few = count <= kFewTensors;
    if (args->bits == 32)
      e = few ? run<32, kFewTensors>(args, first, count, state, total, stream)
              : run<32, kMostTensors>(args, first, count, state, total, stream);
    else
      e = few ? run<8, kFewTensors>(args, first, count, state, total, stream)
              : run<8, kMostTensors>(args, first, count, state, total, stream);
    state += gemm_adamw_state_elements(args->tensors + first, count);
  }
  if (e != cudaSuccess) return ops_cuda_fail(e, "AdamW launch");
  count_kernel<<<1, 1, 0, stream>>>(args->step);
  e = cudaGetLastError();
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "AdamW step count launch");
}

}  // extern "C"
