// layer_norm.cu -- layer norm over the rows of a matrix, and its gradients.
//
// Bound by memory: the forward pass reads x and writes y, the backward pass
// reads x and dy and writes dx.  A row belongs to a group of threads, a warp
// or a block, each thread holding the same columns of every row it meets:
//
//   mean  = sum x / n, then d = x - mean, low = sum d / n,
//   var   = sum d^2 / n - low^2,  h = (d - low) rstd.
//
// The second sum costs no pass of its own and takes out what the rounding of
// the mean to fp32 left in the differences, so that a row far from zero loses
// nothing but its own bits; the backward pass gets both parts of the mean.
// Products with 1 / n are summed instead of values, so no sum overflows; a row
// whose squares do is summed again with differences scaled by 2^-64.
//
// Groups loop over rows.  Where rows are 16-byte aligned a thread copies its
// own vectors of the next rows to shared memory asynchronously (nobody else
// reads them, so no barrier is needed), which keeps kAhead rows of every group
// on their way while one is reduced.  Rows that are not aligned are read
// element by element, lanes side by side.
//
// The weights' gradients: a thread sums its columns over its rows in fp32
// registers; each block leaves one partial, and a second kernel adds those in
// block order.  The sums repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "ops_internal.h"
#include "ptx.cuh"

using namespace spgemm;

namespace {

constexpr int kAhead = 3;        // rows of a group on their way or in work, at most
constexpr int kWarpRows = 8;     // rows a block works on where a warp has one each
constexpr int kFwdItems = 32;    // columns of a thread at most
constexpr int kBwdItems = 16;    // the same where it keeps two sums of each
constexpr size_t kStaticBytes = 1024;  // of shared memory, at least what the kernels declare
constexpr int kMaxCols = 1024 * kFwdItems;  // above it rows are read again from memory

struct Args {
  const void* x;
  int64_t ldx;
  const void* dy;
  int64_t lddy;
  const void* weight;
  const void* bias;
  void* out;            // y or dx, dense
  float* stats;         // 3 x rows
  float* partial;       // backward: blocks x 2 x cols, or nullptr
  int64_t rows;
  int cols;
  float inv;            // 1 / cols
  float eps;
  int ahead;            // rows of a group on their way or in work
};

template <typename T>
__device__ __forceinline__ float to_float(T v) {
  if constexpr (std::is_same_v<T, __half>) return __half2float(v);
  if constexpr (std::is_same_v<T, __nv_bfloat16>) return __bfloat162float(v);
  if constexpr (std::is_same_v<T, float>) return v;
}
template <typename T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
  if constexpr (std::is_same_v<T, __nv_bfloat16>) return __float2bfloat16_rn(v);
  if constexpr (std::is_same_v<T, float>) return v;
}

// kVec neighbouring elements: one 16-byte vector of T, or (1) one element.
template <typename T, int kVec>
struct alignas(kVec == 1 ? sizeof(T) : 16) Vec {
  T v[kVec];
};

// Weights of the same columns, of T or fp32.
template <typename W, int kVec>
__device__ __forceinline__ void load_weights(const void* base, int col, float (&out)[kVec], float otherwise) {
  if (base == nullptr) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) out[j] = otherwise;
    return;
  }
  const W* p = static_cast<const W*>(base) + col;
  if constexpr (kVec == 1) {
    out[0] = to_float(__ldg(p));
  } else {
    constexpr int kEach = 16 / sizeof(W) < kVec ? 16 / sizeof(W) : kVec;
#pragma unroll
    for (int j = 0; j < kVec; j += kEach) {
      const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p + j));
      Vec<W, kEach> w;
      memcpy(&w, &raw, 16);
#pragma unroll
      for (int i = 0; i < kEach; ++i) out[j + i] = to_float(w.v[i]);
    }
  }
}

__device__ __forceinline__ void copy_async16(void* smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(smem)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the newest ahead - 1 groups have landed.
__device__ __forceinline__ void copy_async_wait(int ahead) {
  static_assert(kAhead == 3);
  if (ahead == 3)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (ahead == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Sums of two values over the group, the same in every thread: lanes first,
// then the warps in order.  `red`: 2 x warps x 2 floats, used in turn.
template <int kGroup>
__device__ __forceinline__ float2 group_sum(float a, float b, float* red, int& turn) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  if constexpr (kGroup > 32) {
    constexpr int kWarps = kGroup / 32;
    float2* mine = reinterpret_cast<float2*>(red) + turn * kWarps;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 v = mine[w];
      a += v.x;
      b += v.y;
    }
  }
  return make_float2(a, b);
}

// 1 / sqrt(sum / n + eps) and the mean's lower part, from the sums of d and
// d^2 over n; `again` gives the sum of (2^-64 d)^2 / n.
template <typename F>
__device__ __forceinline__ float row_rstd(float low, float squares, float eps, F again) {
  float var = fmaxf(squares - low * low, 0.0f);
  if (squares != squares) return squares;  // NaN stays NaN (fmaxf would drop it)
  if (squares > 3e38f) {  // the same in all threads of the group
    const float s = again();
    return s > 3e38f ? __int_as_float(0x7fc00000) : rsqrtf(s) * 5.421010862427522e-20f;  // 2^-64
  }
  return rsqrtf(var + eps);
}

template <typename T, typename W, int kVec, int kGroup, int kBlocks>
__global__ void __launch_bounds__(kGroup == 32 ? 32 * kWarpRows : kGroup, kBlocks) forward_kernel(const Args p) {
  constexpr int kItems = kFwdItems / kVec;  // vectors of a thread at most
  constexpr int kWarps = kGroup / 32;
  using V = Vec<T, kVec>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[kGroup > 32 ? 4 * kWarps : 1];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  const int tid = kGroup == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int groups = kGroup == 32 ? kWarpRows : 1, group = kGroup == 32 ? threadIdx.x >> 5 : 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int vecs = p.cols / kVec;                       // of a row
  const int items = (vecs + kGroup - 1) / kGroup;       // of a thread
  V* mine = reinterpret_cast<V*>(ring) + static_cast<size_t>(group) * p.ahead * items * kGroup + tid;
  const T* x = static_cast<const T*>(p.x);
  int turn = 0;

  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
  auto fetch = [&](int64_t r, int slot) {
    if (r < p.rows) {
      const T* src = x + r * p.ldx;
      for (int i = 0; i < items; ++i)
        if (tid + i * kGroup < vecs) copy_async16(mine + (slot * items + i) * kGroup, src + (tid + i * kGroup) * kVec);
    }
    copy_async_commit();
  };
  if constexpr (kVec > 1)
    for (int s = 0; s < p.ahead - 1; ++s) fetch(row + s * step, s);

  for (int slot = 0; row < p.rows; row += step) {
    float v[kItems * kVec];
    if constexpr (kVec > 1) {
      fetch(row + (p.ahead - 1) * step, slot == 0 ? p.ahead - 1 : slot - 1);
      copy_async_wait(p.ahead);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        V u;
        if (tid + i * kGroup < vecs) u = mine[(slot * items + i) * kGroup];
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[i * kVec + j] = tid + i * kGroup < vecs ? to_float(u.v[j]) : 0.0f;
      }
      slot = slot == p.ahead - 1 ? 0 : slot + 1;
    } else {
      const T* src = x + row * p.ldx;
#pragma unroll
      for (int i = 0; i < kItems; ++i) v[i] = tid + i * kGroup < vecs ? to_float(src[tid + i * kGroup]) : 0.0f;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kItems * kVec; ++i) sum = fmaf(v[i], p.inv, sum);
    const float mean = group_sum<kGroup>(sum, 0.0f, red, turn).x;
    float low = 0.0f, squares = 0.0f;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (tid + i * kGroup < vecs) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          float& d = v[i * kVec + j];
          d -= mean;
          low = fmaf(d, p.inv, low);
          squares = fmaf(d * p.inv, d, squares);
        }
      }
    const float2 both = group_sum<kGroup>(low, squares, red, turn);
    low = both.x;
    const float rstd = row_rstd(low, both.y, p.eps, [&]() {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kItems * kVec; ++i) {
        const float d = v[i] * 5.421010862427522e-20f;
        if (tid + (i / kVec) * kGroup < vecs) s = fmaf(d * p.inv, d, s);
      }
      return group_sum<kGroup>(s, 0.0f, red, turn).x;
    });
    if (p.stats != nullptr && tid == 0) {
      p.stats[row] = mean;
      p.stats[p.rows + row] = low;
      p.stats[2 * p.rows + row] = rstd;
    }
    T* out = static_cast<T*>(p.out) + row * p.cols;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int at = tid + i * kGroup;
      if (at < vecs) {
        float w[kVec], b[kVec];
        load_weights<W, kVec>(p.weight, at * kVec, w, 1.0f);
        load_weights<W, kVec>(p.bias, at * kVec, b, 0.0f);
        V u;
#pragma unroll
        for (int j = 0; j < kVec; ++j) u.v[j] = from_float<T>(fmaf((v[i * kVec + j] - low) * rstd, w[j], b[j]));
        *reinterpret_cast<V*>(out + at * kVec) = u;
      }
    }
  }
}

// Rows of more columns than a block holds: read three times, the second and
// third mostly from L2.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) forward_long_kernel(const Args p) {
  __shared__ float red[4 * 32];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    float sum = 0.0f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) sum = fmaf(to_float(x[c]), p.inv, sum);
    const float mean = group_sum<1024>(sum, 0.0f, red, turn).x;
    float low = 0.0f, squares = 0.0f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float d = to_float(x[c]) - mean;
      low = fmaf(d, p.inv, low);
      squares = fmaf(d * p.inv, d, squares);
    }
    const float2 both = group_sum<1024>(low, squares, red, turn);
    low = both.x;
    const float rstd = row_rstd(low, both.y, p.eps, [&]() {
      float s = 0.0f;
      for (int c = threadIdx.x; c < p.cols; c += 1024) {
        const float d = (to_float(x[c]) - mean) * 5.421010862427522e-20f;
        s = fmaf(d * p.inv, d, s);
      }
      return group_sum<1024>(s, 0.0f, red, turn).x;
    });
    if (p.stats != nullptr && threadIdx.x == 0) {
      p.stats[row] = mean;
      p.stats[p.rows + row] = low;
      p.stats[2 * p.rows + row] = rstd;
    }
    T* out = static_cast<T*>(p.out) + row * p.cols;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      float w[1], b[1];
      load_weights<W, 1>(p.weight, c, w, 1.0f);
      load_weights<W, 1>(p.bias, c, b, 0.0f);
      out[c] = from_float<T>(fmaf((to_float(x[c]) - mean - low) * rstd, w[0], b[0]));
    }
  }
}

template <typename T, typename W, int kVec, int kGroup, int kItemCols, int kBlocks>
__global__ void __launch_bounds__(kGroup == 32 ? 32 * kWarpRows : kGroup, kBlocks) backward_kernel(const Args p) {
  constexpr int kItems = kItemCols / kVec;
  constexpr int kWarps = kGroup / 32;
  using V = Vec<T, kVec>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[kGroup > 32 ? 4 * kWarps : 1];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  const int tid = kGroup == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int groups = kGroup == 32 ? kWarpRows : 1, group = kGroup == 32 ? threadIdx.x >> 5 : 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int vecs = p.cols / kVec;
  const int items = (vecs + kGroup - 1) / kGroup;
  // [slot][x, dy][item][thread]
  V* mine = reinterpret_cast<V*>(ring) + static_cast<size_t>(group) * p.ahead * 2 * items * kGroup + tid;
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  int turn = 0;
  float dw[kItems * kVec], db[kItems * kVec];
#pragma unroll
  for (int i = 0; i < kItems * kVec; ++i) dw[i] = db[i] = 0.0f;

  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
  auto fetch = [&](int64_t r, int slot) {
    if (r < p.rows) {
      const T* sx = x + r * p.ldx;
      const T* sd = dy + r * p.lddy;
      V* to = mine + slot * 2 * items * kGroup;
      for (int i = 0; i < items; ++i)
        if (tid + i * kGroup < vecs) {
          copy_async16(to + i * kGroup, sx + (tid + i * kGroup) * kVec);
          copy_async16(to + (items + i) * kGroup, sd + (tid + i * kGroup) * kVec);
        }
    }
    copy_async_commit();
  };
  float next_mean = 0.0f, next_low = 0.0f, next_rstd = 0.0f;
  auto fetch_stats = [&](int64_t r) {
    if (r < p.rows) {
      next_mean = __ldg(p.stats + r);
      next_low = __ldg(p.stats + p.rows + r);
      next_rstd = __ldg(p.stats + 2 * p.rows + r);
    }
  };
  if constexpr (kVec > 1)
    for (int s = 0; s < p.ahead - 1; ++s) fetch(row + s * step, s);
  fetch_stats(row);

  for (int slot = 0; row < p.rows; row += step) {
    const float mean = next_mean, low = next_low, rstd = next_rstd;
    fetch_stats(row + step);
    T ex[kVec == 1 ? kItems : 1], ed[kVec == 1 ? kItems : 1];
    if constexpr (kVec > 1) {
      fetch(row + (p.ahead - 1) * step, slot == 0 ? p.ahead - 1 : slot - 1);
      copy_async_wait(p.ahead);
    } else {
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (tid + i * kGroup < vecs) {
          ex[i] = x[row * p.ldx + tid + i * kGroup];
          ed[i] = dy[row * p.lddy + tid + i * kGroup];
        }
    }
    // dy, h and g of this thread's vector i; both passes over the row take them from
    // shared memory (or the elements' registers), which costs less than holding them.
    auto values = [&](int i, float (&d)[kVec], float (&h)[kVec], float (&g)[kVec]) {
      V ux, ud;
      if constexpr (kVec > 1) {
        ux = mine[(slot * 2 * items + i) * kGroup];
        ud = mine[(slot * 2 * items + items + i) * kGroup];
      } else {
        ux.v[0] = ex[i];
        ud.v[0] = ed[i];
      }
      load_weights<W, kVec>(p.weight, (tid + i * kGroup) * kVec, g, 1.0f);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        d[j] = to_float(ud.v[j]);
        h[j] = ((to_float(ux.v[j]) - mean) - low) * rstd;
        g[j] *= d[j];
      }
    };
    float gs = 0.0f, ghs = 0.0f;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (tid + i * kGroup < vecs) {
        float d[kVec], h[kVec], g[kVec];
        values(i, d, h, g);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const int k = i * kVec + j;
          dw[k] = fmaf(d[j], h[j], dw[k]);
          db[k] += d[j];
          gs = fmaf(g[j], p.inv, gs);
          ghs = fmaf(g[j] * p.inv, h[j], ghs);
        }
      }
    if (p.out != nullptr) {
      const float2 means = group_sum<kGroup>(gs, ghs, red, turn);
      T* out = static_cast<T*>(p.out) + row * p.cols;
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (tid + i * kGroup < vecs) {
          float d[kVec], h[kVec], g[kVec];
          values(i, d, h, g);
          V u;
#pragma unroll
          for (int j = 0; j < kVec; ++j) u.v[j] = from_float<T>(rstd * (g[j] - means.x - h[j] * means.y));
          *reinterpret_cast<V*>(out + (tid + i * kGroup) * kVec) = u;
        }
    }
    slot = slot == p.ahead - 1 ? 0 : slot + 1;
  }

  if (p.partial == nullptr) return;
  float* to = p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.cols;
  if constexpr (kGroup == 32) {
    // The block's warps one after another, each adding to the sum before it.
    float* sums = reinterpret_cast<float*>(ring);
    copy_async_wait(1);
    for (int turn_of = 0; turn_of < kWarpRows; ++turn_of) {
      __syncthreads();
      if (turn_of != group) continue;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int at = tid + i * kGroup;
        if (at < vecs)
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            float* s = sums + at * kVec + j;
            s[0] = group == 0 ? dw[i * kVec + j] : s[0] + dw[i * kVec + j];
            s[p.cols] = group == 0 ? db[i * kVec + j] : s[p.cols] + db[i * kVec + j];
          }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.cols; c += 32 * kWarpRows) to[c] = sums[c];
  } else {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int at = tid + i * kGroup;
      if (at < vecs)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          to[at * kVec + j] = dw[i * kVec + j];
          to[p.cols + at * kVec + j] = db[i * kVec + j];
        }
    }
  }
}

// Rows of more columns than a block holds: a block sums a share of the rows
// into its own partial in memory.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) backward_long_kernel(const Args p) {
  __shared__ float red[4 * 32];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  int turn = 0;
  float* to = p.partial ? p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.cols : nullptr;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const float mean = __ldg(p.stats + row), low = __ldg(p.stats + p.rows + row);
    const float rstd = __ldg(p.stats + 2 * p.rows + row);
    float gs = 0.0f, ghs = 0.0f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float d = to_float(dy[c]), h = ((to_float(x[c]) - mean) - low) * rstd;
      float w[1];
      load_weights<W, 1>(p.weight, c, w, 1.0f);
      gs = fmaf(d * w[0], p.inv, gs);
      ghs = fmaf(d * w[0] * p.inv, h, ghs);
      if (to) {  // the thread's own columns
        const bool first = row == blockIdx.x;
        to[c] = first ? d * h : to[c] + d * h;
        to[p.cols + c] = first ? d : to[p.cols + c] + d;
      }
    }
    if (p.out == nullptr) continue;
    const float2 means = group_sum<1024>(gs, ghs, red, turn);
    T* out = static_cast<T*>(p.out) + row * p.cols;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      float w[1];
      load_weights<W, 1>(p.weight, c, w, 1.0f);
      const float d = to_float(dy[c]), h = ((to_float(x[c]) - mean) - low) * rstd;
      out[c] = from_float<T>(rstd * (d * w[0] - means.x - h * means.y));
    }
  }
}

// The blocks' partials in order: 32 columns a block, its warps sharing the
// partials, then the warps in order.
constexpr int kSumThreads = 1024;
template <typename W>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const float* partial, int blocks, int cols, W* dweight, W* dbias) {
  __shared__ float sums[32][33];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  W* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int each = (blocks + 31) / 32;
  const float* src = partial + static_cast<size_t>(blockIdx.y) * cols + col;
  float s = 0.0f;
  if (col < cols) {
    const int end = min(blocks, (warp + 1) * each);
#pragma unroll 4
    for (int b = warp * each; b < end; ++b) s += __ldcg(src + static_cast<size_t>(b) * 2 * cols);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= cols) return;
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < 32; ++w) total += sums[w][lane];
  out[col] = from_float<W>(total);
}

gemm_status_t check(const gemm_layer_norm_args_t* a, bool backward) {
  if (!a) return ops_fail(GEMM_ERR_INVALID_ARG, "args is NULL");
  if (a->rows < 0 || a->cols < 1)
    return ops_fail(GEMM_ERR_INVALID_ARG, "rows %lld < 0 or cols %lld < 1", (long long)a->rows, (long long)a->cols);
  if (a->cols > kOpsMaxDim / 4 || a->rows > (int64_t{1} << 40))
    return ops_fail(GEMM_ERR_INVALID_ARG, "cols above 2^29 or rows above 2^40");
  if (a->dtype < GEMM_IN_F16 || a->dtype > GEMM_IN_F32)
    return ops_fail(GEMM_ERR_INVALID_ARG, "dtype %d out of range", static_cast<int>(a->dtype));
  if (a->weight_dtype != a->dtype && a->weight_dtype != GEMM_IN_F32)
    return ops_fail(GEMM_ERR_INVALID_ARG, "weight_dtype must be dtype or fp32");
  if (a->ldx < a->cols) return ops_fail(GEMM_ERR_INVALID_ARG, "ldx %lld < cols", (long long)a->ldx);
  if (backward && a->lddy < a->cols) return ops_fail(GEMM_ERR_INVALID_ARG, "lddy %lld < cols", (long long)a->lddy);
  if (!backward && !(a->eps >= 0.0f)) return ops_fail(GEMM_ERR_INVALID_ARG, "eps must be at least 0");
  if (a->rows > 0) {
    if (!a->x) return ops_fail(GEMM_ERR_INVALID_ARG, "x is NULL");
    if (backward && (!a->dy || !a->stats)) return ops_fail(GEMM_ERR_INVALID_ARG, "dy or stats is NULL");
    if (!backward && !a->y) return ops_fail(GEMM_ERR_INVALID_ARG, "y is NULL");
  }
  const uintptr_t size = a->dtype == GEMM_IN_F32 ? 4 : 2, wsize = a->weight_dtype == GEMM_IN_F32 ? 4 : 2;
  const void* ptrs[] = {a->x, a->y, a->dy, a->dx};
  const void* weights[] = {a->weight, a->bias, a->dweight, a->dbias};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & (size - 1))
      return ops_fail(GEMM_ERR_INVALID_ARG, "x, y, dy or dx is not aligned to its elements");
  for (const void* q : weights)
    if (reinterpret_cast<uintptr_t>(q) & (wsize - 1))
      return ops_fail(GEMM_ERR_INVALID_ARG, "weight, bias or a gradient of them is not aligned to its elements");
  if (reinterpret_cast<uintptr_t>(a->stats) & 3u) return ops_fail(GEMM_ERR_INVALID_ARG, "stats is not 4-byte aligned");
  return GEMM_OK;
}

// Outputs against inputs and each other.
gemm_status_t check_overlap(const gemm_layer_norm_args_t* a, bool backward, const void* ws, size_t ws_bytes) {
  const size_t size = a->dtype == GEMM_IN_F32 ? 4 : 2, wsize = a->weight_dtype == GEMM_IN_F32 ? 4 : 2;
  const size_t R = a->rows, C = a->cols;
  struct Range {
    const void* p;
    size_t n;
    const char* name;
  };
  const void* dy = backward ? a->dy : nullptr;
  const Range in[] = {{a->x, R ? ((R - 1) * a->ldx + C) * size : 0, "x"},
                      {dy, R && backward ? ((R - 1) * a->lddy + C) * size : 0, "dy"},
                      {a->weight, C * wsize, "weight"},
                      {backward ? nullptr : a->bias, C * wsize, "bias"},
                      {backward ? a->stats : nullptr, 12 * R, "stats"}};
  const Range out[] = {{backward ? nullptr : a->y, R * C * size, "y"},
                       {backward ? nullptr : a->stats, 12 * R, "stats"},
                       {backward ? a->dx : nullptr, R * C * size, "dx"},
                       {backward ? a->dweight : nullptr, C * wsize, "dweight"},
                       {backward ? a->dbias : nullptr, C * wsize, "dbias"},
                       {ws, ws_bytes, "the workspace"}};
  constexpr int kOut = sizeof(out) / sizeof(out[0]);
  for (int i = 0; i < kOut; ++i) {
    for (const Range& r : in) {
      // A row is read before it is written, by the same threads.
      const bool same = (out[i].p == a->x && r.p == a->x && i == 0 && a->ldx == a->cols) ||
                        (i == 2 && out[i].p == dy && r.p == dy && a->lddy == a->cols);
      if (!same && overlap(out[i].p, out[i].n, r.p, r.n))
        return ops_fail(GEMM_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, r.name);
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return ops_fail(GEMM_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
  }
  return GEMM_OK;
}

bool aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 15u) return false;
  return true;
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Threads that share a row: enough that each has at most `items` columns.
int group_of(int64_t cols, int items) {
  if (cols <= 32 * items) return 32;
  if (cols <= 256 * items) return 256;
  return cols <= 512 * items ? 512 : 1024;
}

// Blocks of a launch, each block's ring and the rows it holds.
struct Shape {
  int threads, blocks, ahead;
  size_t smem;
};

// Bytes that one row of `arrays` arrays takes of a block's ring.
size_t row_bytes(int64_t vecs, int group, int arrays) {
  const int rows = group == 32 ? kWarpRows : 1;
  return static_cast<size_t>(rows) * arrays * ceil_div(vecs, int64_t{group}) * group * 16;
}
size_t most_smem(const gemm_ops* ops) { return ops->smem_optin - kStaticBytes; }

template <int kVec>
Shape shape_of(const gemm_ops* ops, const Args& p, int group, int per_sm, int arrays) {
  const int rows = group == 32 ? kWarpRows : 1;
  const size_t most = most_smem(ops), row = kVec == 1 ? 0 : row_bytes(p.cols / kVec, group, arrays);
  int ahead = kAhead;
  while (ahead > 2 && ahead * row * per_sm > most) --ahead;
  while (ahead > 1 && ahead * row > most) --ahead;
  size_t smem = ahead * row;
  if (arrays == 2 && group == 32) smem = std::max(smem, static_cast<size_t>(p.cols) * 2 * sizeof(float));
  const int64_t blocks = std::min<int64_t>(ceil_div(p.rows, int64_t{rows}), static_cast<int64_t>(ops->sm_count) * per_sm);
  return {group == 32 ? 32 * rows : group, static_cast<int>(blocks), ahead, smem};
}

template <typename T, typename W, int kVec, int kGroup, int kBlocks>
cudaError_t forward_as(const gemm_ops* ops, Args p, cudaStream_t stream) {
  const Shape s = shape_of<kVec>(ops, p, kGroup, kBlocks, 1);
  p.ahead = s.ahead;
  return launch(forward_kernel<T, W, kVec, kGroup, kBlocks>, dim3(s.blocks), s.threads, s.smem, stream, p);
}
template <typename T, typename W, int kVec>
cudaError_t forward_vec(const gemm_ops* ops, const Args& p, cudaStream_t stream) {
  switch (group_of(p.cols, kFwdItems)) {
    case 32: return forward_as<T, W, kVec, 32, 3>(ops, p, stream);
    case 256: return forward_as<T, W, kVec, 256, 3>(ops, p, stream);
    case 512: return forward_as<T, W, kVec, 512, 1>(ops, p, stream);
    default: return forward_as<T, W, kVec, 1024, 1>(ops, p, stream);
  }
}
template <typename T, typename W>
cudaError_t forward(const gemm_ops* ops, const Args& p, bool vec, cudaStream_t stream) {
  if (p.cols > kMaxCols)
    return launch(forward_long_kernel<T, W>, dim3(static_cast<unsigned>(std::min<int64_t>(p.rows, 2 * ops->sm_count))),
                  1024, 0, stream, p);
  return vec ? forward_vec<T, W, 16 / sizeof(T)>(ops, p, stream) : forward_vec<T, W, 1>(ops, p, stream);
}

// Blocks of an SM of the backward kernel, by the threads that share a row.
constexpr int bwd_blocks(int group) { return group <= 256 ? 2 : 1; }
// Columns above which a thread has twice as many.
constexpr int kBwdWide = 1024 * kBwdItems;

int backward_blocks(const gemm_ops* ops, int64_t rows, int64_t cols) {
  if (cols > kMaxCols) return static_cast<int>(std::min<int64_t>(rows, 2 * ops->sm_count));
  const int group = group_of(cols, kBwdItems);
  return static_cast<int>(std::min<int64_t>(ceil_div(rows, int64_t{group == 32 ? kWarpRows : 1}),
                                            static_cast<int64_t>(ops->sm_count) * bwd_blocks(group)));
}

template <typename T, typename W, int kVec, int kGroup, int kItemCols>
cudaError_t backward_as(const gemm_ops* ops, Args p, cudaStream_t stream) {
  constexpr int kBlocks = bwd_blocks(kGroup);
  const Shape s = shape_of<kVec>(ops, p, kGroup, kBlocks, 2);
  p.ahead = s.ahead;
  return launch(backward_kernel<T, W, kVec, kGroup, kItemCols, kBlocks>, dim3(s.blocks), s.threads, s.smem, stream, p);
}
template <typename T, typename W, int kVec>
cudaError_t backward_vec(const gemm_ops* ops, const Args& p, cudaStream_t stream) {
  if (p.cols > kBwdWide) return backward_as<T, W, kVec, 1024, 2 * kBwdItems>(ops, p, stream);
  switch (group_of(p.cols, kBwdItems)) {
    case 32: return backward_as<T, W, kVec, 32, kBwdItems>(ops, p, stream);
    case 256: return backward_as<T, W, kVec, 256, kBwdItems>(ops, p, stream);
    case 512: return backward_as<T, W, kVec, 512, kBwdItems>(ops, p, stream);
    default: return backward_as<T, W, kVec, 1024, kBwdItems>(ops, p, stream);
  }
}
template <typename T, typename W>
cudaError_t backward(const gemm_ops* ops, const Args& p, bool vec, W* dweight, W* dbias, cudaStream_t stream) {
  const int blocks = backward_blocks(ops, p.rows, p.cols);
  cudaError_t e;
  if (p.cols > kMaxCols)
    e = launch(backward_long_kernel<T, W>, dim3(blocks), 1024, 0, stream, p);
  else
    e = vec ? backward_vec<T, W, 16 / sizeof(T)>(ops, p, stream) : backward_vec<T, W, 1>(ops, p, stream);
  if (e != cudaSuccess || !p.partial) return e;
  return launch(sum_kernel<W>, dim3(static_cast<unsigned>(ceil_div(p.cols, int64_t{32})), 2), kSumThreads, 0, stream,
                static_cast<const float*>(p.partial), blocks, p.cols, dweight, dbias);
}

template <typename T, typename W, int kVec>
cudaError_t set_smem_vec(size_t smem) {
  const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const int bytes = static_cast<int>(smem - kStaticBytes);
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, attr, bytes);
  };
  set(forward_kernel<T, W, kVec, 32, 3>);
  set(forward_kernel<T, W, kVec, 256, 3>);
  set(forward_kernel<T, W, kVec, 512, 1>);
  set(forward_kernel<T, W, kVec, 1024, 1>);
  set(backward_kernel<T, W, kVec, 32, kBwdItems, bwd_blocks(32)>);
  set(backward_kernel<T, W, kVec, 256, kBwdItems, bwd_blocks(256)>);
  set(backward_kernel<T, W, kVec, 512, kBwdItems, bwd_blocks(512)>);
  set(backward_kernel<T, W, kVec, 1024, kBwdItems, bwd_blocks(1024)>);
  set(backward_kernel<T, W, kVec, 1024, 2 * kBwdItems, bwd_blocks(1024)>);
  return e;
}

Args args_of(const gemm_layer_norm_args_t* a) {
  Args p{};
  p.x = a->x;
  p.ldx = a->ldx;
  p.weight = a->weight;
  p.stats = a->stats;
  p.rows = a->rows;
  p.cols = static_cast<int>(a->cols);
  p.inv = static_cast<float>(1.0 / static_cast<double>(a->cols));
  return p;
}

}  // namespace

namespace spgemm {

cudaError_t layer_norm_set_smem(size_t smem) {
  cudaError_t e = set_smem_vec<__half, __half, 8>(smem);
  if (e == cudaSuccess) e = set_smem_vec<__half, float, 8>(smem);
  if (e == cudaSuccess) e = set_smem_vec<__nv_bfloat16, __nv_bfloat16, 8>(smem);
  if (e == cudaSuccess) e = set_smem_vec<__nv_bfloat16, float, 8>(smem);
  if (e == cudaSuccess) e = set_smem_vec<float, float, 4>(smem);
  return e;
}

}  // namespace spgemm

extern "C" {

gemm_status_t gemm_layer_norm(gemm_ops_t* ops, const gemm_layer_norm_args_t* args, void* stream_handle) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops) return ops_fail(GEMM_ERR_INVALID_ARG, "ops is NULL");
  gemm_status_t st = check(args, false);
  if (st == GEMM_OK) st = check_overlap(args, false, nullptr, 0);
  if (st != GEMM_OK || args->rows == 0) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  Args p = args_of(args);
  p.bias = args->bias;
  p.out = args->y;
  p.eps = args->eps;
  const int64_t per = args->dtype == GEMM_IN_F32 ? 4 : 8;
  const bool vec = p.cols % per == 0 && p.ldx % per == 0 && aligned16({p.x, p.out, p.weight, p.bias});
  const bool wide = args->weight_dtype == GEMM_IN_F32;
  cudaError_t e;
  if (args->dtype == GEMM_IN_F32)
    e = forward<float, float>(ops, p, vec, stream);
  else if (args->dtype == GEMM_IN_F16)
    e = wide ? forward<__half, float>(ops, p, vec, stream) : forward<__half, __half>(ops, p, vec, stream);
  else
    e = wide ? forward<__nv_bfloat16, float>(ops, p, vec, stream)
             : forward<__nv_bfloat16, __nv_bfloat16>(ops, p, vec, stream);
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "layer norm launch");
}

gemm_status_t gemm_layer_norm_backward_workspace(gemm_ops_t* ops, const gemm_layer_norm_args_t* args, size_t* bytes) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops || !bytes) return ops_fail(GEMM_ERR_INVALID_ARG, "NULL argument");
  const gemm_status_t st = check(args, true);
  if (st != GEMM_OK) return st;
  *bytes = 0;
  if (args->rows > 0 && (args->dweight || args->dbias))
    *bytes = static_cast<size_t>(backward_blocks(ops, args->rows, args->cols)) * 2 * args->cols * sizeof(float);
  return GEMM_OK;
}

gemm_status_t gemm_layer_norm_backward(gemm_ops_t* ops, const gemm_layer_norm_args_t* args, void* workspace,
                                       size_t workspace_bytes, void* stream_handle) {
  size_t need = 0;
  gemm_status_t st = gemm_layer_norm_backward_workspace(ops, args, &need);
  if (st != GEMM_OK) return st;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return ops_fail(GEMM_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return ops_fail(GEMM_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
  st = check_overlap(args, true, workspace, need);
  if (st != GEMM_OK) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  const bool wide = args->weight_dtype == GEMM_IN_F32;
  if (args->rows == 0) {  // sums over no rows
    const size_t n = static_cast<size_t>(args->cols) * (wide ? 4 : 2);
    cudaError_t e = cudaSuccess;
    if (args->dweight) e = cudaMemsetAsync(args->dweight, 0, n, stream);
    if (e == cudaSuccess && args->dbias) e = cudaMemsetAsync(args->dbias, 0, n, stream);
    return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "cudaMemsetAsync(weight gradients)");
  }
  if (!args->dx && !args->dweight && !args->dbias) return GEMM_OK;
  Args p = args_of(args);
  p.dy = args->dy;
  p.lddy = args->lddy;
  p.out = args->dx;
  p.partial = need ? static_cast<float*>(workspace) : nullptr;
  const int64_t per = args->dtype == GEMM_IN_F32 ? 4 : 8;
  bool vec = p.cols % per == 0 && p.ldx % per == 0 && p.lddy % per == 0 && aligned16({p.x, p.dy, p.out, p.weight});
  // (fp32 rows of more than 28672 columns fit no ring.)
  if (vec && p.cols <= kMaxCols && row_bytes(p.cols / per, group_of(p.cols, kBwdItems), 2) > most_smem(ops)) vec = false;
  cudaError_t e;
  void *dw = args->dweight, *db = args->dbias;
  auto run = [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    return backward<T, W>(ops, p, vec, static_cast<W*>(dw), static_cast<W*>(db), stream);
  };
  if (args->dtype == GEMM_IN_F32)
    e = run(float(), float());
  else if (args->dtype == GEMM_IN_F16)
    e = wide ? run(__half(), float()) : run(__half(), __half());
  else
    e = wide ? run(__nv_bfloat16(), float()) : run(__nv_bfloat16(), __nv_bfloat16());
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "layer norm gradient launch");
}

}  // extern "C"
