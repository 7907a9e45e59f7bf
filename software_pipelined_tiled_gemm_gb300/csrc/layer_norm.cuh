// layer_norm.cuh -- layer norm over the rows of a matrix, and its gradients:
// kernels and launches (layer_norm_*.cu: one type of rows each; layer_norm.cu:
// argument checks).
//
// Bound by memory: the forward pass reads x and writes y, the backward pass
// reads x and dy and writes dx.  A row belongs to a group of threads, from a
// warp to a block, each thread holding the same columns (up to 32) of every row
// it meets:
//
//   mean  = sum x / n, then d = x - mean, low = sum d / n,
//   var   = sum d^2 / n - low^2,  h = (d - low) rstd.
//
// The second sum costs no pass of its own and takes out what the rounding of
// the mean to fp32 left in the differences, so that a row far from zero loses
// nothing but its own bits; the backward pass gets both parts of the mean.  A
// row whose sums leave fp32's range, or are mostly the mean's rounding, is taken
// again by itself, scaled (careful_row).
//
// Groups loop over rows.  A thread copies its vectors of the next rows to shared
// memory asynchronously, which keeps rows of every group on their way while one
// is reduced; nobody else reads them, so no barrier is needed.  Rows that are not
// 16-byte aligned, or of no whole number of vectors (kShifted), go by the aligned
// vectors that cover them: a group's rows are a multiple of 8 (fp32: 4) apart, so
// all of them begin at the same place of a vector, and a thread has the same
// columns in each, as with aligned rows.  Only what a row's first and last vector
// holds of other rows is cleared, and its own elements there are written one by
// one.  (A matrix whose rows begin elsewhere in a vector than x's is read or
// written element by element.)  The arithmetic runs on pairs of values, and a
// thread has many columns, so that the reductions over a row (some 25
// instructions each) cost little.
//
// 16384 x 4096 bf16: forward 46 us, backward 76 us (672 MB in all, 5.5 TB/s; with
// scalars and 16 columns a thread the forward pass took 89 us).  fp32: 98 and 124 us
// (5.5 and 6.5 TB/s); 8192 x 8192 96 and 131 us, 4096 x 16384, without rows ahead, 111 and
// 155 us.  16384 x 4097 bf16: 100 and 142 us (read element by element, without copies
// ahead: 300 and 494 us).  Rows a little wider than 1024, 2048, 4096 or 8192 columns
// leave half of their group idle (16384 x 4104: 66 and 110 us), and the masks and
// element stores of unaligned rows are a larger part of narrow ones (262144 x 255: 174
// and 258 us, x 256: 87 and 157).
//
// The weights' gradients: a thread sums its columns over its rows in fp32
// registers; each block leaves one partial, and a second kernel adds those in
// block order.  The sums repeat bit for bit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "layer_norm.h"
#include "packed_f32.cuh"
#include "ptx_block.cuh"

namespace spgemm {
namespace {

constexpr int kAhead = 3;        // rows of a group on their way or in work, at most
constexpr int kItems = 32;       // columns of a thread, at most
constexpr int kMinThreads = 256; // of a block: smaller groups share one
constexpr float kMost = 3.4028235e38f;  // the largest fp32

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

// Two values as they lie in memory, to a pair and back.
template <typename T>
__device__ __forceinline__ F32x2 pair_of(uint32_t w) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>)  // a bf16 is the upper half of its fp32
    return pack_f32(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_f32(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ uint32_t word_of(F32x2 v) {
  const float2 f = unpack_f32(v);
  uint32_t w;
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    memcpy(&w, &h, 4);
  } else {
    const __half2 h = __floats2half2_rn(f.x, f.y);
    memcpy(&w, &h, 4);
  }
  return w;
}

// Elements of 16 bytes.
template <typename T>
constexpr int kVecOf = 16 / static_cast<int>(sizeof(T));

template <typename T>
__device__ __forceinline__ void from_words(uint4 a, F32x2 (&v)[kVecOf<T> / 2]) {
  if constexpr (std::is_same_v<T, float>) {
    v[0] = pack_f32(__uint_as_float(a.x), __uint_as_float(a.y));
    v[1] = pack_f32(__uint_as_float(a.z), __uint_as_float(a.w));
  } else {
    v[0] = pair_of<T>(a.x);
    v[1] = pair_of<T>(a.y);
    v[2] = pair_of<T>(a.z);
    v[3] = pair_of<T>(a.w);
  }
}
template <typename T>
__device__ __forceinline__ uint4 to_words(const F32x2 (&v)[kVecOf<T> / 2]) {
  if constexpr (std::is_same_v<T, float>) {
    const float2 a = unpack_f32(v[0]), b = unpack_f32(v[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  } else {
    return make_uint4(word_of<T>(v[0]), word_of<T>(v[1]), word_of<T>(v[2]), word_of<T>(v[3]));
  }
}
// kN neighbouring columns from p (16-byte aligned), in pairs.
template <typename W, int kN>
__device__ __forceinline__ void load_cols(const W* p, F32x2 (&v)[kN / 2]) {
  constexpr int kEach = kVecOf<W>;
#pragma unroll
  for (int i = 0; i < kN / kEach; ++i) {
    F32x2 part[kEach / 2];
    from_words<W>(reinterpret_cast<const uint4*>(p)[i], part);
#pragma unroll
    for (int j = 0; j < kEach / 2; ++j) v[i * (kEach / 2) + j] = part[j];
  }
}

__device__ __forceinline__ int bytes_past(const void* p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u); }

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

// A thread's vectors of its group's rows.  Of kShifted rows, a group's first vector
// may hold the end of another row and its last one another's beginning.  All threads
// mask those two vectors (others' masks are all ones): a branch for the thread that
// has them would keep its row's threads waiting.
template <typename T, bool kShifted, int kGroup>
struct Share {
  static constexpr int kVec = kVecOf<T>;
  int tid, cols;
  int back;        // elements of a row's first vector before the row
  int vecs;        // of a row
  int used;        // of a thread at most, in any group
  int round;       // in which the group has the last vector
  uint4 head, tail;    // masks of this thread's vectors 0 and `round`
  int tail_bytes;  // of its vector `round`, up to the row's end
  bool edge;       // whether a lane of this warp has one of the two vectors

  // `row`: the group's first
  __device__ __forceinline__ Share(int tid_, int cols_, const T* row) : tid(tid_), cols(cols_) {
    back = kShifted ? bytes_past(row) / static_cast<int>(sizeof(T)) : 0;
    vecs = (back + cols + kVec - 1) / kVec;
    used = (cols + (kShifted ? kVec - 1 : 0) + kVec * kGroup - 1) / (kVec * kGroup);
    round = (vecs - 1) / kGroup;
    tail_bytes = min(16, (cols - col(round)) * static_cast<int>(sizeof(T)));
    head = mask_of(0);
    tail = mask_of(round);
    edge = kShifted && __any_sync(0xffffffffu, partial(0) || (has(round) && partial(round)));
  }
  __device__ __forceinline__ bool has(int i) const { return tid + i * kGroup < vecs; }
  __device__ __forceinline__ int col(int i) const { return (tid + i * kGroup) * kVec - back; }  // of vector i's first element
  __device__ __forceinline__ bool partial(int i) const { return kShifted && (col(i) < 0 || col(i) + kVec > cols); }
  __device__ __forceinline__ bool in(int c) const { return !kShifted || (c >= 0 && c < cols); }
  __device__ __forceinline__ bool fits(const T* row) const { return !kShifted || bytes_past(row) == back * static_cast<int>(sizeof(T)); }

  __device__ __forceinline__ uint4 mask_of(int i) const {
    uint32_t m[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if constexpr (sizeof(T) == 2)
        m[w] = (in(col(i) + 2 * w) ? 0xffffu : 0u) | (in(col(i) + 2 * w + 1) ? 0xffff0000u : 0u);
      else
        m[w] = in(col(i) + w) ? ~0u : 0u;
    }
    return make_uint4(m[0], m[1], m[2], m[3]);
  }
  static __device__ __forceinline__ uint4 both_of(uint4 a, uint4 m) { return make_uint4(a.x & m.x, a.y & m.y, a.z & m.z, a.w & m.w); }

  // Elements of vector i that are not the row's become zero: as they lie in memory, and in fp32.
  __device__ __forceinline__ uint4 own(int i, uint4 a) const {
    if constexpr (kShifted) {
      if (i == 0) a = both_of(a, head);
      if (i == round) a = both_of(a, tail);
    }
    return a;
  }
  static __device__ __forceinline__ void mask_pairs(F32x2 (&v)[kVec / 2], uint4 mask) {
    const uint32_t m[4] = {mask.x, mask.y, mask.z, mask.w};
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j) {
      if constexpr (sizeof(T) == 2)
        v[j] &= static_cast<F32x2>(__byte_perm(m[j], 0u, 0x3232)) << 32 | __byte_perm(m[j], 0u, 0x1010);
      else
        v[j] &= static_cast<F32x2>(m[2 * j + 1]) << 32 | m[2 * j];
    }
  }
  __device__ __forceinline__ void own(int i, F32x2 (&v)[kVec / 2]) const {
    if constexpr (kShifted) {
      if (i == 0) mask_pairs(v, head);
      if (i == round) mask_pairs(v, tail);
    }
  }

  // Copies a row to its place in the ring (`to`: this thread's).  Nothing behind
  // the row is read, nor anything before the matrix.
  template <int kVecs>
  __device__ __forceinline__ void fetch(uint4* to, const T* row, const T* matrix, bool fit) const {
    const T* src = row + (tid * kVec - back);
    if (kShifted && (!fit || row - back < matrix)) {
#pragma unroll 1
      for (int i = 0; i < used; ++i) {
        T* one = reinterpret_cast<T*>(to + i * kGroup);
#pragma unroll 1
        for (int j = 0; j < kVec; ++j) one[j] = in(col(i) + j) ? row[col(i) + j] : from_float<T>(0.0f);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (!has(i)) continue;
      if (kShifted && i == round)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_addr(to + i * kGroup)),
                     "l"(src + i * (kGroup * kVec)), "r"(tail_bytes)
                     : "memory");
      else
        copy_async16(to + i * kGroup, src + i * (kGroup * kVec));
    }
  }

  // Vector i of a row of results.
  __device__ __forceinline__ void store(int i, T* row, bool fit, const F32x2 (&v)[kVec / 2]) const {
    const uint4 y = to_words<T>(v);
    T* to = row + (tid * kVec - back) + i * (kGroup * kVec);
    if (kShifted && (!fit || (edge && (i == 0 || i == round) && partial(i)))) {
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (!in(col(i) + j)) continue;
        if constexpr (sizeof(T) == 2)
          reinterpret_cast<uint16_t*>(to)[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
        else
          reinterpret_cast<uint32_t*>(to)[j] = w[j];
      }
    } else {
      *reinterpret_cast<uint4*>(to) = y;
    }
  }
};

constexpr int block_threads(int group) { return group < kMinThreads ? kMinThreads : group; }

__device__ __forceinline__ F32x2 from_lane(F32x2 v, int d) { return __shfl_xor_sync(0xffffffffu, v, d); }
__device__ __forceinline__ float from_lane(float v, int d) { return __shfl_xor_sync(0xffffffffu, v, d); }
__device__ __forceinline__ F32x2 sum_of(F32x2 a, F32x2 b) { return add_f32x2(a, b); }
__device__ __forceinline__ float sum_of(float a, float b) { return a + b; }

// One value or a pair of the whole group (`op`: a sum, or the least of them), the
// same in every thread: over the lanes, then over the warps, each as a tree.
// `red`: 2 x warps of the group, used in turn.
template <int kGroup, typename V, typename F>
__device__ __forceinline__ V group_reduce(V a, F32x2* red, int& turn, F op) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) a = op(a, from_lane(a, d));
  if constexpr (kGroup > 32) {
    constexpr int kWarps = kGroup / 32;
    V* mine = reinterpret_cast<V*>(red + turn * kWarps);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) mine[(threadIdx.x % kGroup) >> 5] = a;
    if constexpr (kGroup < kMinThreads)
      ptx::named_barrier_sync(1 + threadIdx.x / kGroup, kGroup);
    else
      __syncthreads();
    a = mine[threadIdx.x % kWarps];
#pragma unroll
    for (int d = kWarps / 2; d > 0; d /= 2) a = op(a, from_lane(a, d));
  }
  return a;
}
template <int kGroup, typename V>
__device__ __forceinline__ V group_sum(V a, F32x2* red, int& turn) {
  return group_reduce<kGroup>(a, red, turn, [](V x, V y) { return sum_of(x, y); });
}
// The least of each of two values.
template <int kGroup>
__device__ __forceinline__ float2 group_least(float a, float b, F32x2* red, int& turn) {
  return unpack_f32(group_reduce<kGroup>(pack_f32(a, b), red, turn, [](F32x2 x, F32x2 y) {
    const float2 f = unpack_f32(x), g = unpack_f32(y);
    return pack_f32(fminf(f.x, g.x), fminf(f.y, g.y));
  }));
}
__device__ __forceinline__ float both(F32x2 v) {
  const float2 f = unpack_f32(v);
  return f.x + f.y;
}

template <typename W>
__device__ __forceinline__ float weight_at(const void* base, int col, float otherwise) {
  return base ? to_float(static_cast<const W*>(base)[col]) : otherwise;
}

// This thread's elements of a row in its ring, and of one in memory, with their columns.
template <typename T, int kGroup>
struct InRing {
  const uint4* from;
  int col, cols;  // of the first vector's first element; of the row
  template <typename F>
  __device__ __forceinline__ void operator()(F f) const {
#pragma unroll 1
    for (int i = 0, c = col; c < cols; ++i, c += kGroup * kVecOf<T>)
#pragma unroll 1
      for (int j = 0; j < kVecOf<T>; ++j)
        if (c + j >= 0 && c + j < cols) f(to_float(reinterpret_cast<const T*>(from + i * kGroup)[j]), c + j);
  }
};
template <typename T>
struct InMemory {
  const T* x;
  int cols;
  template <typename F>
  __device__ __forceinline__ void operator()(F f) const {
#pragma unroll 1
    for (int c = threadIdx.x; c < cols; c += 1024) f(to_float(x[c]), c);
  }
};

// Whether a row's sums tell its variance (given with eps added): not where they left
// fp32's range, nor where the mean's rounding, which low takes out of the squares, is
// more than what is left (a constant row far from zero), nor where squares may have
// been too small for fp32 and eps does not hide that.
__device__ __forceinline__ bool sums_do(float squares, float low, float variance) {
  return squares <= kMost && low * low <= variance && variance >= 8.271806125530277e-25f;  // 2^-80
}

// A row whose sums do not, by itself: its statistics and its results.  `each(f)` hands this
// thread's elements and their columns to f.
//
// The row is taken times the power of two that brings its largest magnitude to [1, 2)
// (at the ends of fp32's exponents: to [2^-23, 4)), where no sum of up to 2^29 columns
// leaves the range.  The mean's first part is kept between the least and the greatest
// element, so that a constant row has differences of 0, and the variance is that of
// what both parts leave.  It is 0 or so large that it hides an eps that the scale takes
// below fp32's range.  NaN and infinities have NaN differences, and so give NaN.
//
// Weights are read from memory and elements one by one, so that the loop around it needs
// no registers for this.  (An even number of reductions: the caller's `turn` holds.)
template <typename T, typename W, int kGroup, typename Each>
__device__ __forceinline__ void careful_row(const Each& each, const LayerNormJob& p, int64_t row, bool keeps, F32x2* red, int turn) {
  float2 least = make_float2(__int_as_float(0x7f800000), __int_as_float(0x7f800000));  // of x, and of -x
  each([&](float x, int) {
    least.x = fminf(least.x, x);
    least.y = fminf(least.y, -x);
  });
  least = group_least<kGroup>(least.x, least.y, red, turn);
  // Biased exponents of the scale, 254 - e, and of 1 / scale, e: both normal numbers.
  const uint32_t e = min(max(__float_as_uint(fmaxf(fabsf(least.x), fabsf(least.y))) >> 23, 1u), 253u);
  const float scale = __uint_as_float((254u - e) << 23), unscale = __uint_as_float(e << 23);
  float sum = 0.0f;
  each([&](float x, int) { sum += x * scale; });
  const float mean = fminf(fmaxf(group_sum<kGroup>(sum, red, turn) * p.inv, least.x * scale), -least.y * scale);
  sum = 0.0f;
  each([&](float x, int) { sum += x * scale - mean; });
  const float low = group_sum<kGroup>(sum, red, turn) * p.inv;
  sum = 0.0f;
  each([&](float x, int) {
    const float d = (x * scale - mean) - low;
    sum = fmaf(d, d, sum);
  });
  const float variance = group_sum<kGroup>(sum, red, turn) * p.inv;
  // Of the scaled row, and of the row.
  const float eps = p.eps * scale * scale;
  float scaled = rsqrtf(variance + eps), rstd = scaled * scale;
  if (variance == 0.0f || eps > kMost) {  // eps alone
    rstd = rsqrtf(p.eps);
    scaled = rstd <= kMost ? fminf(rstd * unscale, kMost) : rstd;  // (differences of 0 stay so)
  }
  if (p.stats != nullptr && keeps) {
    p.stats[row] = mean * unscale;
    p.stats[p.rows + row] = low * unscale;
    p.stats[2 * p.rows + row] = rstd;
  }
  T* out = static_cast<T*>(p.out) + row * p.cols;
  each([&](float x, int c) {
    const float h = ((x * scale - mean) - low) * scaled;
    out[c] = from_float<T>(fmaf(h, weight_at<W>(p.weight, c, 1.0f), weight_at<W>(p.bias, c, 0.0f)));
  });
}

// How a kernel meets its weights.
constexpr int kInRegisters = 0, kInShared = 1, kInMemory = 2;
// fp32 weights: registers, and two blocks an SM, where a block's registers
// hold them.  16-bit ones: shared memory and three blocks.  (Registers and shared
// memory, 16384 x 4096 with fp32 weights: 41 and 60 us; 8192 x 8192 with bf16
// weights: 45 and 41 us.)  Unaligned rows, whose masks take registers: shared memory
// and two blocks (16384 x 5001 with bf16 weights: 106 us, three blocks 124 us; 65536 x
// 1001: 67 and 83 us).  Four bytes a column of 32768 columns fit no shared memory: read from L2.
template <typename W>
constexpr int weights_at(int group, bool shifted) {
  if (group == 1024) return kInMemory;
  return shifted ? kInShared : group == 32 || (group <= 256 && sizeof(W) == 4) ? kInRegisters : kInShared;
}

// fp32 weights of columns [col, col + kN), in pairs; `cols`: of the row, which may
// not have all of them (0: it has, and they are aligned).
template <typename W, int kN>
__device__ __forceinline__ void weights_of(const void* base, int col, int cols, float otherwise, F32x2 (&out)[kN / 2]) {
  const W* w = static_cast<const W*>(base) + col;
  if (base == nullptr) {
#pragma unroll
    for (int j = 0; j < kN / 2; ++j) out[j] = both_f32(otherwise);
  } else if (cols > 0 && (col < 0 || col + kN > cols || bytes_past(w) != 0)) {
    auto at = [&](int j) { return col + j >= 0 && col + j < cols ? to_float(w[j]) : 0.0f; };
#pragma unroll
    for (int j = 0; j < kN / 2; ++j) out[j] = pack_f32(at(2 * j), at(2 * j + 1));
  } else if constexpr (kN >= kVecOf<W>) {  // (rows of fp32 have fp32 weights)
    load_cols<W, kN>(w, out);
  }
}

template <typename T, typename W, bool kShifted, int kGroup, int kBlocks>
__global__ void __launch_bounds__(block_threads(kGroup), kBlocks) forward_kernel(const LayerNormJob p) {
  constexpr int kVec = kVecOf<T>;
  constexpr int kVecs = kItems / kVec;          // vectors of a thread
  constexpr int kPairs = kVec / 2;              // pairs of a vector
  constexpr int kGroups = block_threads(kGroup) / kGroup;
  constexpr int kWeights = weights_at<W>(kGroup, kShifted);
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ F32x2 red_all[kGroup > 32 ? 2 * block_threads(kGroup) / 32 : 1];
  ptx::pdl_launch_dependents();
  const int tid = threadIdx.x % kGroup, group = threadIdx.x / kGroup;
  F32x2* red = red_all + (kGroup > 32 ? group * 2 * (kGroup / 32) : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  const int edge = kShifted ? p.cols : 0;
  const T* x = static_cast<const T*>(p.x);
  int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const Share<T, kShifted, kGroup> share(tid, p.cols, x + row * p.ldx);
  const W* weights = nullptr;  // kInShared: columns as in memory
  const W* biases = nullptr;
  uint8_t* rows = ring;
  ptx::pdl_wait_prior_grid();
  F32x2 w[kWeights == kInRegisters ? kVecs : 1][kPairs], b[kWeights == kInRegisters ? kVecs : 1][kPairs];
  if constexpr (kWeights == kInRegisters) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (share.has(i)) {
        weights_of<W, kVec>(p.weight, share.col(i), edge, 1.0f, w[i]);
        weights_of<W, kVec>(p.bias, share.col(i), edge, 0.0f, b[i]);
      }
  }
  if constexpr (kWeights == kInShared) {
    // (Each thread reads back what it wrote itself, or another group wrote there too.)
    const int wide = kShifted ? share.used * kGroup * kVec : p.cols;
    W* to = reinterpret_cast<W*>(ring) + (kShifted ? group * 2 * wide : 0);
    weights = to;
    biases = to + wide;
    auto bring = [&](W* dst, const void* base) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        if (!share.has(i)) continue;
        const W* src = static_cast<const W*>(base) + share.col(i);
        W* own = dst + (tid + i * kGroup) * kVec;
        if (kShifted && (share.partial(i) || bytes_past(src) != 0)) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) own[j] = share.in(share.col(i) + j) ? src[j] : from_float<W>(0.0f);
        } else {
#pragma unroll
          for (int j = 0; j < kVec * static_cast<int>(sizeof(W)) / 16; ++j)
            reinterpret_cast<uint4*>(own)[j] = reinterpret_cast<const uint4*>(src)[j];
        }
      }
    };
    if (p.weight) bring(to, p.weight);
    if (p.bias) bring(to + wide, p.bias);
    rows += p.weight_bytes;
  }
  const int row_vecs = share.used * kGroup;  // in the ring
  uint4* mine = reinterpret_cast<uint4*>(rows) + group * p.ahead * row_vecs + tid;
  int turn = 0;
  const bool fit = share.fits(static_cast<const T*>(p.out) + row * p.cols);

  auto fetch = [&](int64_t r, int slot) {
    if (r < p.rows) share.template fetch<kVecs>(mine + slot * row_vecs, x + r * p.ldx, x, true);
    copy_async_commit();
  };
  for (int s = 0; s < p.ahead - 1; ++s) fetch(row + s * step, s);

  for (int slot = 0; row < p.rows; row += step) {
    F32x2 v[kVecs][kPairs];
    fetch(row + (p.ahead - 1) * step, slot == 0 ? p.ahead - 1 : slot - 1);
    copy_async_wait(p.ahead);
    const uint4* from = mine + slot * row_vecs;
    slot = slot == p.ahead - 1 ? 0 : slot + 1;
    F32x2 sum = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (share.has(i)) {
        from_words<T>(share.own(i, from[i * kGroup]), v[i]);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) sum = add_f32x2(sum, v[i][j]);
      }
    }
    const float mean = group_sum<kGroup>(both(sum), red, turn) * p.inv;
    F32x2 lows = 0, squares = 0;
    const F32x2 minus = both_f32(-mean);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (share.has(i)) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) v[i][j] = add_f32x2(v[i][j], minus);
        share.own(i, v[i]);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          lows = add_f32x2(lows, v[i][j]);
          squares = fma_f32x2(v[i][j], v[i][j], squares);
        }
      }
    const float2 sums = unpack_f32(group_sum<kGroup>(pack_f32(both(lows), both(squares)), red, turn));
    const float low = sums.x * p.inv, variance = fmaxf(sums.y * p.inv - low * low, 0.0f) + p.eps;
    if (!sums_do(sums.y, low, variance)) {  // the same in all threads of the group
      careful_row<T, W, kGroup>(InRing<T, kGroup>{from, share.col(0), p.cols}, p, row, tid == 0, red, turn);
      continue;
    }
    const float rstd = rsqrtf(variance);
    if (p.stats != nullptr && tid == 0) {
      p.stats[row] = mean;
      p.stats[p.rows + row] = low;
      p.stats[2 * p.rows + row] = rstd;
    }
    T* out = static_cast<T*>(p.out) + row * p.cols;
    const F32x2 scale = both_f32(rstd), shift = both_f32(-low * rstd);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (share.has(i)) {
        F32x2 wi[kPairs], bi[kPairs], y[kPairs];
        if constexpr (kWeights == kInShared) {
          weights_of<W, kVec>(p.weight ? weights : nullptr, (tid + i * kGroup) * kVec, 0, 1.0f, wi);
          weights_of<W, kVec>(p.bias ? biases : nullptr, (tid + i * kGroup) * kVec, 0, 0.0f, bi);
        } else if constexpr (kWeights == kInMemory) {
          weights_of<W, kVec>(p.weight, share.col(i), edge, 1.0f, wi);
          weights_of<W, kVec>(p.bias, share.col(i), edge, 0.0f, bi);
        }
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const F32x2 h = fma_f32x2(v[i][j], scale, shift);
          y[j] = kWeights == kInRegisters ? fma_f32x2(h, w[i][j], b[i][j]) : fma_f32x2(h, wi[j], bi[j]);
        }
        share.store(i, out, fit, y);
      }
  }
}

// Rows of more columns than a block holds: read three times, the second and
// third mostly from L2.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) forward_long_kernel(const LayerNormJob p) {
  __shared__ F32x2 red[2 * 32];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    float sum = 0.0f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) sum = fmaf(to_float(x[c]), p.inv, sum);
    const float mean = group_sum<1024>(sum, red, turn);
    float low = 0.0f, squares = 0.0f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float d = to_float(x[c]) - mean;
      low = fmaf(d, p.inv, low);
      squares = fmaf(d * p.inv, d, squares);
    }
    const float2 both = unpack_f32(group_sum<1024>(pack_f32(low, squares), red, turn));
    low = both.x;
    const float variance = fmaxf(both.y - low * low, 0.0f) + p.eps;
    if (!sums_do(both.y, low, variance)) {
      careful_row<T, W, 1024>(InMemory<T>{x, p.cols}, p, row, threadIdx.x == 0, red, turn);
      continue;
    }
    const float rstd = rsqrtf(variance);
    if (p.stats != nullptr && threadIdx.x == 0) {
      p.stats[row] = mean;
      p.stats[p.rows + row] = low;
      p.stats[2 * p.rows + row] = rstd;
    }
    T* out = static_cast<T*>(p.out) + row * p.cols;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float w = weight_at<W>(p.weight, c, 1.0f), b = weight_at<W>(p.bias, c, 0.0f);
      out[c] = from_float<T>(fmaf((to_float(x[c]) - mean - low) * rstd, w, b));
    }
  }
}

// h = (x down + minus) rstd + shift, as the backward pass takes it.  Where mean rstd leaves
// fp32's range the row is a constant one (others' deviations are 2^-24 mean / sqrt(n) or more):
// h is 0, also of the zeros that stand for what lies beside an unaligned row.  Where the
// deviation is so large that a difference from the mean may leave the range (2^128 in a row of
// up to 2^29 columns: a deviation of 2^113 at least) a quarter of x and mean is taken.
struct ToNormal {
  float down, minus, rstd, shift;
  __device__ __forceinline__ ToNormal(float mean, float low, float r) {
    const bool large = r < 7.888609052210118e-31f;  // 2^-100
    down = large ? 0.25f : 1.0f;
    minus = -mean * down;
    rstd = fabsf(mean * r) > kMost / 2 ? 0.0f : r;
    shift = -low * rstd;
    if (large) rstd *= 4.0f;
  }
  __device__ __forceinline__ float h(float x) const { return fmaf(fmaf(x, down, minus), rstd, shift); }
};

template <typename T, typename W, bool kShifted, int kGroup>
__global__ void __launch_bounds__(block_threads(kGroup), 1) backward_kernel(const LayerNormJob p) {
  constexpr int kVec = kVecOf<T>, kVecs = kItems / kVec, kPairs = kVec / 2;
  constexpr int kGroups = block_threads(kGroup) / kGroup;
  constexpr bool kHeld = kGroup <= 256;  // weights in registers
  constexpr bool kKept = kGroup <= 256;  // and h and g between the two passes over a row
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ F32x2 red_all[kGroup > 32 ? 2 * block_threads(kGroup) / 32 : 1];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  const int tid = threadIdx.x % kGroup, group = threadIdx.x / kGroup;
  F32x2* red = red_all + (kGroup > 32 ? group * 2 * (kGroup / 32) : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  const Share<T, kShifted, kGroup> share(tid, p.cols, x + row * p.ldx);
  const bool fit = share.fits(static_cast<const T*>(p.out) + row * p.cols), fit_dy = share.fits(dy + row * p.lddy);
  const int edge = kShifted ? p.cols : 0;
  // [slot][x, dy][vector][thread]
  const int row_vecs = share.used * kGroup;
  uint4* mine = reinterpret_cast<uint4*>(ring) + group * p.ahead * 2 * row_vecs + tid;
  int turn = 0;
  F32x2 dw[kVecs][kPairs], db[kVecs][kPairs], w[kHeld ? kVecs : 1][kPairs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) dw[i][j] = db[i][j] = 0;
    if (kHeld && share.has(i)) weights_of<W, kVec>(p.weight, share.col(i), edge, 1.0f, w[kHeld ? i : 0]);
  }

  auto fetch = [&](int64_t r, int slot) {
    if (r < p.rows) {
      uint4* to = mine + slot * 2 * row_vecs;
      share.template fetch<kVecs>(to, x + r * p.ldx, x, true);
      share.template fetch<kVecs>(to + row_vecs, dy + r * p.lddy, dy, fit_dy);
    }
    copy_async_commit();
  };
  float next_mean = 0.0f, next_low = 0.0f, next_rstd = 0.0f;
  auto fetch_stats = [&](int64_t r) {
    if (r < p.rows) {
      next_mean = p.stats[r];
      next_low = p.stats[p.rows + r];
      next_rstd = p.stats[2 * p.rows + r];
    }
  };
  for (int s = 0; s < p.ahead - 1; ++s) fetch(row + s * step, s);
  fetch_stats(row);

  for (int slot = 0; row < p.rows; row += step) {
    const float rstd = next_rstd;
    const ToNormal to_h(next_mean, next_low, rstd);
    const F32x2 down = both_f32(to_h.down), minus = both_f32(to_h.minus), up = both_f32(to_h.rstd), shift = both_f32(to_h.shift), scale = both_f32(rstd);
    fetch(row + (p.ahead - 1) * step, slot == 0 ? p.ahead - 1 : slot - 1);
    copy_async_wait(p.ahead);
    fetch_stats(row + step);
    const uint4* from = mine + slot * 2 * row_vecs;
    slot = slot == p.ahead - 1 ? 0 : slot + 1;
    // dy, h and g of this thread's vector i, from shared memory.  The second pass over the row finds h and g in registers where one
    // block an SM leaves it enough of them (16384 x 4096 bf16,
    // forward and backward together: 119.5 us without, 117.3 us so).
    auto values = [&](int i, F32x2 (&d)[kPairs], F32x2 (&h)[kPairs], F32x2 (&g)[kPairs]) {
      from_words<T>(share.own(i, from[i * kGroup]), h);
      from_words<T>(share.own(i, from[row_vecs + i * kGroup]), d);
      if constexpr (!kHeld) weights_of<W, kVec>(p.weight, share.col(i), edge, 1.0f, g);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        h[j] = fma_f32x2(fma_f32x2(h[j], down, minus), up, shift);
        g[j] = mul_f32x2(kHeld ? w[kHeld ? i : 0][j] : g[j], d[j]);
      }
    };
    F32x2 gs = 0, ghs = 0;
    F32x2 hs[kKept ? kVecs : 1][kPairs], gk[kKept ? kVecs : 1][kPairs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (share.has(i)) {
        F32x2 d[kPairs], h[kPairs], g[kPairs];
        values(i, d, h, g);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          if (kKept) hs[kKept ? i : 0][j] = h[j], gk[kKept ? i : 0][j] = g[j];
          dw[i][j] = fma_f32x2(d[j], h[j], dw[i][j]);
          db[i][j] = add_f32x2(db[i][j], d[j]);
          gs = add_f32x2(gs, g[j]);
          ghs = fma_f32x2(g[j], h[j], ghs);
        }
      }
    if (p.out != nullptr) {
      const float2 sums = unpack_f32(group_sum<kGroup>(pack_f32(both(gs), both(ghs)), red, turn));
      // rstd (g - <g> - h <g h>)
      const F32x2 m1 = both_f32(-sums.x * p.inv * rstd), m2 = both_f32(-sums.y * p.inv * rstd);
      T* out = static_cast<T*>(p.out) + row * p.cols;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (share.has(i)) {
          F32x2 d[kPairs], h[kPairs], g[kPairs];
          if (!kKept) values(i, d, h, g);
#pragma unroll
          for (int j = 0; j < kPairs; ++j)
            d[j] = kKept ? fma_f32x2(hs[kKept ? i : 0][j], m2, fma_f32x2(gk[kKept ? i : 0][j], scale, m1))
                         : fma_f32x2(h[j], m2, fma_f32x2(g[j], scale, m1));
          share.store(i, out, fit, d);
        }
    }
  }

  if (p.partial == nullptr) return;
  float* to = p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.cols;
  auto each = [&](auto&& f) {  // this thread's sums, by column
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (share.has(i))
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float2 a = unpack_f32(dw[i][j]), c = unpack_f32(db[i][j]);
          const int col = share.col(i) + 2 * j;
          if (share.in(col)) f(col, a.x, c.x);
          if (share.in(col + 1)) f(col + 1, a.y, c.y);
        }
  };
  if constexpr (kGroups > 1) {
    // The block's groups one after another, each adding to the sum before it.
    float* sums = reinterpret_cast<float*>(ring);
    copy_async_wait(1);
    for (int turn_of = 0; turn_of < kGroups; ++turn_of) {
      __syncthreads();
      if (turn_of != group) continue;
      each([&](int col, float a, float c) {
        sums[col] = group == 0 ? a : sums[col] + a;
        sums[p.cols + col] = group == 0 ? c : sums[p.cols + col] + c;
      });
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.cols; c += block_threads(kGroup)) to[c] = sums[c];
  } else {
    each([&](int col, float a, float c) {
      to[col] = a;
      to[p.cols + col] = c;
    });
  }
}

// Rows of more columns than a block holds: a block sums a share of the rows
// into its own partial in memory.
template <typename T, typename W>
__global__ void __launch_bounds__(1024, 2) backward_long_kernel(const LayerNormJob p) {
  __shared__ F32x2 red[2 * 32];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  int turn = 0;
  float* to = p.partial ? p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.cols : nullptr;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const float mean = p.stats[row], low = p.stats[p.rows + row];
    const float rstd = p.stats[2 * p.rows + row];
    const ToNormal to_h(mean, low, rstd);
    float gs = 0.0f, ghs = 0.0f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float d = to_float(dy[c]), h = to_h.h(to_float(x[c]));
      const float w = weight_at<W>(p.weight, c, 1.0f);
      gs = fmaf(d * w, p.inv, gs);
      ghs = fmaf(d * w * p.inv, h, ghs);
      if (to) {  // the thread's own columns
        const bool first = row == blockIdx.x;
        to[c] = first ? d * h : to[c] + d * h;
        to[p.cols + c] = first ? d : to[p.cols + c] + d;
      }
    }
    if (p.out == nullptr) continue;
    const float2 means = unpack_f32(group_sum<1024>(pack_f32(gs, ghs), red, turn));
    T* out = static_cast<T*>(p.out) + row * p.cols;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float w = weight_at<W>(p.weight, c, 1.0f);
      const float d = to_float(dy[c]), h = to_h.h(to_float(x[c]));
      out[c] = from_float<T>(rstd * (d * w - means.x - h * means.y));
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
    constexpr int kFlight = 10;  // loads on their way: all of a warp's where there are two blocks an SM
    for (int b = warp * each; b < end; b += kFlight) {
      float v[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) v[i] = b + i < end ? __ldcg(src + static_cast<size_t>(b + i) * 2 * cols) : 0.0f;
#pragma unroll
      for (int i = 0; i < kFlight; ++i) s += v[i];
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= cols) return;
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < 32; ++w) total += sums[w][lane];
  out[col] = from_float<W>(total);
}

// Threads that share a row.
template <typename F>
cudaError_t by_group(int64_t cols, F f) {
  using std::integral_constant;
  if (cols <= 32 * kItems) return f(integral_constant<int, 32>());
  if (cols <= 64 * kItems) return f(integral_constant<int, 64>());
  if (cols <= 128 * kItems) return f(integral_constant<int, 128>());
  if (cols <= 256 * kItems) return f(integral_constant<int, 256>());
  if (cols <= 512 * kItems) return f(integral_constant<int, 512>());
  return f(integral_constant<int, 1024>());
}

// Blocks of an SM that the registers are shared out for.
template <typename W>
constexpr int forward_blocks(int group, bool shifted) {
  if (group >= 512) return 1;
  return weights_at<W>(group, shifted) == kInShared && !shifted ? 3 : 2;
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

// A group has one row, or rows that lie a multiple of 8 apart.
int grid_of(const gemm_ops* ops, int64_t rows, int groups, int per_sm) {
  const int64_t most = std::max<int64_t>(8, static_cast<int64_t>(ops->sm_count) * per_sm / 8 * 8);
  return static_cast<int>(std::min(ceil_div(rows, int64_t{groups}), most));
}

// The ring's depth: p->ahead rows of `row` bytes a block beside `beside` bytes,
// so that `per_sm` blocks fit an SM with two rows each if they can.  False: not one row fits.
bool ring_of(const gemm_ops* ops, LayerNormJob* p, size_t row, size_t beside, int per_sm, size_t* smem) {
  const size_t most = ops->smem_optin - kLayerNormStatic;
  p->ahead = kAhead;
  while (p->ahead > 2 && (p->ahead * row + beside + kLayerNormStatic) * per_sm > ops->smem_optin) --p->ahead;
  while (p->ahead > 1 && p->ahead * row + beside > most) --p->ahead;
  *smem = p->ahead * row + beside;
  return *smem <= most;
}

// Columns that a group's threads need room for: unaligned rows may begin anywhere
// in their first vector.
template <typename T, bool kShifted>
int64_t room_of(int64_t cols) {
  return cols + (kShifted ? kVecOf<T> - 1 : 0);
}
// Vectors of a block's threads for a row of each group.
template <typename T, bool kShifted>
size_t block_vecs(int64_t cols, int group) {
  return static_cast<size_t>(block_threads(group)) * ceil_div(room_of<T, kShifted>(cols), int64_t{kVecOf<T>} * group);
}

template <typename T, typename W, bool kShifted>
cudaError_t forward_rows(const gemm_ops* ops, LayerNormJob p, cudaStream_t stream) {
  return by_group(room_of<T, kShifted>(p.cols), [&](auto g) {
    constexpr int kGroup = g(), kBlocks = forward_blocks<W>(kGroup, kShifted), kThreads = block_threads(kGroup);
    const size_t vecs = block_vecs<T, kShifted>(p.cols, kGroup);
    p.weight_bytes = 0;
    if (weights_at<W>(kGroup, kShifted) == kInShared)
      p.weight_bytes = static_cast<int>(2 * sizeof(W) * (kShifted ? vecs * kVecOf<T> : round8(p.cols)));
    size_t smem;
    if (!ring_of(ops, &p, vecs * 16, p.weight_bytes, kBlocks, &smem)) return cudaErrorInvalidValue;
    return launch(forward_kernel<T, W, kShifted, kGroup, kBlocks>, dim3(grid_of(ops, p.rows, kThreads / kGroup, kBlocks)),
                  kThreads, smem, stream, p);
  });
}

int long_grid(const gemm_ops* ops, int64_t rows) { return static_cast<int>(std::min<int64_t>(rows, 2 * ops->sm_count)); }

template <typename T, bool kShifted>
int backward_grid(const gemm_ops* ops, int64_t rows, int64_t cols) {
  int n = 0;
  by_group(room_of<T, kShifted>(cols), [&](auto g) {
    n = grid_of(ops, rows, block_threads(g()) / g(), 1);
    return cudaSuccess;
  });
  return n;
}

// Whether one row of x and dy fits the ring (fp32 rows of more than 28672 columns do not).
template <typename T, bool kShifted>
bool backward_fits(const gemm_ops* ops, int64_t cols) {
  bool fits = room_of<T, kShifted>(cols) <= kLayerNormMaxCols;
  by_group(room_of<T, kShifted>(cols), [&](auto g) {
    fits = fits && block_vecs<T, kShifted>(cols, g()) * 32 <= ops->smem_optin - kLayerNormStatic;
    return cudaSuccess;
  });
  return fits;
}

template <typename T, typename W, bool kShifted>
cudaError_t backward_rows(const gemm_ops* ops, LayerNormJob p, int blocks, cudaStream_t stream) {
  return by_group(room_of<T, kShifted>(p.cols), [&](auto g) {
    constexpr int kGroup = g(), kThreads = block_threads(kGroup);
    size_t smem;
    if (!ring_of(ops, &p, block_vecs<T, kShifted>(p.cols, kGroup) * 32, 0, 1, &smem)) return cudaErrorInvalidValue;
    if (kThreads > kGroup) smem = std::max(smem, static_cast<size_t>(p.cols) * 2 * sizeof(float));
    return launch(backward_kernel<T, W, kShifted, kGroup>, dim3(blocks), kThreads, smem, stream, p);
  });
}

template <typename T, typename W>
cudaError_t forward(const gemm_ops* ops, const LayerNormJob& p, bool vec, cudaStream_t stream) {
  if (room_of<T, true>(p.cols) > kLayerNormMaxCols && !(vec && p.cols <= kLayerNormMaxCols))
    return launch(forward_long_kernel<T, W>, dim3(long_grid(ops, p.rows)), 1024, 0, stream, p);
  return vec ? forward_rows<T, W, false>(ops, p, stream) : forward_rows<T, W, true>(ops, p, stream);
}

template <typename T, typename W>
cudaError_t backward(const gemm_ops* ops, const LayerNormJob& p, bool vec, void* dweight, void* dbias, cudaStream_t stream) {
  const bool fits = vec ? backward_fits<T, false>(ops, p.cols) : backward_fits<T, true>(ops, p.cols);
  const int blocks = !fits ? long_grid(ops, p.rows)
                     : vec ? backward_grid<T, false>(ops, p.rows, p.cols)
                           : backward_grid<T, true>(ops, p.rows, p.cols);
  const cudaError_t e = !fits ? launch(backward_long_kernel<T, W>, dim3(blocks), 1024, 0, stream, p)
                        : vec ? backward_rows<T, W, false>(ops, p, blocks, stream)
                              : backward_rows<T, W, true>(ops, p, blocks, stream);
  if (e != cudaSuccess || !p.partial) return e;
  return launch(sum_kernel<W>, dim3(static_cast<unsigned>(ceil_div(p.cols, int64_t{32})), 2), kSumThreads, 0, stream,
                static_cast<const float*>(p.partial), blocks, p.cols, static_cast<W*>(dweight), static_cast<W*>(dbias));
}

template <typename T, typename W, bool kShifted>
cudaError_t set_smem(size_t smem) {
  const int bytes = static_cast<int>(smem - kLayerNormStatic);
  cudaError_t e = cudaSuccess;
  auto set = [&](auto g) {
    constexpr int kGroup = g();
    const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(forward_kernel<T, W, kShifted, kGroup, forward_blocks<W>(kGroup, kShifted)>, attr, bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(backward_kernel<T, W, kShifted, kGroup>, attr, bytes);
    return e;
  };
  for (int64_t cols = 1024; cols <= kLayerNormMaxCols; cols *= 2) by_group(cols, set);
  return e;
}

}  // namespace
}  // namespace spgemm

#define SPGEMM_DEFINE_LAYER_NORM(NAME, T)                                                                       \
  namespace spgemm {                                                                                            \
  cudaError_t layer_norm_set_smem_##NAME(size_t smem) {                                                         \
    cudaError_t e = set_smem<T, T, false>(smem);                                                                \
    if (e == cudaSuccess) e = set_smem<T, float, false>(smem);                                                  \
    if (e == cudaSuccess) e = set_smem<T, T, true>(smem);                                                       \
    if (e == cudaSuccess) e = set_smem<T, float, true>(smem);                                                   \
    return e;                                                                                                   \
  }                                                                                                             \
  cudaError_t layer_norm_forward_##NAME(const gemm_ops* ops, const LayerNormJob& p, bool vec, bool wide,        \
                                        cudaStream_t stream) {                                                  \
    return wide ? forward<T, float>(ops, p, vec, stream) : forward<T, T>(ops, p, vec, stream);                  \
  }                                                                                                             \
  cudaError_t layer_norm_backward_##NAME(const gemm_ops* ops, const LayerNormJob& p, bool vec, bool wide,       \
                                         void* dweight, void* dbias, cudaStream_t stream) {                     \
    return wide ? backward<T, float>(ops, p, vec, dweight, dbias, stream)                                       \
                : backward<T, T>(ops, p, vec, dweight, dbias, stream);                                          \
  }                                                                                                             \
  }
