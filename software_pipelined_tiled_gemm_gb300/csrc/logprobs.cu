// logprobs.cu -- log probabilities of tokens under rows of logits, with the
// row's entropy and best alternatives, and their gradient.
//
// One pass over the logits, bound by memory.  In base 2, with L = fp32(log2 e)
// and an integer reference N near the largest x L,
//   t_j = x_j L - N (one fused multiply-add: one rounding, of the difference),
//   s = sum 2^t,  w = sum 2^t t,
//   log2 p_j = t_j - log2 s,  H = ln 2 (log2 s - w / s).
// Each thread keeps N, s and w of its own elements in fp32; when a larger
// element comes, N grows by an integer d and s' = 2^-d s, w' = 2^-d (w - d s)
// (exact scalings).  Threads, warps and the blocks that share a row are
// combined in a fixed order by the same step.
//
// A block's producer thread streams its rows through a shared-memory ring by
// bulk copies, running ahead into the next row while the block still reduces
// the last one.  Pairs of values go through the packed fp32 instructions;
// masked logits (-inf, or a large negative value) are raised to a finite
// floor first (fp32 and bf16 -2^22, fp16 its lowest value), so that 2^t t is 0
// and not 0 x inf.  A row whose maximum is within reach of that floor (all
// masked by a finite value) or above 4e6 is summed again by the slow form
// (x - m): there N would be too coarse beside it.
//
// Alternatives.  While streaming, each thread also keeps its largest element,
// the first 16-byte vector that holds it and the largest of its other
// vectors.  As keys (value, then lower column first), the k-th largest of 32,
// 64 or 128 groups of threads (at least twice k) is a lower bound of the
// row's k-th best, so only the threads at or above it (k to 2 k of them) have
// anything to offer: each reads its best vector again (from L2), and the few
// whose other vectors reach the bound too have all of theirs read by the
// block.  The elements at or above the bound are collected and ranked.  The
// column in the bound keeps a row of equal logits from offering more than its
// first vectors.  A row that offers more than the list holds (its largest
// elements all in a few threads' vectors) is searched k times.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ops_internal.h"
#include "ptx_block.cuh"

using namespace spgemm;

namespace {

// Threads of a block that compute (one warp more copies): small blocks where
// each takes whole rows, since a block's warps wait for one another several
// times a row (8192 x 500 bf16: 128 threads and five blocks an SM 18 us, 256
// and three 48 us); larger ones where a cluster shares a row (one row of
// 131072, 20 alternatives: 256 threads 10 us, 128 threads 14 us).
constexpr int kRowThreads = 128, kRowBlocks = 5;
constexpr int kShareThreads = 256;
constexpr int kLpUnroll = 4;          // vectors of a thread in a chunk
constexpr int kLpStages = 4;          // chunks of a block's ring
template <int kThreads>
constexpr uint32_t kChunkBytes = kThreads * kLpUnroll * 16u;
constexpr int kLpCandidates = 1024;
constexpr int kMaxTopK = GEMM_LOGPROBS_MAX_TOP_K;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kExpCut = -200.0f;    // 2^-200 is 0 in fp32
constexpr int kBwdThreads = 256;

struct LpArgs {
  const void* logits;
  int64_t ld;
  int vocab;
  int top_k;
  const int64_t* tokens;
  float *logprobs, *entropy, *lse, *lse_low, *top_logprobs;
  int64_t* top_ids;
  // backward
  const float *d_logprobs, *d_entropy;
  void* d_logits;
  int64_t ldd;
  int64_t rows;
  int* status;
  unsigned long long timeout_ns;
  int inject_fault;  // test hook, see gemm_ops_configure
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Unsigned words in the order of the floats: -inf < ... < -0 = +0 < ... <
// +inf < NaN (any).  Between 0 and ~0, so that a key is neither 0 (none) nor
// all ones (the search's start, which every key is below).
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xfffffffeu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z),
    v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    return *reinterpret_cast<const uint4*>(h);
  }
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Vec<__half> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    __half2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    return *reinterpret_cast<const uint4*>(h);
  }
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};

// Two floats in one register pair, for the packed instructions.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack_f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack_f2(F2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ F2 fma_f2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 add_f2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Per type: the largest of a vector's elements (NaN if one is), the vector
// with its elements raised to the floor, and the range of row maxima for
// which the fast sums hold: 2^((floor - m) L) is 0, and |m| L is below 2^23, so
// that the reference is at most 1 from m L (from 2^31 on the fp32 product is
// more than 127 off, and 2^t inf or 0).  kStart: the first reference, below any
// such maximum's and so far above the floor's that masked elements add 0 from
// the start.  Every floor is exact in its type.
template <typename T>
struct Fast;
template <>
struct Fast<float> {
  static constexpr float kFloor = -4194304.0f, kStart = -6050000.0f, kLow = -4193000.0f, kHigh = 4e6f;
  static __device__ __forceinline__ float max(const uint4& w) {
    return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                   max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
  static __device__ __forceinline__ void pairs(const uint4& w, F2 (&v)[2]) {
    v[0] = pack_f2(fmaxf(__uint_as_float(w.x), kFloor), fmaxf(__uint_as_float(w.y), kFloor));
    v[1] = pack_f2(fmaxf(__uint_as_float(w.z), kFloor), fmaxf(__uint_as_float(w.w), kFloor));
  }
};
template <>
struct Fast<__nv_bfloat16> {
  static constexpr float kFloor = -4194304.0f, kStart = -6050000.0f, kLow = -4193000.0f, kHigh = 4e6f;
  static __device__ __forceinline__ __nv_bfloat162 at(const uint32_t& w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  static __device__ __forceinline__ float max(const uint4& w) {
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(at(w.x), at(w.y)), __hmax2_nan(at(w.z), at(w.w)));
    return max_nan(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void pairs(const uint4& w, F2 (&v)[4]) {
    const __nv_bfloat162 lo = __float2bfloat162_rn(kFloor);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 r = __hmax2(at(a[i]), lo);
      const uint32_t b = *reinterpret_cast<const uint32_t*>(&r);
      v[i] = pack_f2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
    }
  }
};
template <>
struct Fast<__half> {
  static constexpr float kFloor = -65504.0f, kStart = -94000.0f, kLow = -65000.0f, kHigh = 65505.0f;
  static __device__ __forceinline__ __half2 at(const uint32_t& w) {
    return *reinterpret_cast<const __half2*>(&w);
  }
  static __device__ __forceinline__ float max(const uint4& w) {
    const __half2 m = __hmax2_nan(__hmax2_nan(at(w.x), at(w.y)), __hmax2_nan(at(w.z), at(w.w)));
    return max_nan(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void pairs(const uint4& w, F2 (&v)[4]) {
    const __half2 lo = __float2half2_rn(kFloor);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(__hmax2(at(a[i]), lo));
      v[i] = pack_f2(f.x, f.y);
    }
  }
};

// A row of logits: `head` elements before the first 16-byte boundary, then
// whole vectors (vector v from column head + v kN), then `tail` elements.
template <typename T>
struct Row {
  static constexpr int kN = Vec<T>::kN;
  const T* p;
  int head, vectors, tail;
  __device__ Row(const T* row, int vocab) : p(row) {
    head = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / sizeof(T));
    head = min(head, vocab);
    vectors = (vocab - head) / kN;
    tail = vocab - head - vectors * kN;
  }
  __device__ __forceinline__ int column(int v) const { return head + v * kN; }
  __device__ __forceinline__ const uint4* at(int v) const {
    return reinterpret_cast<const uint4*>(p + column(v));
  }
  // Columns outside the vectors, by number: fewer than 2 kN of them.
  __device__ __forceinline__ int edges() const { return head + tail; }
  __device__ __forceinline__ int edge_column(int i) const { return i < head ? i : i + vectors * kN; }
};

struct Stats {
  float m;        // the largest element, NaN if one is
  float n, s, w;  // reference, sum 2^t, sum 2^t t
};

// s and w for a reference larger by d >= 0.
__device__ __forceinline__ void lower(float d, float& s, float& w) {
  const float e = fmaxf(-d, kExpCut), f = exp2_approx(e);
  w = f * fmaf(e, s, w);
  s *= f;
}

// Combines the threads of each group of kLanes lanes, for all of them alike:
// the largest reference first, then plain sums in a fixed order.
template <int kLanes>
__device__ __forceinline__ void warp_combine(Stats& t) {
  float n = t.n;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    t.m = max_nan(t.m, __shfl_xor_sync(0xffffffffu, t.m, o));
    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
  }
  lower(n - t.n, t.s, t.w);
  t.n = n;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    t.s += __shfl_xor_sync(0xffffffffu, t.s, o);
    t.w += __shfl_xor_sync(0xffffffffu, t.w, o);
  }
}

template <int kThreads>
struct LpShared {
  uint64_t full[kLpStages], empty[kLpStages];
  Stats warp[2][kThreads / 32];     // of this row and the last one
  Stats block;
  int count, offering;
  uint64_t bound;
  uint64_t best[kMaxTopK];          // this block's best keys, best first
  uint64_t list[kLpCandidates];
  uint64_t group[2 * kMaxTopK];     // the largest key of each group of threads
  int2 offer[kThreads];           // threads with more than one vector to read, and their best
};
template <int kThreads>
constexpr size_t kLpSmem = 128 + kLpStages * static_cast<size_t>(kChunkBytes<kThreads>) + sizeof(LpShared<kThreads>);

// Barrier of the computing warps.
template <int kThreads>
__device__ __forceinline__ void compute_sync() { ptx::named_barrier_sync(1, kThreads); }
__device__ __forceinline__ uint64_t key_of(float x, int column) {
  return (static_cast<uint64_t>(order_of(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(column));
}

// Writes the k largest of list[0, n) to out, in order, and 0 in places that
// no key takes.  Eight lanes count for one key.
template <int kThreads>
__device__ __forceinline__ void rank_keys(const uint64_t* list, int n, int k, uint64_t* out) {
  for (int i = threadIdx.x; i < k; i += kThreads)
    if (i >= n) out[i] = 0;
  for (int base = 0; base < n; base += kThreads / 8) {
    const int i = base + static_cast<int>(threadIdx.x) / 8;
    const uint64_t mine = i < n ? list[i] : 0;
    int rank = 0;
#pragma unroll 4
    for (int j = threadIdx.x % 8; j < n; j += 8) rank += list[j] > mine ? 1 : 0;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (i < n && rank < k && threadIdx.x % 8 == 0) out[rank] = mine;
  }
}

// The k best of the columns this block streamed (vectors v0 + i kThreads +
// thread below v1, and `edge`, the thread's column outside the vectors or
// -1), to sh.best.  top, top_v, second: this thread's largest element, the
// first vector that holds it and the largest element of its other vectors.
// nan: the row holds one, which these do not show.
template <typename T, int kThreads>
__device__ __noinline__ void block_top(const Row<T>& row, int v0, int v1, int edge, int k, float top,
                                       int top_v, float second, bool nan, LpShared<kThreads>& sh) {
  constexpr int kN = Row<T>::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // 32, 64 or 128 groups of threads: at least two for each of the k.
  const int span = kThreads / (k <= 16 ? 32 : (k <= 32 ? 64 : 128));
  const uint64_t key = v0 + tid < v1 ? key_of(top, row.column(top_v)) : 0;
  uint64_t best = key;
  for (int o = span / 2; o > 0; o >>= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
    best = other > best ? other : best;
  }
  if (tid % span == 0) sh.group[tid / span] = best;
  if (tid == 0) {
    sh.count = sh.offering = 0;
    sh.bound = 0;
  }
  compute_sync<kThreads>();
  // The bound: the k-th of the groups' keys (0 if fewer than k have one).  A
  // group's threads share the counting of its rank.
  {
    const int groups = kThreads / span;
    int rank = 0;
#pragma unroll 4
    for (int j = tid % span; j < groups; j += span) rank += sh.group[j] > best ? 1 : 0;
    for (int o = span / 2; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (rank == k - 1 && best != 0 && tid % span == 0) sh.bound = best;  // keys are distinct
  }
  compute_sync<kThreads>();
  const uint64_t bound = sh.bound;
  const float bound_x = value_of(static_cast<uint32_t>(bound >> 32));
  const int bound_c = static_cast<int>(0xffffffffu - static_cast<uint32_t>(bound));
  // Whether an element of the vector from column `first` is at or above it.
  auto reaches = [&](float x, int first) {
    return bound == 0 || x > bound_x || (x == bound_x && first <= bound_c);
  };
  auto take = [&](const uint4& w, int first) {
    float x[kN];
    Vec<T>::unpack(w, x);
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < kN; ++j) mask |= reaches(x[j], first) ? 1u << j : 0u;
    if (mask == 0) return;
    int at = atomicAdd(&sh.count, __popc(mask));
#pragma unroll
    for (int j = 0; j < kN; ++j)
      if ((mask >> j) & 1u) {
        if (at < kLpCandidates) sh.list[at] = key_of(x[j], first + j);
        ++at;
      }
  };
  if (edge >= 0) {
    const float x = Vec<T>::get(row.p[edge]);
    if (reaches(x, edge)) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kLpCandidates) sh.list[at] = key_of(x, edge);
    }
  }
  if (key != 0 && key >= bound) {
    take(__ldg(row.at(top_v)), row.column(top_v));
    // Its other vectors lie at other columns, any of which may be within the bound's.
    if (bound == 0 || second >= bound_x) sh.offer[atomicAdd(&sh.offering, 1)] = make_int2(tid, top_v);
  }
  compute_sync<kThreads>();
  // The other vectors of the threads that have more to offer, a thread's by a warp.
  const int offering = sh.offering;
#pragma unroll 1
  for (int o = warp; o < offering; o += (kThreads / 32)) {
    const int2 who = sh.offer[o];
#pragma unroll 1
    for (int v = v0 + who.x + lane * kThreads; v < v1; v += 32 * kThreads)
      if (v != who.y) take(__ldg(row.at(v)), row.column(v));
  }
  compute_sync<kThreads>();
  const int n = sh.count;
  if (n <= kLpCandidates && !nan) {
    rank_keys<kThreads>(sh.list, n, k, sh.best);
    compute_sync<kThreads>();
    return;
  }
  // More than the list holds, or NaN: the largest key below the last one, k times.
  uint64_t below = ~0ull;
  for (int i = 0; i < k; ++i) {
    best = 0;
    auto offer = [&](float x, int c) {
      const uint64_t candidate = key_of(x, c);
      if (candidate < below && candidate > best) best = candidate;
    };
    if (edge >= 0) offer(Vec<T>::get(row.p[edge]), edge);
    for (int v = v0 + tid; v < v1; v += kThreads) {
      float x[kN];
      Vec<T>::unpack(__ldg(row.at(v)), x);
#pragma unroll
      for (int j = 0; j < kN; ++j) offer(x[j], row.column(v) + j);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
      best = other > best ? other : best;
    }
    if (lane == 0) sh.group[tid >> 5] = best;
    compute_sync<kThreads>();
    for (int j = 0; j < (kThreads / 32); ++j) best = sh.group[j] > best ? sh.group[j] : best;
    if (tid == 0) sh.best[i] = best;
    below = best;
    compute_sync<kThreads>();
  }
}

// The sums of this block's share of a row whose maximum m (finite) is outside
// the fast form's range: t = (x - m) L, the difference first.  The reference
// of the result is m itself.
template <typename T, int kThreads>
__device__ __noinline__ void slow_sums(const Row<T>& row, int v0, int v1, int edge, float m, Stats& t) {
  t.s = t.w = 0.0f;
  auto add = [&](float x) {
    const float e2 = fmaxf((x - m) * kLog2e, kExpCut), e = exp2_approx(e2);
    t.s += e;
    t.w = fmaf(e, e2, t.w);
  };
  if (edge >= 0) add(Vec<T>::get(row.p[edge]));
  for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += kThreads) {
    float x[Row<T>::kN];
    Vec<T>::unpack(__ldg(row.at(v)), x);
#pragma unroll
    for (int j = 0; j < Row<T>::kN; ++j) add(x[j]);
  }
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ float peer_f32(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ptx::map_shared_rank(addr, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t peer_u64(uint32_t addr, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(ptx::map_shared_rank(addr, rank)) : "memory");
  return v;
}

// Bounded wait on a ring barrier; a wait that runs out is recorded.
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, const LpArgs& a, int detail) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ptx::globaltimer_ns() - t0 > a.timeout_ns) {
      if (atomicCAS(a.status, 0, kStatusTimeout) == 0) atomicExch(a.status + 1, detail);
      return false;
    }
  }
  return true;
}

// A row's sums over the block: into sh.block by warp 0, in a fixed order.
template <int kThreads>
__device__ __forceinline__ Stats block_stats(Stats t, LpShared<kThreads>& sh, int parity) {
  warp_combine<32>(t);
  if ((threadIdx.x & 31) == 0) sh.warp[parity][threadIdx.x >> 5] = t;
  compute_sync<kThreads>();
  t = sh.warp[parity][threadIdx.x & (kThreads / 32 - 1)];
  warp_combine<kThreads / 32>(t);
  return t;
}

// Rows row0, row0 + step, ... with one block each; or, launched as clusters
// (few rows), one row per cluster, each block taking a share of its vectors.
template <typename T, bool kTop, int kThreads>
__global__ void __launch_bounds__(kThreads + 32, kThreads == kRowThreads ? kRowBlocks : 1)
    logprobs_kernel(const LpArgs a) {
  constexpr bool kCluster = kThreads == kShareThreads;
  constexpr int kWarps = kThreads / 32, kChunkVecs = kThreads * kLpUnroll;
  constexpr uint32_t kChunk = kChunkBytes<kThreads>;
  constexpr int kN = Vec<T>::kN;
  extern __shared__ uint8_t lp_smem[];
  uint8_t* ring = lp_smem + ((128u - (ptx::smem_addr(lp_smem) & 127u)) & 127u);
  LpShared<kThreads>& sh = *reinterpret_cast<LpShared<kThreads>*>(ring + kLpStages * kChunk);
  const uint32_t ring_addr = ptx::smem_addr(ring);
  const uint32_t full = ptx::smem_addr(sh.full), empty = ptx::smem_addr(sh.empty);
  const uint32_t blocks = kCluster ? cluster_size() : 1u;
  const uint32_t rank = kCluster ? ptx::cluster_ctarank() : 0u;
  const int64_t row0 = blockIdx.x / blocks, step = gridDim.x / blocks;
  const int tid = threadIdx.x;
  if (tid == 0) {
    for (int i = 0; i < kLpStages; ++i) {
      ptx::mbar_init(full + 8u * i, 1);
      ptx::mbar_init(empty + 8u * i, kWarps);
    }
    ptx::fence_barrier_init();
  }
  __syncthreads();
  // The next kernel starts early only behind the few blocks of a shared row:
  // blocks of a large one, resident beside a full grid, slowed it and
  // themselves (8192 x 65536 bf16, forward and gradient in turn: 546 us with
  // the early start, 476 without).
  if constexpr (kCluster) ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();

  auto share = [&](const Row<T>& row, int& v0, int& v1) {
    v0 = static_cast<int>(static_cast<int64_t>(row.vectors) * rank / blocks);
    v1 = static_cast<int>(static_cast<int64_t>(row.vectors) * (rank + 1) / blocks);
  };

  if (tid >= kThreads) {
    // ------------------------------------------------------------ producer --
    if (tid == kThreads) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      uint32_t used = 0, parity = 0;
      const uint64_t pol = ptx::l2_policy_evict_first();
      for (int64_t r = row0; ok && r < a.rows; r += step) {
        const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, a.vocab);
        int v0, v1;
        share(row, v0, v1);
        for (int v = v0; v < v1; v += kChunkVecs) {
          if (!ring_wait(empty + 8u * stage, phase ^ 1u, a, kDetailProducerEmpty)) {
            ok = false;
            break;
          }
          const uint32_t bytes = static_cast<uint32_t>(min(v1 - v, kChunkVecs)) * 16u;
          ptx::mbar_arrive_expect_tx(full + 8u * stage, bytes);
          if (a.inject_fault && blockIdx.x == 0 && used == 0)
            ;  // announced but never copied
          else if constexpr (kTop)  // read again, in part
            ptx::bulk_load(ring_addr + stage * kChunk, row.at(v), bytes, full + 8u * stage);
          else
            ptx::bulk_load_hint(ring_addr + stage * kChunk, row.at(v), bytes, full + 8u * stage, pol);
          used |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kLpStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Every copy lands before the block may leave.
      for (int i = 0; i < kLpStages; ++i)
        if (used & (1u << i)) ring_wait(full + 8u * i, (parity >> i) & 1u, a, kDetailProducerDrain);
    }
    __syncwarp();
    if constexpr (kCluster) {
      ptx::cluster_sync();
      ptx::cluster_sync();
    }
    return;
  }

  // ---------------------------------------------------------------- compute --
  int stage = 0, turn = 0;
  uint32_t phase = 0;
  const F2 l2 = pack_f2(kLog2e, kLog2e);
  bool ok = true;
  for (int64_t r = row0; r < a.rows; r += step, ++turn) {
    const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, a.vocab);
    int v0, v1;
    share(row, v0, v1);
    // This thread's column outside the vectors, if it has one: the head's go
    // with the first block's share, the tail's with the last one's.
    const int edge = tid < row.edges() && rank == (tid < row.head ? 0u : blocks - 1u)
                         ? row.edge_column(tid)
                         : -1;
    // One warp writes the row's results, another one each row: its first lane
    // has the token's logit by then.
    const bool writer = tid == (turn % kWarps) * 32;
    int64_t token = -1;
    float token_x = 0.0f;
    if (writer && a.tokens && a.logprobs && rank == 0) {
      token = a.tokens[r];
      if (token >= 0 && token < a.vocab) token_x = Vec<T>::get(row.p[token]);
    }
    Stats t = {-INFINITY, Fast<T>::kStart, 0.0f, 0.0f};
    F2 s2 = 0, w2 = 0;  // (0.0f, 0.0f)
    float top = -INFINITY;  // the largest element of this thread's vectors,
    int top_v = v0 + tid;   // the first that holds it,
    float second = -INFINITY;  // and the largest of the others'
    // A larger element (its x L, not above the next integer) moves the reference.
    auto reach = [&](float m) {
      t.m = max_nan(t.m, m);
      const float n = m * kLog2e;
      if (n > t.n) {
        const float up = ceilf(n);
        float sa, sb, wa, wb;
        unpack_f2(s2, sa, sb);
        unpack_f2(w2, wa, wb);
        lower(up - t.n, sa, wa);
        lower(up - t.n, sb, wb);
        s2 = pack_f2(sa, sb);
        w2 = pack_f2(wa, wb);
        t.n = up;
      }
    };
    if (edge >= 0) {
      const float x = Vec<T>::get(row.p[edge]);
      reach(x);
      const float e2 = fmaf(fmaxf(x, Fast<T>::kFloor), kLog2e, -t.n), e = exp2_approx(e2);
      s2 = add_f2(s2, pack_f2(e, 0.0f));
      w2 = add_f2(w2, pack_f2(e * e2, 0.0f));
    }
    for (int v = v0; v < v1; v += kChunkVecs) {
      if (ok) ok = ring_wait(full + 8u * stage, phase, a, kDetailMmaFull);
      const uint32_t src = ring_addr + stage * kChunk + static_cast<uint32_t>(tid) * 16u;
      const int left = v1 - v - tid;  // this thread's vectors: u kThreads < left
      uint4 w[kLpUnroll];
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u)
        if (u * kThreads < left) w[u] = ptx::ld_shared_v4(src + u * (kThreads * 16u));
      // The slot goes back at once, and the next copy may land at once: these
      // reads come before it only by a fence between the two proxies.
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if ((tid & 31) == 0) ptx::mbar_arrive(empty + 8u * stage);
      if (++stage == kLpStages) {
        stage = 0;
        phase ^= 1u;
      }
      float m = -INFINITY;
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u)
        if (u * kThreads < left) {
          const float vm = Fast<T>::max(w[u]);
          m = max_nan(m, vm);
          if constexpr (kTop) {
            second = fmaxf(second, fminf(vm, top));
            if (vm > top) {
              top = vm;
              top_v = v + tid + u * kThreads;
            }
          }
        }
      reach(m);
      const F2 n2 = pack_f2(-t.n, -t.n);
#pragma unroll
      for (int u = 0; u < kLpUnroll; ++u)
        if (u * kThreads < left) {
          F2 x[kN / 2];
          Fast<T>::pairs(w[u], x);
#pragma unroll
          for (int j = 0; j < kN / 2; ++j) {
            const F2 e2 = fma_f2(x[j], l2, n2);
            float ea, eb;
            unpack_f2(e2, ea, eb);
            const F2 e = pack_f2(exp2_approx(ea), exp2_approx(eb));
            s2 = add_f2(s2, e);
            w2 = fma_f2(e, e2, w2);
          }
        }
    }
    {
      float sa, sb, wa, wb;
      unpack_f2(s2, sa, sb);
      unpack_f2(w2, wa, wb);
      t.s = sa + sb;
      t.w = wa + wb;
    }
    t = block_stats(t, sh, turn & 1);  // the same in every warp
    if constexpr (kTop)
      block_top<T, kThreads>(row, v0, v1, edge, a.top_k, top, top_v, second, t.m != t.m, sh);

    // The blocks of a cluster share their sums (their maxima, if the slow
    // form is needed: then again).
    if constexpr (kCluster) {
      if (tid == 0) sh.block = t;
      ptx::cluster_sync();
      const uint32_t at = ptx::smem_addr(&sh.block), peer = tid & 7;
      t = {-INFINITY, -INFINITY, 0.0f, 0.0f};
      if (peer < blocks)
        t = {peer_f32(at, peer), peer_f32(at + 4, peer), peer_f32(at + 8, peer), peer_f32(at + 12, peer)};
      warp_combine<8>(t);
      if constexpr (kTop) {
        if (rank == 0) {
          const uint32_t best = ptx::smem_addr(sh.best);
          const int n = static_cast<int>(blocks) * a.top_k;
          for (uint32_t b = tid / 32; b < blocks; b += kWarps)
            for (int i = tid % 32; i < a.top_k; i += 32)
              sh.list[b * a.top_k + i] = peer_u64(best + 8u * i, b);
          compute_sync<kThreads>();
          rank_keys<kThreads>(sh.list, n, a.top_k, sh.best);
          compute_sync<kThreads>();
        }
      }
    }
    const bool slow = t.m > -INFINITY && t.m < INFINITY && !(t.m > Fast<T>::kLow && t.m < Fast<T>::kHigh);
    if (slow && rank == 0) {  // a cluster's first block sums the whole row
      Stats u = {t.m, 0.0f, 0.0f, 0.0f};
      slow_sums<T, kThreads>(row, 0, row.vectors, tid < row.edges() ? row.edge_column(tid) : -1, t.m, u);
      compute_sync<kThreads>();  // the last row's sums have been read
      t = block_stats(u, sh, turn & 1);
    }
    if constexpr (kCluster) {  // no block leaves while another reads its memory
      ptx::cluster_arrive();
      if (rank != 0) {
        ptx::cluster_wait();
        return;
      }
    }
    if (!writer && !(kTop && tid < a.top_k)) continue;
    // log p and H are taken from the largest element, whose own term e_m the
    // sums hold exactly: a row with one possible token has log p = 0, H = 0.
    const float t_m = slow ? 0.0f : fmaf(t.m, kLog2e, -t.n);
    const float e_m = exp2_approx(t_m);
    const float log_s = log2f(t.s / e_m);
    auto log_p = [&](float x) {
      // The difference in the logits' own base: x L overflows near the type's lowest value.
      return x == -INFINITY ? x : x - t.m - log_s * kLn2;
    };
    // lse = m + ln s as two floats: beside a large m the sum's logarithm is in
    // the second one.
    const float ln_s = __fmul_rn(log_s, kLn2);
    float lse = __fadd_rn(t.m, ln_s);
    const float taken = __fsub_rn(lse, t.m);  // ln s as far as lse holds it
    float low = __fadd_rn(__fsub_rn(t.m, __fsub_rn(lse, taken)), __fsub_rn(ln_s, taken));
    float h = t.s == e_m ? 0.0f : (log_s + (t_m - t.w / t.s)) * kLn2;
    bool none = false;
    if (t.m == -INFINITY) {  // all masked: nothing is possible, and nothing to choose between
      lse = -INFINITY;
      low = h = 0.0f;
    } else if (!(t.m < INFINITY)) {  // NaN or +inf: no distribution
      lse = low = h = NAN;
      none = true;
    }
    if (writer) {
      if (a.lse) a.lse[r] = lse;
      if (a.lse_low) a.lse_low[r] = low;
      if (a.entropy) a.entropy[r] = h;
      if (a.tokens && a.logprobs) {
        float lp = 0.0f;  // negative: the position does not count
        if (token >= a.vocab)
          lp = NAN;
        else if (token >= 0)
          lp = none && token_x != -INFINITY ? NAN : log_p(token_x);
        a.logprobs[r] = lp;
      }
    }
    if constexpr (kTop) {
      if (tid < a.top_k) {
        const uint64_t key = sh.best[tid];
        const float x = value_of(static_cast<uint32_t>(key >> 32));
        a.top_ids[r * a.top_k + tid] = 0xffffffffu - static_cast<uint32_t>(key);
        a.top_logprobs[r * a.top_k + tid] = none && x != -INFINITY ? NAN : log_p(x);
      }
    }
  }
  if constexpr (kCluster) {
    __syncwarp();
    ptx::cluster_wait();
  }
}

// dx_j = gl ([j = token] - p_j) - gh p_j (log p_j + H): one read of the
// logits, one write of their gradient.  log p_j = x_j - lse with lse in two
// floats: in one, rounded to |m| 2^-24, all p_j of a row of 1e6 were 3 % off,
// and those of a row of the type's lowest value 1 instead of 1 / n.  Grid: steps of a row, rows.  Where
// the two start at different offsets from a 16-byte boundary, elements go
// one by one.
template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kBwdThreads) logprobs_backward_kernel(const LpArgs a, int chunks) {
  constexpr int kN = Vec<T>::kN;
  ptx::pdl_wait_prior_grid();
  const int64_t r = blockIdx.x / chunks;
  const int chunk = static_cast<int>(blockIdx.x - r * chunks);
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, a.vocab);
  T* out = static_cast<T*>(a.d_logits) + r * a.ldd;
  const int64_t token = a.tokens ? a.tokens[r] : -1;
  const float gl = token >= 0 && a.d_logprobs ? a.d_logprobs[r] : 0.0f;
  const float gh = kEntropy ? a.d_entropy[r] : 0.0f;
  const float lse = a.lse[r], low = a.lse_low ? a.lse_low[r] : 0.0f;
  const float h = kEntropy ? a.entropy[r] : 0.0f;
  auto gradient = [&](float x) {
    const float lp = x == -INFINITY ? x : x - lse - low;  // an all-masked row: lse is -inf too
    const float p = exp2_approx(lp * kLog2e);
    // p (log p + H) is 0 where p is.
    return kEntropy ? -p * fmaf(gh, fmaxf(lp, kExpCut) + h, gl) : -p * gl;
  };
  if (chunk == 0 && static_cast<int>(threadIdx.x) < row.edges()) {
    const int c = row.edge_column(threadIdx.x);
    out[c] = Vec<T>::put(gradient(Vec<T>::get(row.p[c])) + (c == token ? gl : 0.0f));
  }
  const bool same = (reinterpret_cast<uintptr_t>(out + row.head) & 15u) == 0;
  const int base = chunk * kLpUnroll * kBwdThreads + threadIdx.x;
  uint4 w[kLpUnroll];
#pragma unroll
  for (int u = 0; u < kLpUnroll; ++u)
    if (base + u * kBwdThreads < row.vectors) w[u] = __ldcs(row.at(base + u * kBwdThreads));
#pragma unroll
  for (int u = 0; u < kLpUnroll; ++u) {
    const int v = base + u * kBwdThreads;
    if (v >= row.vectors) break;
    float x[kN];
    Vec<T>::unpack(w[u], x);
    const int c0 = row.column(v);
#pragma unroll
    for (int j = 0; j < kN; ++j) x[j] = gradient(x[j]);
    if (token >= c0 && token < c0 + kN) {
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (c0 + j == token) x[j] += gl;
    }
    if (same) {
      __stcs(reinterpret_cast<uint4*>(out + c0), Vec<T>::pack(x));
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) out[c0 + j] = Vec<T>::put(x[j]);
    }
  }
}

template <typename... P, typename... A>
cudaError_t launch_rows(void (*kernel)(P...), int64_t grid, int threads, size_t smem, int cluster,
                        cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
cudaError_t forward(const LpArgs& a, int64_t grid, int cluster, cudaStream_t stream) {
  if (cluster > 1)
    return launch_rows(a.top_k > 0 ? logprobs_kernel<T, true, kShareThreads>
                                   : logprobs_kernel<T, false, kShareThreads>,
                       grid, kShareThreads + 32, kLpSmem<kShareThreads>, cluster, stream, a);
  return launch_rows(a.top_k > 0 ? logprobs_kernel<T, true, kRowThreads>
                                 : logprobs_kernel<T, false, kRowThreads>,
                     grid, kRowThreads + 32, kLpSmem<kRowThreads>, 1, stream, a);
}

template <typename T>
cudaError_t backward(const LpArgs& a, cudaStream_t stream) {
  const int chunks = static_cast<int>(std::max<int64_t>(1, ceil_div(a.vocab / Vec<T>::kN, kLpUnroll * kBwdThreads)));
  return launch_rows(a.d_entropy ? logprobs_backward_kernel<T, true> : logprobs_backward_kernel<T, false>,
                     a.rows * chunks, kBwdThreads, 0, 1, stream, a, chunks);
}

size_t elem_bytes(gemm_in_t t) { return t == GEMM_IN_F32 ? 4 : 2; }

gemm_status_t check(const gemm_ops* ops, const gemm_logprobs_args_t* g, bool bwd) {
  if (!ops || !g) return ops_fail(GEMM_ERR_INVALID_ARG, "ops or args is NULL");
  if (g->rows < 0 || g->vocab < 1)
    return ops_fail(GEMM_ERR_INVALID_ARG, "rows %lld < 0 or vocab %lld < 1", (long long)g->rows,
                    (long long)g->vocab);
  // Columns are counted in 32 bits, the gradient's blocks (at most one for
  // every 4096 columns of a row) in the grid's 31.
  if (g->vocab > kOpsMaxDim / 2 || g->rows > kOpsMaxDim ||
      g->rows * (1 + g->vocab / (4 * kLpUnroll * kBwdThreads)) > kOpsMaxDim)
    return ops_fail(GEMM_ERR_INVALID_ARG, "too many rows or columns");
  if (g->dtype != GEMM_IN_F16 && g->dtype != GEMM_IN_BF16 && g->dtype != GEMM_IN_F32)
    return ops_fail(GEMM_ERR_INVALID_ARG, "dtype %d out of range", static_cast<int>(g->dtype));
  if (g->ld < g->vocab) return ops_fail(GEMM_ERR_INVALID_ARG, "ld %lld < vocab", (long long)g->ld);
  if (reinterpret_cast<uintptr_t>(g->logits) % elem_bytes(g->dtype))
    return ops_fail(GEMM_ERR_INVALID_ARG, "logits are not aligned to their elements");
  if (!bwd) {
    if (g->top_k < 0 || g->top_k > kMaxTopK || g->top_k > g->vocab)
      return ops_fail(GEMM_ERR_INVALID_ARG, "top_k %d outside [0, min(%d, vocab)]", g->top_k, kMaxTopK);
  } else {
    if (g->ldd < g->vocab) return ops_fail(GEMM_ERR_INVALID_ARG, "ldd %lld < vocab", (long long)g->ldd);
    if (reinterpret_cast<uintptr_t>(g->d_logits) % elem_bytes(g->dtype))
      return ops_fail(GEMM_ERR_INVALID_ARG, "d_logits is not aligned to its elements");
  }
  if (g->rows == 0) return GEMM_OK;
  if (!g->logits) return ops_fail(GEMM_ERR_INVALID_ARG, "logits is NULL");
  if (!bwd) {
    if (g->top_k > 0 && (!g->top_ids || !g->top_logprobs))
      return ops_fail(GEMM_ERR_INVALID_ARG, "top_ids or top_logprobs is NULL");
    if (g->logprobs && !g->tokens) return ops_fail(GEMM_ERR_INVALID_ARG, "logprobs without tokens");
  } else {
    if (!g->d_logits || !g->lse) return ops_fail(GEMM_ERR_INVALID_ARG, "d_logits or lse is NULL");
    if (g->d_logprobs && !g->tokens) return ops_fail(GEMM_ERR_INVALID_ARG, "d_logprobs without tokens");
    if (g->d_entropy && !g->entropy) return ops_fail(GEMM_ERR_INVALID_ARG, "d_entropy without entropy");
    // In place is fine, anything in between is not.
    const uintptr_t x = reinterpret_cast<uintptr_t>(g->logits), d = reinterpret_cast<uintptr_t>(g->d_logits);
    const size_t nx = ((g->rows - 1) * g->ld + g->vocab) * elem_bytes(g->dtype);
    const size_t nd = ((g->rows - 1) * g->ldd + g->vocab) * elem_bytes(g->dtype);
    if (x < d + nd && d < x + nx && !(x == d && g->ld == g->ldd))
      return ops_fail(GEMM_ERR_INVALID_ARG, "d_logits overlaps the logits without being them");
  }
  return GEMM_OK;
}

LpArgs kernel_args(const gemm_ops* ops, const gemm_logprobs_args_t* g) {
  LpArgs a{};
  a.rows = g->rows;
  a.status = ops->d_status;
  a.timeout_ns = ops->timeout_ns;
  a.inject_fault = ops->debug_fault;
  a.logits = g->logits;
  a.ld = g->ld;
  a.vocab = static_cast<int>(g->vocab);
  a.top_k = g->top_k;
  a.tokens = g->tokens;
  a.logprobs = g->logprobs;
  a.entropy = g->entropy;
  a.lse = g->lse;
  a.lse_low = g->lse_low;
  a.top_logprobs = g->top_logprobs;
  a.top_ids = g->top_ids;
  a.d_logprobs = g->d_logprobs;
  a.d_entropy = g->d_entropy;
  a.d_logits = g->d_logits;
  a.ldd = g->ldd;
  return a;
}

}  // namespace

namespace spgemm {
// More shared memory than a kernel gets by default (per device, once).
template <typename T, int kThreads>
static cudaError_t set_smem_of() {
  const int bytes = static_cast<int>(kLpSmem<kThreads>);
  const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<T, false, kThreads>, attr, bytes);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(logprobs_kernel<T, true, kThreads>, attr, bytes);
}
template <typename T>
static cudaError_t set_smem_both() {
  const cudaError_t e = set_smem_of<T, kRowThreads>();
  return e != cudaSuccess ? e : set_smem_of<T, kShareThreads>();
}

cudaError_t logprobs_set_smem() {
  cudaError_t e = set_smem_both<float>();
  if (e == cudaSuccess) e = set_smem_both<__nv_bfloat16>();
  if (e == cudaSuccess) e = set_smem_both<__half>();
  return e;
}
}  // namespace spgemm

extern "C" {

gemm_status_t gemm_token_logprobs(gemm_ops_t* ops, const gemm_logprobs_args_t* args, void* stream_handle) {
  ops_fail(GEMM_OK, "%s", "");
  const gemm_status_t st = check(ops, args, false);
  if (st != GEMM_OK || args->rows == 0) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  // Few rows: each is shared by a cluster of blocks, as many as keep one
  // chunk of vectors each, until the SMs are covered.
  const int64_t chunks = ceil_div(args->vocab * static_cast<int64_t>(elem_bytes(args->dtype)), kChunkBytes<kShareThreads>);
  int cluster = 1;
  while (cluster < 8 && args->rows * cluster * 2 <= ops->sm_count && cluster < chunks) cluster *= 2;
  const int64_t grid = cluster > 1 ? args->rows * cluster
                                   : std::min<int64_t>(args->rows, static_cast<int64_t>(ops->sm_count) * kRowBlocks);
  const LpArgs a = kernel_args(ops, args);
  cudaError_t e;
  if (args->dtype == GEMM_IN_F32)
    e = forward<float>(a, grid, cluster, stream);
  else if (args->dtype == GEMM_IN_BF16)
    e = forward<__nv_bfloat16>(a, grid, cluster, stream);
  else
    e = forward<__half>(a, grid, cluster, stream);
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "log probability launch");
}

gemm_status_t gemm_token_logprobs_backward(gemm_ops_t* ops, const gemm_logprobs_args_t* args,
                                           void* stream_handle) {
  ops_fail(GEMM_OK, "%s", "");
  const gemm_status_t st = check(ops, args, true);
  if (st != GEMM_OK || args->rows == 0) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  const LpArgs a = kernel_args(ops, args);
  cudaError_t e;
  if (args->dtype == GEMM_IN_F32)
    e = backward<float>(a, stream);
  else if (args->dtype == GEMM_IN_BF16)
    e = backward<__nv_bfloat16>(a, stream);
  else
    e = backward<__half>(a, stream);
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "log probability gradient launch");
}

}  // extern "C"
