// logprobs.cu -- log probabilities of tokens under rows of logits, with the
// row's entropy and best alternatives, and their gradient.
//
//   m = max x, s = sum e^(x - m), w = sum e^(x - m) (x - m)
//   lse = m + ln s,  log p_t = x_t - lse,  H = ln s - w / s
//
// One pass over the logits, bound by memory: each thread keeps m, s and w of
// its own elements in fp32, rescaled when its maximum grows
//   s' = f s,  w' = f (w + (m - m') s),  f = e^(m - m')
// and the block (or, for few rows, the cluster of blocks that shares a row)
// combines them in a fixed order.  Exponents are taken base 2 of
// (x - m) log2 e, the difference first, so large logits lose nothing; the
// exponent is cut at -200 (2^-200 is 0 in fp32), which keeps masked logits
// (-inf, or the type's lowest value) from making 0 x inf.
//
// Alternatives.  While streaming, each thread also keeps the largest of its
// elements and the first 16-byte vector that holds it.  The k-th largest of
// these is a lower bound of the row's k-th largest element, so only the
// threads at or above it (about k of them) have anything to offer: their
// vectors are read again (from L2), the few elements at or above the bound
// are collected and ranked.  A key of (value, index) orders equal values by
// index, and the bound is a pair too, so a row of equal logits offers no
// more than the first k vectors.  A row that offers more than the list holds
// (its largest elements all in a few threads' vectors) is searched k times.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ops_internal.h"
#include "ptx.cuh"

using namespace spgemm;

namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpUnroll = 4;          // vectors a thread has in flight
constexpr int kLpCandidates = 1024;
constexpr int kMaxTopK = GEMM_LOGPROBS_MAX_TOP_K;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kExpCut = -200.0f;

struct LpArgs {
  const void* logits;
  int64_t ld;
  int vocab;
  int top_k;
  const int64_t* tokens;
  float *logprobs, *entropy, *lse, *top_logprobs;
  int64_t* top_ids;
  // backward
  const float *d_logprobs, *d_entropy;
  void* d_logits;
  int64_t ldd;
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
// +inf < NaN (any).
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
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

// A row of logits as 16-byte vectors from the aligned address at or before
// its first element: element j of vector v is column v kN + j - shift.  The
// first and last vector may hold columns that do not exist; those are read
// one element at a time, and -inf stands in their place (and for a vector
// -1, which no row has).
template <typename T>
struct Row {
  static constexpr int kN = Vec<T>::kN;
  const T* p;
  int vocab, shift, vectors;
  __device__ Row(const T* row, int v) : p(row), vocab(v) {
    shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    vectors = static_cast<int>((static_cast<int64_t>(v) + shift + kN - 1) / kN);
  }
  __device__ __forceinline__ bool whole(int v) const {
    const int64_t c = static_cast<int64_t>(v) * kN - shift;
    return c >= 0 && c + kN <= vocab;
  }
  __device__ __forceinline__ void load_edge(int v, float (&x)[kN]) const {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int64_t c = static_cast<int64_t>(v) * kN + j - shift;
      x[j] = v >= 0 && c >= 0 && c < vocab ? Vec<T>::get(p[c]) : -INFINITY;
    }
  }
  __device__ __forceinline__ const uint4* at(int v) const {
    return reinterpret_cast<const uint4*>(p + (static_cast<int64_t>(v) * kN - shift));
  }
  __device__ __forceinline__ void load(int v, float (&x)[kN]) const {
    if (whole(v))
      Vec<T>::unpack(__ldg(at(v)), x);
    else
      load_edge(v, x);
  }
};

struct Stats {
  float m, s, w;  // w in units of ln 2
};

__device__ __forceinline__ Stats combine(const Stats& a, const Stats& b) {
  Stats r;
  r.m = max_nan(a.m, b.m);
  const float da = fmaxf((a.m - r.m) * kLog2e, kExpCut), db = fmaxf((b.m - r.m) * kLog2e, kExpCut);
  const float fa = exp2_approx(da), fb = exp2_approx(db);
  r.s = fa * a.s + fb * b.s;
  r.w = fa * fmaf(da, a.s, a.w) + fb * fmaf(db, b.s, b.w);
  return r;
}

__device__ __forceinline__ Stats shuffle_xor(const Stats& a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
          __shfl_xor_sync(0xffffffffu, a.w, o)};
}

struct LpShared {
  Stats warp[kLpWarps];
  Stats block;
  int count;
  uint64_t best[kMaxTopK];          // this block's best keys, best first
  uint64_t list[kLpCandidates];
  uint64_t reduce[kLpWarps];
};

__device__ __forceinline__ uint64_t key_of(float x, int column) {
  return (static_cast<uint64_t>(order_of(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(column));
}

// Writes the k largest of sh.list[0, n) to out, in order, and 0 in places
// that no key takes.
__device__ __forceinline__ void rank_keys(const uint64_t* list, int n, int k, uint64_t* out) {
  for (int i = threadIdx.x; i < k; i += kLpThreads)
    if (i >= n) out[i] = 0;
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const uint64_t mine = list[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[j] > mine ? 1 : 0;
    if (rank < k) out[rank] = mine;
  }
}

// The k best of the columns this block streamed (vectors v0 + i kLpThreads +
// thread), to sh.best.  top: order of this thread's largest element (0: it
// has none); top_v: the first vector that holds it.
template <typename T>
__device__ void block_top(const Row<T>& row, int v0, int v1, int k, uint32_t top, int top_v,
                          LpShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31;
  // The bound: the largest order that at least k threads reach (0 if fewer
  // have anything), or one that k to 2 k threads reach.
  uint32_t lo = 0, hi = 0xffffffffu;
  int reach = kLpThreads;
  if (__syncthreads_count(top == 0xffffffffu) >= k) lo = hi;  // NaNs
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const int c = __syncthreads_count(top >= mid);
    if (c >= k) {
      lo = mid;
      reach = c;
      if (c <= 2 * k) break;
    } else {
      hi = mid;
    }
  }
  // Many threads end on the same value: of those, the first vectors only.
  int last_v = v1;
  if (lo > 0 && reach > 2 * k) {
    const int want = k - __syncthreads_count(top > lo);
    int a = v0 - 1, b = v1;  // count(top_v <= a) < want <= count(top_v <= b)
    while (b - a > 1) {
      const int mid = a + (b - a) / 2;
      if (__syncthreads_count(top == lo && top_v <= mid) >= want)
        b = mid;
      else
        a = mid;
    }
    last_v = b;
  }
  if (tid == 0) sh.count = 0;
  __syncthreads();
  const bool offers = top > lo || (top == lo && top != 0 && top_v <= last_v);
  uint32_t ask = __ballot_sync(0xffffffffu, offers);
  while (ask) {  // the warp reads one offering thread's vectors together
    const int src = __ffs(ask) - 1;
    ask &= ask - 1;
    for (int v = v0 + (tid - lane + src) + lane * kLpThreads; v < v1; v += 32 * kLpThreads) {
      float x[Row<T>::kN];
      row.load(v, x);
#pragma unroll
      for (int j = 0; j < Row<T>::kN; ++j) {
        const int64_t c = static_cast<int64_t>(v) * Row<T>::kN + j - row.shift;
        const uint32_t o = order_of(x[j]);
        if (c >= 0 && c < row.vocab && (o > lo || (o == lo && v <= last_v))) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kLpCandidates) sh.list[at] = key_of(x[j], static_cast<int>(c));
        }
      }
    }
  }
  __syncthreads();
  const int n = sh.count;
  if (n <= kLpCandidates) {
    rank_keys(sh.list, n, k, sh.best);
    __syncthreads();
    return;
  }
  // More than the list holds: the largest key below the last one, k times.
  uint64_t below = ~0ull;
  for (int i = 0; i < k; ++i) {
    uint64_t best = 0;
    for (int v = v0 + tid; v < v1; v += kLpThreads) {
      float x[Row<T>::kN];
      row.load(v, x);
#pragma unroll
      for (int j = 0; j < Row<T>::kN; ++j) {
        const int64_t c = static_cast<int64_t>(v) * Row<T>::kN + j - row.shift;
        if (c < 0 || c >= row.vocab) continue;
        const uint64_t key = key_of(x[j], static_cast<int>(c));
        if (key < below && key > best) best = key;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
      best = other > best ? other : best;
    }
    if (lane == 0) sh.reduce[tid >> 5] = best;
    __syncthreads();
    for (int j = 0; j < kLpWarps; ++j) best = sh.reduce[j] > best ? sh.reduce[j] : best;
    if (tid == 0) sh.best[i] = best;
    below = best;
    __syncthreads();
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

// One row per cluster (of one block or more; see launch below).
template <typename T, bool kTop>
__global__ void __launch_bounds__(kLpThreads, 2) logprobs_kernel(const LpArgs a) {
  constexpr int kN = Vec<T>::kN;
  __shared__ LpShared sh;
  const uint32_t blocks = cluster_size();
  const uint32_t rank = blocks > 1 ? ptx::cluster_ctarank() : 0u;
  const int64_t r = blockIdx.x / blocks;
  const int tid = threadIdx.x;
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, a.vocab);
  const int v0 = static_cast<int>(static_cast<int64_t>(row.vectors) * rank / blocks);
  const int v1 = static_cast<int>(static_cast<int64_t>(row.vectors) * (rank + 1) / blocks);

  Stats t = {-INFINITY, 0.0f, 0.0f};
  uint32_t top = 0;
  int top_v = 0;
  for (int base = v0 + tid; base < v1; base += kLpUnroll * kLpThreads) {
    uint4 w[kLpUnroll];
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      const int v = base + u * kLpThreads;
      if (v < v1 && row.whole(v)) {
        w[u] = __ldg(row.at(v));
      } else {
        float x[kN];
        row.load_edge(v < v1 ? v : -1, x);
        w[u] = Vec<T>::pack(x);
      }
    }
    float m = t.m;
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      float x[kN];
      Vec<T>::unpack(w[u], x);
      float vm = x[0];
#pragma unroll
      for (int j = 1; j < kN; ++j) vm = max_nan(vm, x[j]);
      if constexpr (kTop) {
        const uint32_t o = order_of(vm);
        if (o > top && base + u * kLpThreads < v1) {
          top = o;
          top_v = base + u * kLpThreads;
        }
      }
      m = max_nan(m, vm);
    }
    const float d = fmaxf((t.m - m) * kLog2e, kExpCut), f = exp2_approx(d);
    t.w = f * fmaf(d, t.s, t.w);
    t.s *= f;
    t.m = m;
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      float x[kN];
      Vec<T>::unpack(w[u], x);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const float e2 = fmaxf((x[j] - m) * kLog2e, kExpCut);
        const float e = exp2_approx(e2);
        t.s += e;
        t.w = fmaf(e, e2, t.w);
      }
    }
  }
  // Block, in a fixed order.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t = combine(t, shuffle_xor(t, o));
  if ((tid & 31) == 0) sh.warp[tid >> 5] = t;
  __syncthreads();
  if (tid < 32) {
    t = sh.warp[tid & (kLpWarps - 1)];
#pragma unroll
    for (int o = kLpWarps / 2; o > 0; o >>= 1) t = combine(t, shuffle_xor(t, o));
    if (tid == 0) sh.block = t;
  }
  if constexpr (kTop) block_top<T>(row, v0, v1, a.top_k, top, top_v, sh);
  __syncthreads();
  t = sh.block;

  if (blocks > 1) {
    ptx::cluster_sync();
    if (rank == 0) {
      const uint32_t at = ptx::smem_addr(&sh.block);
      for (uint32_t b = 1; b < blocks; ++b)
        t = combine(t, Stats{peer_f32(at, b), peer_f32(at + 4, b), peer_f32(at + 8, b)});
      if constexpr (kTop) {
        const uint32_t best = ptx::smem_addr(sh.best);
        const int n = static_cast<int>(blocks) * a.top_k;
        for (int i = tid; i < n; i += kLpThreads)
          sh.list[i] = peer_u64(best + 8u * (i % a.top_k), i / a.top_k);
        __syncthreads();
        rank_keys(sh.list, n, a.top_k, sh.best);
        __syncthreads();
      }
    }
    ptx::cluster_sync();  // no block leaves while another reads its memory
    if (rank != 0) return;
  }
  // Infinite (or NaN) largest logit: no distribution.  All masked: nothing
  // is possible, and there is nothing to choose between.  log p is taken as
  // (x - m) - ln s, which for large logits keeps the digits x - lse loses.
  const float ln_s = logf(t.s);
  float lse = t.m + ln_s, h = ln_s - t.w * kLn2 / t.s;
  if (t.m == -INFINITY) {
    lse = -INFINITY;
    h = 0.0f;
  } else if (!(t.m < INFINITY)) {
    lse = h = NAN;
  }
  if (tid == 0) {
    if (a.lse) a.lse[r] = lse;
    if (a.entropy) a.entropy[r] = h;
    if (a.tokens && a.logprobs) {
      const int64_t token = a.tokens[r];
      float lp = 0.0f;  // negative: the position does not count
      if (token >= a.vocab) {
        lp = NAN;
      } else if (token >= 0) {
        const float x = Vec<T>::get(row.p[token]);
        lp = x == -INFINITY ? x : (x - t.m) - ln_s;
      }
      a.logprobs[r] = lp;
    }
  }
  if constexpr (kTop) {
    if (tid < a.top_k) {
      const uint64_t key = sh.best[tid];
      const float x = value_of(static_cast<uint32_t>(key >> 32));
      a.top_ids[r * a.top_k + tid] = 0xffffffffu - static_cast<uint32_t>(key);
      a.top_logprobs[r * a.top_k + tid] = x == -INFINITY ? x : (x - t.m) - ln_s;
    }
  }
}

// dx_j = gl ([j = token] - p_j) - gh p_j (log p_j + H): one read of the
// logits, one write of their gradient.  Grid: x over steps of a row, y over
// rows.  The two may start at different offsets from a 16-byte boundary
// (then, and at the ends of a row, elements go one by one).
template <typename T>
__global__ void __launch_bounds__(kLpThreads, 2) logprobs_backward_kernel(const LpArgs a, int64_t rows,
                                                                          int chunks) {
  constexpr int kN = Vec<T>::kN;
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  const int64_t r = blockIdx.x / chunks;
  const int chunk = static_cast<int>(blockIdx.x - r * chunks);
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, a.vocab);
  T* out = static_cast<T*>(a.d_logits) + r * a.ldd;
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15u) == (reinterpret_cast<uintptr_t>(row.p) & 15u);
  const int64_t token = a.tokens ? a.tokens[r] : -1;
  const float gl = token >= 0 && a.d_logprobs ? a.d_logprobs[r] : 0.0f;
  const float gh = a.d_entropy ? a.d_entropy[r] : 0.0f;
  const float lse = a.lse[r];
  const float h = a.d_entropy ? a.entropy[r] : 0.0f;
  const int base = chunk * kLpUnroll * kLpThreads + threadIdx.x;
  uint4 w[kLpUnroll];
#pragma unroll
  for (int u = 0; u < kLpUnroll; ++u) {
    const int v = base + u * kLpThreads;
    if (v < row.vectors && row.whole(v)) w[u] = __ldcs(row.at(v));
  }
#pragma unroll
  for (int u = 0; u < kLpUnroll; ++u) {
    const int v = base + u * kLpThreads;
    if (v >= row.vectors) break;
    const bool whole = row.whole(v);
    float x[kN];
    if (whole)
      Vec<T>::unpack(w[u], x);
    else
      row.load_edge(v, x);
    const int64_t c0 = static_cast<int64_t>(v) * kN - row.shift;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const float lp = x[j] == -INFINITY ? -INFINITY : x[j] - lse;
      const float p = exp2_approx(lp * kLog2e);
      // p (log p + H) is 0 where p is.
      x[j] = -p * fmaf(gh, fmaxf(lp, kExpCut) + h, gl);
      if (c0 + j == token) x[j] += gl;
    }
    if (whole && same) {
      __stcs(reinterpret_cast<uint4*>(out + c0), Vec<T>::pack(x));
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (c0 + j >= 0 && c0 + j < a.vocab) out[c0 + j] = Vec<T>::put(x[j]);
    }
  }
}

template <typename... P, typename... A>
cudaError_t launch_rows(void (*kernel)(P...), int64_t grid, int cluster, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kLpThreads, 1, 1);
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
cudaError_t forward(const LpArgs& a, int64_t rows, int cluster, cudaStream_t stream) {
  return a.top_k > 0 ? launch_rows(logprobs_kernel<T, true>, rows * cluster, cluster, stream, a)
                     : launch_rows(logprobs_kernel<T, false>, rows * cluster, cluster, stream, a);
}

template <typename T>
cudaError_t backward(const LpArgs& a, int64_t rows, cudaStream_t stream) {
  const int64_t vectors = ceil_div(a.vocab + Vec<T>::kN - 1, Vec<T>::kN);
  const int chunks = static_cast<int>(ceil_div(vectors, kLpUnroll * kLpThreads));
  return launch_rows(logprobs_backward_kernel<T>, rows * chunks, 1, stream, a, rows, chunks);
}

size_t elem_bytes(gemm_in_t t) { return t == GEMM_IN_F32 ? 4 : 2; }

gemm_status_t check(const gemm_ops* ops, const gemm_logprobs_args_t* g, bool bwd) {
  if (!ops || !g) return ops_fail(GEMM_ERR_INVALID_ARG, "ops or args is NULL");
  if (g->rows < 0 || g->vocab < 1)
    return ops_fail(GEMM_ERR_INVALID_ARG, "rows %lld < 0 or vocab %lld < 1", (long long)g->rows,
                    (long long)g->vocab);
  // Columns are counted in 32 bits, blocks of a row (at most 8, or one per 8192
  // columns) in the grid's 31.
  if (g->vocab > kOpsMaxDim / 2 || g->rows > kOpsMaxDim / 8 ||
      g->rows * ceil_div(g->vocab + 8, 4 * kLpUnroll * kLpThreads) > kOpsMaxDim)
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

LpArgs kernel_args(const gemm_logprobs_args_t* g) {
  LpArgs a{};
  a.logits = g->logits;
  a.ld = g->ld;
  a.vocab = static_cast<int>(g->vocab);
  a.top_k = g->top_k;
  a.tokens = g->tokens;
  a.logprobs = g->logprobs;
  a.entropy = g->entropy;
  a.lse = g->lse;
  a.top_logprobs = g->top_logprobs;
  a.top_ids = g->top_ids;
  a.d_logprobs = g->d_logprobs;
  a.d_entropy = g->d_entropy;
  a.d_logits = g->d_logits;
  a.ldd = g->ldd;
  return a;
}

}  // namespace

extern "C" {

gemm_status_t gemm_token_logprobs(gemm_ops_t* ops, const gemm_logprobs_args_t* args, void* stream_handle) {
  ops_fail(GEMM_OK, "%s", "");
  const gemm_status_t st = check(ops, args, false);
  if (st != GEMM_OK || args->rows == 0) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  // Few rows: each is shared by a cluster of blocks, as many as keep one
  // step of vectors each, until the SMs are covered.
  const int64_t steps = ceil_div(args->vocab * static_cast<int64_t>(elem_bytes(args->dtype)),
                                 16 * kLpUnroll * kLpThreads);
  int cluster = 1;
  while (cluster < 8 && args->rows * cluster * 2 <= ops->sm_count && cluster < steps) cluster *= 2;
  const LpArgs a = kernel_args(args);
  cudaError_t e;
  if (args->dtype == GEMM_IN_F32)
    e = forward<float>(a, args->rows, cluster, stream);
  else if (args->dtype == GEMM_IN_BF16)
    e = forward<__nv_bfloat16>(a, args->rows, cluster, stream);
  else
    e = forward<__half>(a, args->rows, cluster, stream);
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
  const LpArgs a = kernel_args(args);
  cudaError_t e;
  if (args->dtype == GEMM_IN_F32)
    e = backward<float>(a, args->rows, stream);
  else if (args->dtype == GEMM_IN_BF16)
    e = backward<__nv_bfloat16>(a, args->rows, stream);
  else
    e = backward<__half>(a, args->rows, stream);
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "log probability gradient launch");
}

}  // extern "C"
