// orthogonal.cu -- the orthogonalised update by Newton-Schulz products.
//
// Matrices with a short side of at most 256 that fit a cluster's shared memory
// take one launch (orthogonal_small.cu).  The others:
//
// Two passes over G normalise it: the sum of squares (one partial per block),
// then X = 2^8 G / max(|G|, eps) in fp16 (every block adds the partials in the
// same order).  Each step is three block products: A = X X^T and B = b A + c
// A^2 on the tiles on and above the diagonal only, and X' = a X + B X.  On
// matrices with more rows than columns the products use
// X^T X and X B instead, reading X as it lies.
//
// fp16 for the iterates: the step's map multiplies errors along small
// singular values by up to a = 3.4 each time; with bf16's 8 bits five steps
// end 1.1e-2 (relative, Frobenius) from exact arithmetic, with fp16's 11 bits
// 1.3e-3, below the bf16 result's own rounding (1.7e-3).  The factor 2^8
// lifts the elements of a normalised matrix (1 / sqrt(m n) in the mean) out
// of fp16's subnormal range; elements stay below 2^8 x 1.3.
//
// B's diagonal stays in fp32 beside it (X' = (a I + D) X + (B - D) X): near
// the end B approaches -2.7 I and X' is 0.7 X, the difference of 3.4 X and 2.7
// X, so that a rounding of the diagonal counts four times; and the rows of a
// matrix far from square have nearly equal norms and the diagonal's elements
// one common rounding error.  With the diagonal in fp16 64 x 7608 ended 2.8e-3
// from exact and 256 x 640 2.1e-3; so 2.0e-3 and 1.9e-3, of which 1.66e-3 is
// the result's rounding.  It costs 0 to 6 % (tall 4097 x 1000 226 -> 236 us,
// 2048 x 8192 unchanged).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ops_internal.h"
#include "orthogonal_load.cuh"
#include "orthogonal_small.h"
#include "ptx.cuh"

using namespace spgemm;

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormVecs = 4;       // 8-element vectors per thread and step
constexpr int kNormStep = kNormThreads * kNormVecs;
constexpr int kNormBlocks = 608;   // at most, over the batch: four per SM

struct NormArgs {
  const void* g;
  int64_t m, n, ld, batch_stride;
  int64_t per;         // vectors of 8 elements in a row (the last may be cut)
  int64_t vectors;     // in a matrix
  int aligned;         // vectors of 8 elements may be loaded whole
  double* partial;     // batch x gridDim.x
  uint16_t* x;
  int64_t ldx;
  float eps;
  int* flags;          // zeroed for the products (BlockScratch)
  int flag_count;
};

// Row and first column of a matrix's vector v.
__device__ __forceinline__ void place(const NormArgs& a, int64_t v, int64_t& r, int64_t& c) {
  r = v < (int64_t{1} << 31) ? static_cast<uint32_t>(v) / static_cast<uint32_t>(a.per) : v / a.per;
  c = (v - r * a.per) * 8;
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) sum_squares_kernel(const NormArgs a) {
  __shared__ double shared[kNormThreads / 32];
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < a.flag_count; i += kNormThreads) a.flags[i] = 0;
  const T* g = static_cast<const T*>(a.g) + blockIdx.y * a.batch_stride;
  SquareSum sum;
  auto pass = [&](auto&& add) {
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * kNormStep + threadIdx.x; s < a.vectors;
         s += static_cast<int64_t>(gridDim.x) * kNormStep) {
      float v[kNormVecs][8];
#pragma unroll
      for (int i = 0; i < kNormVecs; ++i) {
        const int64_t at = s + i * kNormThreads;
        int64_t r, c;
        place(a, at < a.vectors ? at : 0, r, c);
        load8<T>(g + r * a.ld, c, at < a.vectors ? a.n : 0, a.aligned != 0, v[i]);
      }
#pragma unroll
      for (int i = 0; i < kNormVecs; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) add(v[i][j]);
    }
  };
  pass([&](float x) { sum.mid = fmaf(x, x, sum.mid); });
  double total = sum.block_total<kNormThreads>(shared);
  if (!__syncthreads_and(threadIdx.x > 0 || plain_sum_holds(total))) {
    sum = SquareSum();
    pass([&](float x) { sum.add<T>(x); });
    total = sum.block_total<kNormThreads>(shared);
  }
  if (threadIdx.x == 0) a.partial[blockIdx.y * gridDim.x + blockIdx.x] = total;
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) normalize_kernel(const NormArgs a, int parts) {
  __shared__ float shared;
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  if (threadIdx.x < 32) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += 32) sum += __ldcg(a.partial + blockIdx.y * parts + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x == 0) shared = half_scale(sum, a.eps);
  }
  __syncthreads();
  const float scale = shared;
  const T* g = static_cast<const T*>(a.g) + blockIdx.y * a.batch_stride;
  uint16_t* x = a.x + blockIdx.y * a.m * a.ldx;
  for (int64_t s = static_cast<int64_t>(blockIdx.x) * kNormStep + threadIdx.x; s < a.vectors;
       s += static_cast<int64_t>(gridDim.x) * kNormStep) {
    float v[kNormVecs][8];
    int64_t r[kNormVecs], c[kNormVecs];
#pragma unroll
    for (int i = 0; i < kNormVecs; ++i) {
      const int64_t at = s + i * kNormThreads;
      place(a, at < a.vectors ? at : 0, r[i], c[i]);
      load8<T>(g + r[i] * a.ld, c[i], at < a.vectors ? a.n : 0, a.aligned != 0, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kNormVecs; ++i)
      if (s + i * kNormThreads < a.vectors) {
        __half2 h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[j] = __floats2half2_rn(v[i][2 * j] * scale * scale, v[i][2 * j + 1] * scale * scale);
        *reinterpret_cast<uint4*>(x + r[i] * a.ldx + c[i]) = *reinterpret_cast<const uint4*>(h);
      }
  }
}

// Launch that may overlap the previous kernel's tail (both kernels wait for
// it before they touch global memory).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kNormThreads, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
cudaError_t normalize(const NormArgs& a, int64_t batch, int blocks, cudaStream_t stream) {
  const dim3 grid(blocks, static_cast<unsigned>(batch), 1);
  cudaError_t e = launch_early(sum_squares_kernel<T>, grid, stream, a);
  if (e == cudaSuccess) e = launch_early(normalize_kernel<T>, grid, stream, a, blocks);
  return e;
}

struct Layout {
  BlockScratch scratch;
  double* norms;
  uint16_t* x[2];
  uint16_t* a;
  uint16_t* b;
  float* diag;
  int64_t diag_batch;
  int64_t np, s, sp;
  int blocks;
  SmallPlan small;
  float* parts;
  uint16_t* gram;
  size_t bytes;
};

Layout layout(const gemm_ops* ops, const gemm_orthogonalize_args_t* g, void* workspace) {
  Layout l{};
  Carver c(workspace);
  l.small = small_newton_plan(ops, g->m, g->n, g->batch);
  if (l.small.rows > 0) {
    l.norms = static_cast<double*>(c.take(l.small.norm_bytes));
    l.parts = static_cast<float*>(c.take(l.small.part_bytes));
    l.gram = static_cast<uint16_t*>(c.take(l.small.gram_bytes));
    l.bytes = c.used;
    return l;
  }
  l.np = round8(g->n);
  l.s = std::min(g->m, g->n);
  l.sp = round8(l.s);
  const int64_t steps = ceil_div(g->m * (l.np / 8), kNormStep);
  l.blocks = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(steps, kNormBlocks / std::max<int64_t>(1, std::min<int64_t>(g->batch, kNormBlocks)))));
  const size_t x = static_cast<size_t>(g->batch) * g->m * l.np * 2;
  const size_t a = static_cast<size_t>(g->batch) * l.s * l.sp * 2;
  l.scratch = take_scratch(ops, c);
  l.norms = static_cast<double*>(c.take(static_cast<size_t>(g->batch) * l.blocks * sizeof(double)));
  l.x[0] = static_cast<uint16_t*>(c.take(x));
  l.x[1] = static_cast<uint16_t*>(c.take(x));
  l.a = static_cast<uint16_t*>(c.take(a));
  l.b = static_cast<uint16_t*>(c.take(a));
  l.diag_batch = ceil_div(l.s, 64) * 64;
  l.diag = static_cast<float*>(c.take(static_cast<size_t>(g->batch) * l.diag_batch * sizeof(float)));
  l.bytes = c.used;
  return l;
}

size_t elem_bytes(gemm_in_t t) { return t == GEMM_IN_F32 ? 4 : 2; }

gemm_status_t check(const gemm_orthogonalize_args_t* g) {
  if (!g) return ops_fail(GEMM_ERR_INVALID_ARG, "args is NULL");
  if (g->batch < 0 || g->m < 0 || g->n < 0)
    return ops_fail(GEMM_ERR_INVALID_ARG, "negative size batch=%lld m=%lld n=%lld", (long long)g->batch,
                    (long long)g->m, (long long)g->n);
  if (g->m > kOpsMaxDim || g->n > kOpsMaxDim || g->batch > 65535)
    return ops_fail(GEMM_ERR_INVALID_ARG, "m or n above 2^31-1, or batch above 65535");
  if (g->dtype != GEMM_IN_F16 && g->dtype != GEMM_IN_BF16 && g->dtype != GEMM_IN_F32)
    return ops_fail(GEMM_ERR_INVALID_ARG, "dtype %d out of range", static_cast<int>(g->dtype));
  if (g->steps < 1 || g->steps > 100)
    return ops_fail(GEMM_ERR_INVALID_ARG, "steps %d outside [1, 100]", g->steps);
  if (!(g->eps > 0.0f) || !std::isfinite(g->a) || !std::isfinite(g->b) || !std::isfinite(g->c))
    return ops_fail(GEMM_ERR_INVALID_ARG, "eps must be positive and a, b, c finite");
  if (g->batch == 0 || g->m == 0 || g->n == 0) return GEMM_OK;
  if (!g->g || !g->out) return ops_fail(GEMM_ERR_INVALID_ARG, "g or out is NULL");
  if (g->ldg < g->n) return ops_fail(GEMM_ERR_INVALID_ARG, "ldg %lld < n", (long long)g->ldg);
  if (g->batch > 1 && g->batch_stride < 0)
    return ops_fail(GEMM_ERR_INVALID_ARG, "negative batch_stride");
  if ((reinterpret_cast<uintptr_t>(g->g) % elem_bytes(g->dtype)) || (reinterpret_cast<uintptr_t>(g->out) & 1u))
    return ops_fail(GEMM_ERR_INVALID_ARG, "g or out is not aligned to its elements");
  return GEMM_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

}  // namespace

extern "C" {

gemm_status_t gemm_orthogonalize_workspace(gemm_ops_t* ops, const gemm_orthogonalize_args_t* args,
                                           size_t* bytes) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops || !bytes) return ops_fail(GEMM_ERR_INVALID_ARG, "NULL argument");
  const gemm_status_t st = check(args);
  if (st == GEMM_OK) *bytes = layout(ops, args, nullptr).bytes;
  return st;
}

gemm_status_t gemm_orthogonalize(gemm_ops_t* ops, const gemm_orthogonalize_args_t* args,
                                 void* workspace, size_t workspace_bytes, void* stream_handle) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops) return ops_fail(GEMM_ERR_INVALID_ARG, "ops is NULL");
  gemm_status_t st = check(args);
  if (st != GEMM_OK || args->batch == 0 || args->m == 0 || args->n == 0) return st;
  const int64_t m = args->m, n = args->n, batch = args->batch;
  Layout l = layout(ops, args, workspace);
  if ((!workspace && l.bytes > 0) || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < l.bytes)
    return ops_fail(GEMM_ERR_INVALID_ARG, "workspace NULL, not 256-byte aligned or below %zu bytes", l.bytes);
  const size_t g_bytes = (static_cast<size_t>(batch - 1) * (batch > 1 ? args->batch_stride : 0) +
                          static_cast<size_t>(m - 1) * args->ldg + n) * elem_bytes(args->dtype);
  const size_t o_bytes = static_cast<size_t>(batch) * m * n * 2;
  if (overlap(args->out, o_bytes, args->g, g_bytes) || overlap(workspace, l.bytes, args->g, g_bytes) ||
      overlap(workspace, l.bytes, args->out, o_bytes))
    return ops_fail(GEMM_ERR_INVALID_ARG, "g, out and the workspace must not overlap");
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);

  const int64_t vec = 16 / static_cast<int64_t>(elem_bytes(args->dtype));
  const bool aligned = (reinterpret_cast<uintptr_t>(args->g) & 15u) == 0 && args->ldg % vec == 0 &&
                       (batch == 1 || args->batch_stride % vec == 0);
  if (l.small.rows > 0) {
    SmallNewton p{};
    p.g = args->g;
    p.ld = args->ldg;
    p.g_batch = batch > 1 ? args->batch_stride : 0;
    p.type = args->dtype;
    p.tall = m > n;
    p.aligned = aligned;
    p.s = static_cast<int>(std::min(m, n));
    p.l = static_cast<int>(std::max(m, n));
    p.batch = static_cast<int>(batch);
    p.steps = args->steps;
    p.a = args->a;
    p.b = args->b;
    p.c = args->c;
    p.eps = args->eps;
    p.out = static_cast<uint16_t*>(args->out);
    p.norms = l.norms;
    p.parts = l.parts;
    p.gram = l.gram;
    const cudaError_t small = small_newton_launch(ops, l.small, p, stream);
    return small == cudaSuccess ? GEMM_OK : ops_cuda_fail(small, "on-chip iteration launch");
  }

  NormArgs na{};
  na.g = args->g;
  na.m = m;
  na.n = n;
  na.ld = args->ldg;
  na.batch_stride = batch > 1 ? args->batch_stride : 0;
  na.per = l.np / 8;
  na.vectors = m * na.per;
  na.aligned = aligned;
  na.partial = l.norms;
  na.x = l.x[0];
  na.ldx = l.np;
  na.eps = args->eps;
  na.flags = l.scratch.flags;
  na.flag_count = l.scratch.count;
  l.scratch.zeroed = true;
  cudaError_t e;
  if (args->dtype == GEMM_IN_F32)
    e = normalize<float>(na, batch, l.blocks, stream);
  else if (args->dtype == GEMM_IN_BF16)
    e = normalize<__nv_bfloat16>(na, batch, l.blocks, stream);
  else
    e = normalize<__half>(na, batch, l.blocks, stream);
  if (e != cudaSuccess) return ops_cuda_fail(e, "normalisation launch");

  const bool tall = m > n;
  Matrix X{l.x[0], m, n, l.np, m * l.np}, Y{l.x[1], m, n, l.np, m * l.np};
  const Matrix A{l.a, l.s, l.s, l.sp, l.s * l.sp}, B{l.b, l.s, l.s, l.sp, l.s * l.sp};
  const float inv = 1.0f / kIterateScale;
  for (int it = 0; it < args->steps; ++it) {
    BlockProblem p;
    p.batch = batch;
    p.M = p.N = l.s;
    p.symmetric = true;
    p.kind = tall ? BlockProblem::kTN : BlockProblem::kNT;  // A = X^T X or X X^T
    p.K = tall ? m : n;
    p.a = p.b = X;
    p.alpha = inv * inv;
    p.out0 = A;  // the padded row is the iterate's own
    p.out0.cols = l.sp;
    st = run_block(ops, p, l.scratch, stream);
    if (st != GEMM_OK) return st;

    p.kind = BlockProblem::kDiagOut;  // B = c A A^T + b A
    p.K = l.s;
    p.a = p.b = p.d = A;
    p.alpha = args->c;
    p.beta = args->b;
    p.out0 = B;
    p.out0.cols = l.sp;
    p.diag = l.diag;
    p.diag_batch = l.diag_batch;
    st = run_block(ops, p, l.scratch, stream);
    if (st != GEMM_OK) return st;

    const bool last = it + 1 == args->steps;
    p.symmetric = false;
    p.M = m;
    p.N = n;
    if (tall) {  // X B, B symmetric
      p.kind = BlockProblem::kDiagCols;
      p.a = X;
      p.b = B;
    } else {
      p.kind = BlockProblem::kDiagRows;
      p.a = B;
      p.b = X;
    }
    p.d = X;
    p.alpha = last ? inv : 1.0f;
    p.beta = last ? inv * args->a : args->a;
    p.out_bf16 = last;
    p.out0 = last ? Matrix{args->out, m, n, n, m * n} : Matrix{Y.ptr, m, l.np, l.np, m * l.np};
    st = run_block(ops, p, l.scratch, stream);
    if (st != GEMM_OK) return st;
    std::swap(X, Y);
  }
  return GEMM_OK;
}

}  // extern "C"
