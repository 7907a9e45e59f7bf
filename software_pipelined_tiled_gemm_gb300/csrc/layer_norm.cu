// layer_norm.cu -- layer norm: argument checks and the choice of the rows' type
// (kernels and launches: layer_norm.cuh).
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "layer_norm.h"
#include "ops_internal.h"

using namespace spgemm;

namespace {

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

// The kernels' shared memory, set by the first layer norm of a handle: with some hundred
// instances it takes 4 ms, which no other operator's first call should.  (Two calls at once
// may both set it.)
cudaError_t set_up(gemm_ops_t* ops) {
  if (ops->layer_norm_ready.load(std::memory_order_acquire)) return cudaSuccess;
  cudaError_t e = layer_norm_set_smem_f16(ops->smem_optin);
  if (e == cudaSuccess) e = layer_norm_set_smem_bf16(ops->smem_optin);
  if (e == cudaSuccess) e = layer_norm_set_smem_f32(ops->smem_optin);
  if (e == cudaSuccess) ops->layer_norm_ready.store(true, std::memory_order_release);
  return e;
}

LayerNormJob job_of(const gemm_layer_norm_args_t* a) {
  LayerNormJob p{};
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

extern "C" {

gemm_status_t gemm_layer_norm(gemm_ops_t* ops, const gemm_layer_norm_args_t* args, void* stream_handle) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops) return ops_fail(GEMM_ERR_INVALID_ARG, "ops is NULL");
  gemm_status_t st = check(args, false);
  if (st == GEMM_OK) st = check_overlap(args, false, nullptr, 0);
  if (st != GEMM_OK || args->rows == 0) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaError_t e = set_up(ops);
  if (e != cudaSuccess) return ops_cuda_fail(e, "layer norm set-up");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  LayerNormJob p = job_of(args);
  p.bias = args->bias;
  p.out = args->y;
  p.eps = args->eps;
  const int64_t per = args->dtype == GEMM_IN_F32 ? 4 : 8;
  const bool vec = p.cols % per == 0 && p.ldx % per == 0 && aligned16({p.x, p.out, p.weight, p.bias});
  const bool wide = args->weight_dtype == GEMM_IN_F32;
  e = args->dtype == GEMM_IN_F32   ? layer_norm_forward_f32(ops, p, vec, wide, stream)
      : args->dtype == GEMM_IN_F16 ? layer_norm_forward_f16(ops, p, vec, wide, stream)
                                   : layer_norm_forward_bf16(ops, p, vec, wide, stream);
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "layer norm launch");
}

gemm_status_t gemm_layer_norm_backward_workspace(gemm_ops_t* ops, const gemm_layer_norm_args_t* args, size_t* bytes) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops || !bytes) return ops_fail(GEMM_ERR_INVALID_ARG, "NULL argument");
  const gemm_status_t st = check(args, true);
  if (st != GEMM_OK) return st;
  *bytes = 0;
  if (args->rows > 0 && (args->dweight || args->dbias))
    *bytes = static_cast<size_t>(layer_norm_backward_blocks(ops, args->rows, args->cols)) * 2 * args->cols * sizeof(float);
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
  cudaError_t e = set_up(ops);
  if (e != cudaSuccess) return ops_cuda_fail(e, "layer norm set-up");
  LayerNormJob p = job_of(args);
  p.dy = args->dy;
  p.lddy = args->lddy;
  p.out = args->dx;
  p.partial = need ? static_cast<float*>(workspace) : nullptr;
  const int64_t per = args->dtype == GEMM_IN_F32 ? 4 : 8;
  const bool vec = p.cols % per == 0 && p.ldx % per == 0 && p.lddy % per == 0 &&
                   aligned16({p.x, p.dy, p.out, p.weight});
  void *dw = args->dweight, *db = args->dbias;
  e = args->dtype == GEMM_IN_F32   ? layer_norm_backward_f32(ops, p, vec, wide, dw, db, stream)
      : args->dtype == GEMM_IN_F16 ? layer_norm_backward_f16(ops, p, vec, wide, dw, db, stream)
                                   : layer_norm_backward_bf16(ops, p, vec, wide, dw, db, stream);
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "layer norm gradient launch");
}

}  // extern "C"
