// ffn.cu -- the gated feed-forward block: argument checks, padded copies of
// operands that need them, and the products of the forward and backward pass.
//
// Forward: one gated product (both projections, the activation and the
// product of the halves) and one plain product.  Backward: dH = dY Wo with
// dG and dU in its epilogue, then dX, dw_in and dw_out as plain products.
#include <cuda_runtime.h>

#include <cstdint>

#include "few_tokens.h"
#include "ops_internal.h"

using namespace spgemm;

namespace {

struct Ffn {
  const gemm_ffn_args_t* a;
  int64_t M, D, I, Ip;
  bool bf16;
  float* pre;
  uint16_t* h;         // M x I, pitch Ip
  uint16_t* dgu;       // backward: M x 2 I, pitch round8(2 I)
  BlockScratch scratch;
  Matrix x, w_in, w_out, dy;
  bool few_first, few_second;  // forward products that go over the weights as they lie (few_tokens.cu)
  PackJobs pack;
};

size_t pre_bytes(int64_t tokens, int64_t inner) {
  return align256(static_cast<size_t>(2) * ceil_div(tokens, 32) * 32 * inner * sizeof(float));
}

gemm_status_t check(const gemm_ffn_args_t* a, bool backward) {
  if (!a) return ops_fail(GEMM_ERR_INVALID_ARG, "args is NULL");
  if (a->tokens < 0 || a->d_model < 1 || a->d_inner < 1)
    return ops_fail(GEMM_ERR_INVALID_ARG, "tokens %lld < 0 or d_model %lld, d_inner %lld < 1",
                    (long long)a->tokens, (long long)a->d_model, (long long)a->d_inner);
  if (a->tokens > kOpsMaxDim || a->d_model > kOpsMaxDim || a->d_inner > kOpsMaxDim / 2)
    return ops_fail(GEMM_ERR_INVALID_ARG, "size above 2^31-1 (d_inner: 2^30-1)");
  if (a->dtype != GEMM_F16 && a->dtype != GEMM_BF16)
    return ops_fail(GEMM_ERR_INVALID_ARG, "dtype %d out of range", static_cast<int>(a->dtype));
  if (a->act != GEMM_ACT_SILU && a->act != GEMM_ACT_GELU_TANH && a->act != GEMM_ACT_RELU)
    return ops_fail(GEMM_ERR_INVALID_ARG, "activation %d out of range", static_cast<int>(a->act));
  if (a->ldx < a->d_model) return ops_fail(GEMM_ERR_INVALID_ARG, "ldx %lld < d_model", (long long)a->ldx);
  if (backward && a->lddy < a->d_model)
    return ops_fail(GEMM_ERR_INVALID_ARG, "lddy %lld < d_model", (long long)a->lddy);
  if (a->tokens > 0) {
    if (!a->x || !a->w_in || !a->w_out) return ops_fail(GEMM_ERR_INVALID_ARG, "x, w_in or w_out is NULL");
    if (backward && (!a->dy || !a->kept)) return ops_fail(GEMM_ERR_INVALID_ARG, "dy or kept is NULL");
    if (!backward && !a->y) return ops_fail(GEMM_ERR_INVALID_ARG, "y is NULL");
  }
  const void* ptrs[] = {a->x, a->w_in, a->w_out, a->y, a->dy, a->dx, a->dw_in, a->dw_out};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 1u)
      return ops_fail(GEMM_ERR_INVALID_ARG, "matrices must be 2-byte aligned");
  if (reinterpret_cast<uintptr_t>(a->kept) & 255u)
    return ops_fail(GEMM_ERR_INVALID_ARG, "kept must be 256-byte aligned");
  return GEMM_OK;
}

// Outputs against inputs and each other.
gemm_status_t check_overlap(const gemm_ffn_args_t* a, bool backward, const void* ws, size_t ws_bytes) {
  const size_t M = a->tokens, D = a->d_model, I = a->d_inner;
  struct Range {
    const void* p;
    size_t n;
    const char* name;
  };
  const size_t nx = M ? ((M - 1) * a->ldx + D) * 2 : 0, ndy = M && backward ? ((M - 1) * a->lddy + D) * 2 : 0;
  const Range in[] = {{a->x, nx, "x"}, {a->w_in, 4 * I * D, "w_in"}, {a->w_out, 2 * I * D, "w_out"},
                      {backward ? a->dy : nullptr, ndy, "dy"},
                      {backward ? a->kept : nullptr, gemm_ffn_kept_bytes(M, I), "kept"}};
  const Range out[] = {{backward ? nullptr : a->y, 2 * M * D, "y"},
                       {backward ? nullptr : a->kept, gemm_ffn_kept_bytes(M, I), "kept"},
                       {backward ? a->dx : nullptr, 2 * M * D, "dx"},
                       {backward ? a->dw_in : nullptr, 4 * I * D, "dw_in"},
                       {backward ? a->dw_out : nullptr, 2 * I * D, "dw_out"},
                       {ws, ws_bytes, "the workspace"}};
  constexpr int kOut = sizeof(out) / sizeof(out[0]);
  for (int i = 0; i < kOut; ++i) {
    for (const Range& r : in)
      if (overlap(out[i].p, out[i].n, r.p, r.n))
        return ops_fail(GEMM_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, r.name);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return ops_fail(GEMM_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
  }
  return GEMM_OK;
}

// Lays out the workspace (with a null base: only measures it).  An operand
// the copy engine cannot read is replaced by a padded copy.
size_t layout(const gemm_ops* ops, const gemm_ffn_args_t* a, bool backward, void* workspace, Ffn* f) {
  f->a = a;
  f->M = a->tokens;
  f->D = a->d_model;
  f->I = a->d_inner;
  f->Ip = round8(f->I);
  f->bf16 = a->dtype == GEMM_BF16;
  f->x = {a->x, f->M, f->D, a->ldx, 0};
  f->dy = {a->dy, f->M, f->D, a->lddy, 0};
  f->w_in = {a->w_in, 2 * f->I, f->D, f->D, 0};
  f->w_out = {a->w_out, f->D, f->I, f->I, 0};
  // (The fault hook withholds a copy, of which the path for few tokens has none.)
  const bool few = !backward && ops->debug_fault == 0;
  f->few_first = few && few_tokens_fits(ops, f->M, 2 * f->I, f->w_in);
  f->few_second = few && few_tokens_fits(ops, f->M, f->D, f->w_out);
  Carver c(workspace);
  f->scratch = f->few_first && f->few_second ? BlockScratch() : take_scratch(ops, c);
  f->pre = static_cast<float*>(a->kept);
  if (a->kept)
    f->h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a->kept) + pre_bytes(f->M, f->I));
  else
    f->h = static_cast<uint16_t*>(c.take(static_cast<size_t>(f->M) * f->Ip * 2));
  f->dgu = backward
               ? static_cast<uint16_t*>(c.take(static_cast<size_t>(f->M) * round8(2 * f->I) * 2))
               : nullptr;
  f->pack.count = 0;
  auto padded = [&](Matrix* m) {
    if (copyable(*m)) return;
    const int64_t ldp = round8(m->cols);
    uint16_t* dst = static_cast<uint16_t*>(c.take(static_cast<size_t>(m->rows) * ldp * 2));
    f->pack.job[f->pack.count++] = {static_cast<const uint16_t*>(m->ptr), dst, m->rows, m->cols,
                                    m->ld, ldp};
    m->ptr = dst;
    m->ld = ldp;
  };
  if (!f->few_second) padded(&f->w_out);
  if (!f->few_first && (!backward || a->dx)) padded(&f->w_in);
  if (!f->few_first && (!backward || a->dw_in)) padded(&f->x);
  if (backward) padded(&f->dy);
  return c.used;
}

gemm_status_t prepare(gemm_ops_t* ops, const gemm_ffn_args_t* a, bool backward, void* workspace,
                      size_t bytes, Ffn* f) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops) return ops_fail(GEMM_ERR_INVALID_ARG, "ops is NULL");
  gemm_status_t st = check(a, backward);
  if (st != GEMM_OK) return st;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return ops_fail(GEMM_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
  const size_t need = layout(ops, a, backward, workspace, f);
  if (a->tokens > 0 && need > 0 && (!workspace || bytes < need))
    return ops_fail(GEMM_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? bytes : 0,
                    need);
  return check_overlap(a, backward, workspace, need);
}

}  // namespace

extern "C" {

size_t gemm_ffn_kept_bytes(int64_t tokens, int64_t d_inner) {
  if (tokens <= 0 || d_inner <= 0) return 0;
  return pre_bytes(tokens, d_inner) + align256(static_cast<size_t>(tokens) * round8(d_inner) * 2);
}

gemm_status_t gemm_ffn_workspace(gemm_ops_t* ops, const gemm_ffn_args_t* args, int backward,
                                 size_t* bytes) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops || !bytes) return ops_fail(GEMM_ERR_INVALID_ARG, "NULL argument");
  const gemm_status_t st = check(args, backward != 0);
  if (st != GEMM_OK) return st;
  Ffn f;
  *bytes = layout(ops, args, backward != 0, nullptr, &f);
  return GEMM_OK;
}

gemm_status_t gemm_ffn_run(gemm_ops_t* ops, const gemm_ffn_args_t* args, void* workspace,
                           size_t workspace_bytes, void* stream_handle) {
  Ffn f;
  gemm_status_t st = prepare(ops, args, false, workspace, workspace_bytes, &f);
  if (st != GEMM_OK || f.M == 0) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  const cudaError_t e = launch_pack(f.pack, ops->sm_count, stream);
  if (e != cudaSuccess) return ops_cuda_fail(e, "padding copy launch");

  if (f.few_first) {
    FewTokens t{};
    t.x = f.x;
    t.w = f.w_in;
    t.rows = f.I;
    t.gated = true;
    t.bf16 = f.bf16;
    t.out = f.h;
    t.ldo = f.Ip;
    t.pre = f.pre;
    t.act = static_cast<int>(args->act);
    const cudaError_t err = few_tokens_launch(ops, t, stream);
    if (err != cudaSuccess) return ops_cuda_fail(err, "few tokens launch");
  } else {
    BlockProblem g;
    g.kind = BlockProblem::kGated;
    g.M = f.M;
    g.N = f.I;
    g.K = f.D;
    g.a = f.x;
    g.b = f.w_in;
    g.bf16 = g.out_bf16 = f.bf16;
    g.act = static_cast<int>(args->act);
    g.out0 = {f.h, f.M, f.Ip, f.Ip, 0};
    g.pre = f.pre;
    g.stream_b = true;
    st = run_block(ops, g, f.scratch, stream);
    if (st != GEMM_OK) return st;
  }

  const Matrix h{f.h, f.M, f.I, f.Ip, 0};
  if (f.few_second) {
    FewTokens t{};
    t.x = h;
    t.w = f.w_out;
    t.rows = f.D;
    t.bf16 = f.bf16;
    t.weights_ready = f.few_first;
    t.out = static_cast<uint16_t*>(args->y);
    t.ldo = f.D;
    const cudaError_t err = few_tokens_launch(ops, t, stream);
    return err == cudaSuccess ? GEMM_OK : ops_cuda_fail(err, "few tokens launch");
  }
  BlockProblem y;
  y.kind = BlockProblem::kNT;
  y.M = f.M;
  y.N = f.D;
  y.K = f.I;
  y.a = h;
  y.b = f.w_out;
  y.bf16 = y.out_bf16 = f.bf16;
  y.out0 = {args->y, f.M, f.D, f.D, 0};
  y.stream_b = true;
  return run_block(ops, y, f.scratch, stream);
}

gemm_status_t gemm_ffn_backward(gemm_ops_t* ops, const gemm_ffn_args_t* args, void* workspace,
                                size_t workspace_bytes, void* stream_handle) {
  Ffn f;
  gemm_status_t st = prepare(ops, args, true, workspace, workspace_bytes, &f);
  if (st != GEMM_OK) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  const int64_t M = f.M, D = f.D, I = f.I, Gp = round8(2 * I);
  if (M == 0) {  // sums over no tokens
    cudaError_t e = cudaSuccess;
    if (args->dw_in) e = cudaMemsetAsync(args->dw_in, 0, static_cast<size_t>(4) * I * D, stream);
    if (e == cudaSuccess && args->dw_out)
      e = cudaMemsetAsync(args->dw_out, 0, static_cast<size_t>(2) * I * D, stream);
    return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "cudaMemsetAsync(weight gradients)");
  }
  const cudaError_t e = launch_pack(f.pack, ops->sm_count, stream);
  if (e != cudaSuccess) return ops_cuda_fail(e, "padding copy launch");

  if (args->dx || args->dw_in) {
    BlockProblem g;
    g.kind = BlockProblem::kGatedBwd;
    g.M = M;
    g.N = I;
    g.K = D;
    g.a = f.dy;
    g.b = f.w_out;
    g.bf16 = g.out_bf16 = f.bf16;
    g.act = static_cast<int>(args->act);
    g.out0 = {f.dgu, M, I, Gp, 0};      // side by side in one row
    g.out1 = {f.dgu + I, M, I, Gp, 0};
    g.pre = f.pre;
    st = run_block(ops, g, f.scratch, stream);
    if (st != GEMM_OK) return st;
  }
  BlockProblem p;
  p.bf16 = p.out_bf16 = f.bf16;
  if (args->dx) {
    p.kind = BlockProblem::kNN;
    p.M = M;
    p.N = D;
    p.K = 2 * I;
    p.a = {f.dgu, M, 2 * I, Gp, 0};
    p.b = f.w_in;
    p.out0 = {args->dx, M, D, D, 0};
    st = run_block(ops, p, f.scratch, stream);
    if (st != GEMM_OK) return st;
  }
  p.kind = BlockProblem::kTN;
  p.K = M;
  if (args->dw_in) {
    p.M = 2 * I;
    p.N = D;
    p.a = {f.dgu, M, 2 * I, Gp, 0};
    p.b = f.x;
    p.out0 = {args->dw_in, 2 * I, D, D, 0};
    st = run_block(ops, p, f.scratch, stream);
    if (st != GEMM_OK) return st;
  }
  if (args->dw_out) {
    p.M = D;
    p.N = I;
    p.a = f.dy;
    p.b = {f.h, M, I, f.Ip, 0};
    p.out0 = {args->dw_out, D, I, I, 0};
    st = run_block(ops, p, f.scratch, stream);
  }
  return st;
}

}  // extern "C"
