/*
 * gemm_ops.h -- C ABI of the operators built around the GEMM (gemm.h): the
 * gated feed-forward block with its backward pass, the orthogonalised update
 * of a gradient, and the log probabilities of tokens with their gradient.
 *
 * Sizes vary from call to call (a prompt's length, a batch), so these
 * operators take no plan for a problem: one gemm_ops_t per device holds what
 * persists between calls (limits of the device and a status word), and a
 * call's buffers come from the caller: *_workspace says how many bytes a call
 * needs.
 *
 * Pointers are device pointers on the handle's device; matrices are
 * row-major.  A workspace starts 256-byte aligned, holds nothing between calls, and
 * may be reused by the next call on the same stream.  Outputs may not
 * overlap inputs, other outputs or the workspace, except where said.
 *
 * Errors are gemm.h's: argument errors are found on the host before anything
 * is launched, nothing throws, and a device-side wait that runs out of time
 * is recorded in the handle's status word (gemm_ops_check).  Calls are
 * asynchronous and may be captured into a CUDA graph.  One handle serves any
 * number of streams and host threads, but for gemm_ops_configure and
 * gemm_ops_destroy, which need it to themselves.  Calls, and graphs that
 * captured calls, may run beside one another as long as their workspaces,
 * `kept` buffers and outputs are different ones.
 */
#ifndef SPGEMM_GEMM_OPS_H_
#define SPGEMM_GEMM_OPS_H_

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemm_ops gemm_ops_t; /* opaque */

/* Create a handle on `device` (GEMM_ERR_UNSUPPORTED unless sm_103).  On
 * failure *out is set to NULL. */
gemm_status_t gemm_ops_create(gemm_ops_t** out, int device);

/* Wait for the handle's work to finish and free it.  NULL is allowed. */
void gemm_ops_destroy(gemm_ops_t* ops);

/* timeout_ns: the limit of each device-side wait of later calls, 0 for the
 * default (2 s).  debug_fault: test hook, 0 in normal use; 1: the first copy
 * of the first block of each kernel with a copy ring is announced but never
 * made, so that the waits run out and gemm_ops_check reports
 * GEMM_ERR_TIMEOUT.  Nothing faults or hangs. */
gemm_status_t gemm_ops_configure(gemm_ops_t* ops, int64_t timeout_ns, int debug_fault);

/* As gemm_plan_check: synchronise the device, read and clear the status word. */
gemm_status_t gemm_ops_check(gemm_ops_t* ops, int32_t* device_status, int32_t* detail);

/* ---- Gated feed-forward block --------------------------------------------
 *   G = X Wg^T,  U = X Wu^T,  H = act(G) * U,  Y = H Wo^T
 * X: tokens x d_model, row pitch ldx.  w_in: 2 d_inner x d_model, the rows
 * of Wg followed by those of Wu.  w_out: d_model x d_inner.  Y: tokens x
 * d_model.  All in `dtype`; Y, w_in and w_out dense.  G and U stay in fp32;
 * H is rounded to `dtype` once, being the second product's operand (in fp16
 * an element beyond 65504 becomes infinite). */
typedef enum { GEMM_ACT_SILU = 0, GEMM_ACT_GELU_TANH = 1, GEMM_ACT_RELU = 2 } gemm_act_t;

typedef struct {
  int64_t tokens, d_model, d_inner;  /* tokens >= 0, the others >= 1 */
  gemm_dtype_t dtype;
  gemm_act_t act;
  const void* x;
  int64_t ldx;                       /* row pitch of x in elements, >= d_model */
  const void* w_in;
  const void* w_out;
  void* y;                           /* forward only */
  void* kept;                        /* gemm_ffn_kept_bytes bytes, 256-byte aligned: written by
                                        the forward pass, read by the backward pass; NULL in a
                                        forward pass that needs no backward */
  const void* dy;                    /* backward only: tokens x d_model, pitch lddy */
  int64_t lddy;
  void* dx;                          /* tokens x d_model, dense; each gradient may be NULL */
  void* dw_in;                       /* 2 d_inner x d_model */
  void* dw_out;                      /* d_model x d_inner */
} gemm_ffn_args_t;

/* Bytes a forward pass keeps for the backward pass: G and U in fp32 (in the
 * order the kernels read them back) and H in the operands' type. */
size_t gemm_ffn_kept_bytes(int64_t tokens, int64_t d_inner);

/* Workspace of gemm_ffn_run (backward 0) or gemm_ffn_backward (1). */
gemm_status_t gemm_ffn_workspace(gemm_ops_t* ops, const gemm_ffn_args_t* args, int backward,
                                 size_t* bytes);

/* Y, and `kept` where it is given. */
gemm_status_t gemm_ffn_run(gemm_ops_t* ops, const gemm_ffn_args_t* args, void* workspace,
                           size_t workspace_bytes, void* stream);

/* Gradients of a forward pass with the same x, w_in, w_out and act, from dY
 * and what that pass kept:
 *   dH = dY Wo,  dG = dH * U * act'(G),  dU = dH * act(G)
 *   dX = [dG dU] w_in,  dw_in = [dG dU]^T X,  dw_out = dY^T H
 * in `dtype`, each rounded once; dG and dU are rounded to `dtype` as the
 * products' operands, with the same range.  With no tokens the weights' gradients are zero. */
gemm_status_t gemm_ffn_backward(gemm_ops_t* ops, const gemm_ffn_args_t* args, void* workspace,
                                size_t workspace_bytes, void* stream);

/* ---- Orthogonalised update --------------------------------------------------
 * For each matrix G (m x n) of a batch, with X = G / max(|G|_F, eps), `steps`
 * times
 *   X <- a X + (b A + c A^2) X,  A = X X^T   (m <= n)
 *   X <- a X + X (b A + c A^2),  A = X^T X   (m > n: the same, on the short side)
 * which drives the singular values of X towards one.  The iterates are held
 * in fp16 (times 2^8, so that a normalised matrix's small elements keep
 * their 11 bits: against bf16 the result is about eight times closer to
 * exact arithmetic), the products' sums in fp32; the result is rounded to
 * bf16. */
typedef enum { GEMM_IN_F16 = 0, GEMM_IN_BF16 = 1, GEMM_IN_F32 = 2 } gemm_in_t;

typedef struct {
  int64_t batch, m, n;   /* each >= 0; batch <= 65535 */
  gemm_in_t dtype;       /* of g */
  const void* g;
  int64_t ldg;           /* row pitch of g, elements, >= n */
  int64_t batch_stride;  /* pitch of g's matrices, elements */
  void* out;             /* bf16, batch x m x n, dense */
  int steps;             /* 1 .. 100 */
  float a, b, c;
  float eps;             /* > 0 */
} gemm_orthogonalize_args_t;

gemm_status_t gemm_orthogonalize_workspace(gemm_ops_t* ops, const gemm_orthogonalize_args_t* args,
                                           size_t* bytes);
gemm_status_t gemm_orthogonalize(gemm_ops_t* ops, const gemm_orthogonalize_args_t* args,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* ---- Log probabilities of tokens -------------------------------------------
 * For each row x of logits (rows x vocab, row pitch ld), in fp32:
 *   lse = ln sum_j e^x_j,  log p_j = x_j - lse,  H = -sum_j p_j log p_j
 * and the top_k columns of largest log p, best first, equal ones by the
 * lowest column (NaN ranks above all).  A logit of -inf is masked: its log
 * probability is -inf.  A row with nothing but masked logits has lse -inf
 * and H 0; one that holds NaN or +inf has lse and H NaN.  tokens[i] < 0: the
 * position does not count, its log probability is 0 and has no gradient;
 * tokens[i] >= vocab gives NaN. */
#define GEMM_LOGPROBS_MAX_TOP_K 64

typedef struct {
  int64_t rows, vocab;       /* rows >= 0, vocab >= 1 */
  gemm_in_t dtype;           /* of logits and d_logits */
  const void* logits;
  int64_t ld;                /* row pitch, elements, >= vocab */
  const int64_t* tokens;     /* rows, or NULL (no logprobs then) */
  int top_k;                 /* 0 .. min(GEMM_LOGPROBS_MAX_TOP_K, vocab); forward only */
  float* logprobs;           /* rows; written by the forward pass, may be NULL */
  float* entropy;            /* rows; likewise (read by a backward pass with d_entropy) */
  float* lse;                /* rows; likewise (read by the backward pass) */
  float* top_logprobs;       /* rows x top_k */
  int64_t* top_ids;          /* rows x top_k */
  const float* d_logprobs;   /* backward only, each rows or NULL (zero) */
  const float* d_entropy;
  void* d_logits;            /* rows x vocab, row pitch ldd; may be logits itself (ldd == ld) */
  int64_t ldd;
  float* lse_low;            /* rows; what lse's rounding to fp32 lost.  Written by the forward pass,
                                read by the backward pass; may be NULL in either (zero), at the cost
                                of |lse| 2^-24 in log p there */
} gemm_logprobs_args_t;

gemm_status_t gemm_token_logprobs(gemm_ops_t* ops, const gemm_logprobs_args_t* args, void* stream);

/* d_logits_j = g_l ([j = token] - p_j) - g_H p_j (log p_j + H), from the
 * forward pass's lse, lse_low (and entropy). */
gemm_status_t gemm_token_logprobs_backward(gemm_ops_t* ops, const gemm_logprobs_args_t* args,
                                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPGEMM_GEMM_OPS_H_ */
