/*
 * gemm_ops.h -- C ABI of the operators built around the GEMM (gemm.h): the
 * gated feed-forward block with its backward pass, the orthogonalised update
 * of a gradient, the log probabilities of tokens with their gradient,
 * products grouped by expert with their gradients, layer norm with its
 * gradients, and the AdamW step of many tensors.
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

/* ---- Products grouped by expert ---------------------------------------------
 * Group e is the rows offsets[e] .. offsets[e + 1] - 1 of x:
 *   y_r = W_e x_r,  dx_r = W_e^T dy_r,  dW_e = sum_r dy_r x_r^T
 * x: rows x k, w: groups x n x k, y: rows x n; sums in fp32, each output
 * rounded to `dtype` once.  The offsets are read on the device, so a call
 * needs no host copy of them.  They may not decrease nor leave [0, rows];
 * where they do, nothing is written to y, dx and dw and gemm_ops_check
 * reports GEMM_ERR_INVALID_ARG (GEMM_CHECK_OFFSETS).  What rows of no group
 * hold, NaN and infinities too, reaches no output, but they may be read (with
 * the last rows of a group, or by the copy of an operand that is not aligned):
 * nobody else may write them during the call. */
#define GEMM_GROUPED_MAX_GROUPS 4096
/* Details of the status word. */
#define GEMM_CHECK_OFFSETS ((0 << 16) | 17)  /* offsets that decrease or leave the rows */
#define GEMM_WAIT_NEXT_TILE ((3 << 16) | 5)  /* a role waiting for its CTA pair's next tile */
#define GEMM_WAIT_NEXT_FREE ((3 << 16) | 6)  /* the scheduler waiting for the roles to take one */

typedef struct {
  int64_t rows, groups, n, k;  /* rows 0 .. 2^31 - 65536, n, k >= 1, groups 1 .. GEMM_GROUPED_MAX_GROUPS */
  gemm_dtype_t dtype;
  const int64_t* offsets;      /* groups + 1, on the device */
  const void* x;
  int64_t ldx;                 /* row pitch, elements, >= k */
  const void* w;               /* dense */
  void* y;                     /* forward only: rows x n, dense */
  int zero_rest;               /* 1: rows of no group of y and dx become zero; 0: they are left
                                  as they were */
  const void* dy;              /* backward only: rows x n, row pitch lddy */
  int64_t lddy;
  void* dx;                    /* rows x k, dense; each gradient may be NULL */
  void* dw;                    /* groups x n x k; zero for an empty group */
} gemm_grouped_args_t;

/* Workspace of gemm_grouped_run (backward 0) or gemm_grouped_backward (1). */
gemm_status_t gemm_grouped_workspace(gemm_ops_t* ops, const gemm_grouped_args_t* args, int backward,
                                     size_t* bytes);
gemm_status_t gemm_grouped_run(gemm_ops_t* ops, const gemm_grouped_args_t* args, void* workspace,
                               size_t workspace_bytes, void* stream);
gemm_status_t gemm_grouped_backward(gemm_ops_t* ops, const gemm_grouped_args_t* args,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* ---- Layer norm ---------------------------------------------------------------
 * For each row x (rows x cols), in fp32:
 *   y = h weight + bias,  h = (x - mean) rstd,  rstd = 1 / sqrt(var + eps)
 * var being the mean of (x - mean)^2.  The mean is held in two floats, so that
 * a row far from zero keeps its differences; a constant row has a variance of
 * 0.  Rows of finite values of any size, and variances below fp32's range with
 * an eps of 0, have their y; rstd is kept in fp32, so the gradients of a row
 * whose deviation is below 2^-128 with an eps of 0 are not finite.  A row that
 * holds NaN or an infinity becomes NaN. */
typedef struct {
  int64_t rows, cols;       /* rows >= 0, cols >= 1 */
  gemm_in_t dtype;          /* of x, y, dy and dx */
  gemm_in_t weight_dtype;   /* of weight, bias and their gradients: dtype, or GEMM_IN_F32 */
  const void* x;
  int64_t ldx;              /* row pitch, elements, >= cols */
  const void* weight;       /* cols; NULL: ones */
  const void* bias;         /* cols; NULL: zeros.  Forward only */
  float eps;                /* >= 0 */
  void* y;                  /* forward only: rows x cols, dense; may be x itself (ldx == cols) */
  float* stats;             /* 3 x rows: mean, what its rounding to fp32 lost, rstd.  Written by
                               the forward pass (NULL: not kept), read by the backward pass */
  const void* dy;           /* backward only: rows x cols, row pitch lddy */
  int64_t lddy;
  void* dx;                 /* rows x cols, dense; may be dy itself (lddy == cols) */
  void* dweight;            /* cols; each gradient may be NULL */
  void* dbias;
} gemm_layer_norm_args_t;

gemm_status_t gemm_layer_norm(gemm_ops_t* ops, const gemm_layer_norm_args_t* args, void* stream);

/* With g = dy weight and <.> the mean of a row:
 *   dx = rstd (g - <g> - h <g h>),  dweight = sum_rows dy h,  dbias = sum_rows dy
 * The sums over rows have a fixed order.  With no rows they are zero.  Where a
 * row's sums of g or g h leave fp32's range its dx is not finite. */
gemm_status_t gemm_layer_norm_backward_workspace(gemm_ops_t* ops, const gemm_layer_norm_args_t* args,
                                                 size_t* bytes);
gemm_status_t gemm_layer_norm_backward(gemm_ops_t* ops, const gemm_layer_norm_args_t* args,
                                       void* workspace, size_t workspace_bytes, void* stream);

/* ---- AdamW step ------------------------------------------------------------------
 * For every element of every tensor, with g = scale grad and t the step's
 * number (1 for the first), in fp32:
 *   m <- beta1 m + (1 - beta1) g,  v <- beta2 v + (1 - beta2) g^2
 *   p <- p - lr weight_decay p - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * The parameters are updated in place (16-bit ones rounded to nearest), and
 * `copy` receives them in its type.  The states of all tensors lie in one
 * buffer each, in the tensors' order, each tensor's beginning at a multiple
 * of GEMM_ADAMW_BLOCK elements.
 *   bits 32: m and v in fp32.
 *   bits 8: in e4m3, times a scale for each block of GEMM_ADAMW_BLOCK elements:
 *     s = max(2^-120, largest magnitude / 448); m is rounded to nearest.  Of v
 *     the square root r is held.  It moves by far less than half a step of the
 *     format in one call, so that rounding to nearest would never let it
 *     fall: it is rounded down after adding u steps, u = (a j + b t) mod 2^32,
 *     its upper 20 bits as a fraction (element j of the buffer, a =
 *     0xC13FA9A9, b = 0x91E10DA5: the additive recurrence in two dimensions of
 *     the plastic number p, p^3 = p + 1, of which a and b are 1 / p and 1 / p^2
 *     times 2^32, rounded down), which over the steps is evenly spread in
 *     [0, 1); r > 0 is held as 2^-9 s at least.  (A root without gradients
 *     that beta2 = 0.999 takes to 0.47 in 1500 steps is then at 0.43.)  A NaN
 *     or an infinity makes its block NaN.
 * The update itself uses m and v as computed, before they are rounded. */
#define GEMM_ADAMW_BLOCK 256

typedef struct {
  void* param;
  const void* grad;
  void* copy;               /* or NULL */
  int64_t numel;            /* >= 0 */
  int param_type;           /* gemm_in_t, each */
  int grad_type;
  int copy_type;            /* GEMM_IN_F16 or GEMM_IN_BF16 */
  float weight_decay;
} gemm_adamw_tensor_t;

typedef struct {
  const gemm_adamw_tensor_t* tensors;  /* on the host; not needed after the call */
  int64_t count;
  int64_t state_elements;   /* of exp_avg and of exp_avg_sq: gemm_adamw_state_elements */
  int bits;                 /* of the states: 32 or 8 */
  void* exp_avg;            /* fp32 or e4m3, 16-byte aligned */
  void* exp_avg_sq;
  float* scales;            /* bits 8: 2 x blocks, of exp_avg and of exp_avg_sq */
  int64_t* step;            /* on the device: steps made so far, below 2^32; the call adds one */
  double lr;                /* used where lr_device is NULL */
  const float* lr_device;
  double beta1, beta2;      /* in [0, 1) */
  double eps;               /* 0, or in [2^-126, 2^126] */
  const float* scale;       /* on the device; NULL: 1 */
} gemm_adamw_args_t;

/* Elements of each state buffer. */
int64_t gemm_adamw_state_elements(const gemm_adamw_tensor_t* tensors, int64_t count);
gemm_status_t gemm_adamw(gemm_ops_t* ops, const gemm_adamw_args_t* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPGEMM_GEMM_OPS_H_ */
