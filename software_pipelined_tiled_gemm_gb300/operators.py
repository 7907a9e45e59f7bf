"""The operators built around the GEMM: the gated feed-forward block with its
backward pass, the orthogonalised update of a gradient, the log
probabilities of tokens with their gradient, products grouped by expert with
their gradients, layer norm with its gradients, and the AdamW step of many
tensors.

A thin ctypes binding over ``include/gemm_ops.h``.  As in :func:`matmul_nt`,
tensors are CUDA tensors, work goes to the current stream of their device,
nothing synchronises, and there is no fallback.  What a call needs besides
its outputs (a workspace) comes from PyTorch's allocator on that stream.
Nothing is recorded for autograd: outputs have no graph, even where inputs
require gradients; the *_backward functions give those.
One library handle is kept per device; :func:`check_operators` reports what
a kernel recorded in them.
"""
from __future__ import annotations

import collections
import ctypes
import functools
import itertools
import operator
import struct
import threading

__all__ = [
    "gated_ffn", "gated_ffn_backward", "GatedKept", "orthogonalize", "check_operators",
    "close_operators", "FfnArgs", "OrthogonalizeArgs", "NEWTON_SCHULZ", "token_logprobs",
    "token_logprobs_backward", "TokenLogprobs", "LogprobsArgs", "MAX_TOP_K", "grouped_matmul",
    "grouped_matmul_backward", "GroupedArgs", "MAX_GROUPS", "layer_norm", "layer_norm_backward",
    "LayerNormKept", "LayerNormArgs", "adamw", "adamw_state", "AdamWState", "AdamWTensor",
    "AdamWArgs", "ADAMW_BLOCK",
]

_vp, _i64, _ci, _f, _sz, _d = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                               ctypes.c_size_t, ctypes.c_double)

GEMM_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 1, "relu": 2}

# a, b, c of X <- a X + (b A + c A^2) X: steep at zero, so that five steps
# bring every singular value above about 1e-3 of the norm close to one.
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


class FfnArgs(ctypes.Structure):
    """gemm_ffn_args_t"""
    _fields_ = [("tokens", _i64), ("d_model", _i64), ("d_inner", _i64), ("dtype", _ci),
                ("act", _ci), ("x", _vp), ("ldx", _i64), ("w_in", _vp), ("w_out", _vp),
                ("y", _vp), ("kept", _vp), ("dy", _vp), ("lddy", _i64), ("dx", _vp),
                ("dw_in", _vp), ("dw_out", _vp)]


class OrthogonalizeArgs(ctypes.Structure):
    """gemm_orthogonalize_args_t"""
    _fields_ = [("batch", _i64), ("m", _i64), ("n", _i64), ("dtype", _ci), ("g", _vp),
                ("ldg", _i64), ("batch_stride", _i64), ("out", _vp), ("steps", _ci), ("a", _f),
                ("b", _f), ("c", _f), ("eps", _f)]


class LogprobsArgs(ctypes.Structure):
    """gemm_logprobs_args_t"""
    _fields_ = [("rows", _i64), ("vocab", _i64), ("dtype", _ci), ("logits", _vp), ("ld", _i64),
                ("tokens", _vp), ("top_k", _ci), ("logprobs", _vp), ("entropy", _vp),
                ("lse", _vp), ("top_logprobs", _vp), ("top_ids", _vp), ("d_logprobs", _vp),
                ("d_entropy", _vp), ("d_logits", _vp), ("ldd", _i64), ("lse_low", _vp)]


class GroupedArgs(ctypes.Structure):
    """gemm_grouped_args_t"""
    _fields_ = [("rows", _i64), ("groups", _i64), ("n", _i64), ("k", _i64), ("dtype", _ci),
                ("offsets", _vp), ("x", _vp), ("ldx", _i64), ("w", _vp), ("y", _vp),
                ("zero_rest", _ci), ("dy", _vp), ("lddy", _i64), ("dx", _vp), ("dw", _vp)]


class LayerNormArgs(ctypes.Structure):
    """gemm_layer_norm_args_t"""
    _fields_ = [("rows", _i64), ("cols", _i64), ("dtype", _ci), ("weight_dtype", _ci), ("x", _vp),
                ("ldx", _i64), ("weight", _vp), ("bias", _vp), ("eps", _f), ("y", _vp),
                ("stats", _vp), ("dy", _vp), ("lddy", _i64), ("dx", _vp), ("dweight", _vp),
                ("dbias", _vp)]


class AdamWTensor(ctypes.Structure):
    """gemm_adamw_tensor_t"""
    _fields_ = [("param", _vp), ("grad", _vp), ("copy", _vp), ("numel", _i64), ("param_type", _ci),
                ("grad_type", _ci), ("copy_type", _ci), ("weight_decay", _f)]


class AdamWArgs(ctypes.Structure):
    """gemm_adamw_args_t"""
    _fields_ = [("tensors", _vp), ("count", _i64), ("state_elements", _i64), ("bits", _ci), ("exp_avg", _vp),
                ("exp_avg_sq", _vp), ("scales", _vp), ("step", _vp), ("lr", _d),
                ("lr_device", _vp), ("beta1", _d), ("beta2", _d), ("eps", _d), ("scale", _vp)]


ADAMW_BLOCK = 256   # GEMM_ADAMW_BLOCK
MAX_TOP_K = 64      # GEMM_LOGPROBS_MAX_TOP_K
MAX_GROUPS = 4096   # GEMM_GROUPED_MAX_GROUPS

_bound = None
_handles: dict = {}
_lock = threading.Lock()
_sixteen: dict = {}   # torch dtype -> gemm_dtype_t
_inputs: dict = {}    # torch dtype -> gemm_in_t


def _lib():
    """The library, with the operators' signatures set."""
    global _bound
    if _bound is not None:
        return _bound
    import torch
    from . import load_library
    lib = load_library()
    _sixteen.update({torch.float16: 0, torch.bfloat16: 1})
    _inputs.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    psz = ctypes.POINTER(_sz)
    pi32 = ctypes.POINTER(ctypes.c_int32)
    for name, args in {
            "gemm_ops_create": [ctypes.POINTER(_vp), _ci],
            "gemm_ops_check": [_vp, pi32, pi32],
            "gemm_ops_configure": [_vp, _i64, _ci],
            "gemm_ffn_workspace": [_vp, ctypes.POINTER(FfnArgs), _ci, psz],
            "gemm_ffn_run": [_vp, ctypes.POINTER(FfnArgs), _vp, _sz, _vp],
            "gemm_ffn_backward": [_vp, ctypes.POINTER(FfnArgs), _vp, _sz, _vp],
            "gemm_orthogonalize_workspace": [_vp, ctypes.POINTER(OrthogonalizeArgs), psz],
            "gemm_orthogonalize": [_vp, ctypes.POINTER(OrthogonalizeArgs), _vp, _sz, _vp],
            "gemm_token_logprobs": [_vp, ctypes.POINTER(LogprobsArgs), _vp],
            "gemm_token_logprobs_backward": [_vp, ctypes.POINTER(LogprobsArgs), _vp],
            "gemm_grouped_workspace": [_vp, ctypes.POINTER(GroupedArgs), _ci, psz],
            "gemm_grouped_run": [_vp, ctypes.POINTER(GroupedArgs), _vp, _sz, _vp],
            "gemm_grouped_backward": [_vp, ctypes.POINTER(GroupedArgs), _vp, _sz, _vp],
            "gemm_layer_norm": [_vp, ctypes.POINTER(LayerNormArgs), _vp],
            "gemm_layer_norm_backward_workspace": [_vp, ctypes.POINTER(LayerNormArgs), psz],
            "gemm_layer_norm_backward": [_vp, ctypes.POINTER(LayerNormArgs), _vp, _sz, _vp],
            "gemm_adamw": [_vp, ctypes.POINTER(AdamWArgs), _vp]}.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, _ci
    lib.gemm_ops_destroy.argtypes, lib.gemm_ops_destroy.restype = [_vp], None
    lib.gemm_ffn_kept_bytes.argtypes, lib.gemm_ffn_kept_bytes.restype = [_i64, _i64], _sz
    _bound = lib
    return lib


def _check(status, where):
    if status:
        from . import GemmError, gemm_last_error
        raise GemmError(status, where, gemm_last_error())


def _stream(device):
    """The raw handle of the device's current stream."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _handle(device):
    """The handle of a device."""
    h = _handles.get(device.index)
    if h is None:
        with _lock:
            h = _handles.get(device.index)
            if h is None:
                out = _vp()
                _check(_lib().gemm_ops_create(ctypes.byref(out), device.index), "gemm_ops_create")
                h = _handles[device.index] = out.value
    return h


def check_operators() -> None:
    """Synchronise and raise :class:`GemmError` if a kernel of any operator
    recorded an error (a wait that ran out of time).  Every device's record is
    read and cleared; the first error is raised."""
    from . import GemmError, gemm_last_error, gemm_wait_detail_string
    with _lock:
        handles = list(_handles.values())
    errors = []
    for h in handles:
        ds, detail = ctypes.c_int32(0), ctypes.c_int32(0)
        status = _lib().gemm_ops_check(h, ctypes.byref(ds), ctypes.byref(detail))
        if status:
            errors.append(GemmError(status, "gemm_ops_check", gemm_last_error()))
        elif ds.value:
            errors.append(GemmError(ds.value, "operators", gemm_wait_detail_string(detail.value)))
    if errors:
        raise errors[0]


def _configure(device, timeout_ns=0, debug_fault=0) -> None:
    """gemm_ops_configure for the device's handle (tests)."""
    _check(_lib().gemm_ops_configure(_handle(device), timeout_ns, debug_fault), "gemm_ops_configure")


def close_operators() -> None:
    """Close every handle (synchronises their devices).  Not while a CUDA
    graph that captured a call is alive."""
    with _lock:
        while _handles:
            _lib().gemm_ops_destroy(_handles.popitem()[1])


def _rows(t, cols, name):
    """(rows, row pitch) of `t` seen as a matrix of `cols` columns."""
    if t.dim() == 0 or t.shape[-1] != cols:
        raise ValueError("%s must have %d columns" % (name, cols))
    rows = t.numel() // cols
    if t.is_contiguous():
        return rows, cols
    if t.dim() != 2 or (cols > 1 and t.stride(1) != 1) or t.stride(0) < cols:
        raise ValueError("%s must be contiguous, or a matrix of contiguous rows" % name)
    return rows, t.stride(0)


def _on_cuda(device, tensor, name):
    import torch
    if not isinstance(tensor, torch.Tensor) or not tensor.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if tensor.device != device:
        raise ValueError("all tensors must be on the same device (%s is not)" % name)


def _output(out, shape, dtype, device, name="out"):
    import torch
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if (tuple(out.shape) != tuple(shape) or out.dtype != dtype or out.device != device
            or not out.is_contiguous()):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on the inputs' device"
                         % (name, dtype, tuple(shape)))
    return out


def _ptr(t):
    return t.data_ptr() if t is not None else None


# ------------------------------------------------ gated feed-forward block --

# What a forward pass keeps for the backward pass: the fp32 gate and up
# projections and the 16-bit product, in the kernels' own layout.
GatedKept = collections.namedtuple("GatedKept", "buffer tokens d_model d_inner dtype act")


def _ffn_args(x, w_in, w_out, act):
    act_code = GEMM_ACT.get(act)
    if act_code is None:
        raise ValueError("act must be one of %s" % ", ".join(sorted(GEMM_ACT)))
    _on_cuda(getattr(x, "device", None), x, "x")
    _on_cuda(x.device, w_in, "w_in")
    _on_cuda(x.device, w_out, "w_out")
    dtype = x.dtype
    code = _sixteen.get(dtype)
    if code is None:
        raise TypeError("x must be float16 or bfloat16, got %s" % dtype)
    if w_in.dtype != dtype or w_out.dtype != dtype:
        raise TypeError("x, w_in and w_out must have the same dtype")
    if w_out.dim() != 2 or tuple(w_in.shape) != (2 * w_out.shape[1], w_out.shape[0]):
        raise ValueError("w_in must be (2 d_inner, d_model) and w_out (d_model, d_inner)")
    if not (w_in.is_contiguous() and w_out.is_contiguous()):
        raise ValueError("w_in and w_out must be contiguous")
    d, i = w_out.shape
    if d == 0 or i == 0:
        raise ValueError("d_model and d_inner must be at least 1")
    m, ldx = _rows(x, d, "x")
    return FfnArgs(m, d, i, code, act_code, x.data_ptr(), ldx, w_in.data_ptr(), w_out.data_ptr(),
                   None, None, None, d)


def _run(name, query, run, args, device, *which):
    """Workspace from the caching allocator of the current stream, then the call."""
    import torch
    stream = _stream(device)
    h = _handle(device)
    ref, need = ctypes.byref(args), _sz()
    status = query(h, ref, *which, ctypes.byref(need))
    if not status:
        n = need.value
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        status = run(h, ref, ws.data_ptr(), n, stream)
    if status:
        _check(status, name)


def gated_ffn(x, w_in, w_out, act="silu", out=None, save=False):
    """y = (act(x Wg^T) * (x Wu^T)) w_out^T on the current CUDA stream.

    x: (..., d_model), float16 or bfloat16, contiguous or a matrix of
    contiguous rows.  w_in: (2 d_inner, d_model), the rows of Wg followed by
    those of Wu; w_out: (d_model, d_inner); both contiguous, of x's dtype.
    act: "silu", "gelu" (tanh form) or "relu".  Returns y of x's shape and
    dtype (``out`` if given), or ``(y, kept)`` with ``save=True``, kept being
    what :func:`gated_ffn_backward` needs (10 bytes per token and inner
    feature: the projections stay in fp32).

    act(x Wg^T) * (x Wu^T) is rounded to x's dtype before the second product,
    so in float16 an element of it beyond 65504 becomes infinite.  No autograd
    graph: for gradients pass ``save=True`` and call
    :func:`gated_ffn_backward`.
    """
    import torch
    lib = _lib()
    a = _ffn_args(x, w_in, w_out, act)
    y = _output(out, x.shape, x.dtype, x.device)
    a.y = y.data_ptr()
    kept = None
    if save:
        buf = torch.empty(lib.gemm_ffn_kept_bytes(a.tokens, a.d_inner), dtype=torch.uint8,
                          device=x.device)
        a.kept = buf.data_ptr()
        kept = GatedKept(buf, a.tokens, a.d_model, a.d_inner, x.dtype, act)
    if a.tokens:
        _run("gemm_ffn_run", lib.gemm_ffn_workspace, lib.gemm_ffn_run, a, x.device, 0)
    return (y, kept) if save else y


def gated_ffn_backward(dy, x, w_in, w_out, kept, need=(True, True, True), out=(None, None, None)):
    """Gradients (dx, dw_in, dw_out) of :func:`gated_ffn` from dy and what
    the forward pass kept, with the same x, w_in and w_out.

    dy: x's shape and dtype, contiguous or a matrix of contiguous rows.  The
    gradients of the projections are rounded to that dtype as operands of the
    products (in float16 infinite beyond 65504).
    need: which of the three to compute (None in the place of the others).
    out: tensors to write them to.
    """
    if not isinstance(kept, GatedKept):
        raise TypeError("kept must come from gated_ffn(..., save=True)")
    lib = _lib()
    a = _ffn_args(x, w_in, w_out, kept.act)
    _on_cuda(x.device, dy, "dy")
    if dy.dtype != x.dtype or dy.shape != x.shape:
        raise ValueError("dy must have x's shape and dtype")
    if (a.tokens, a.d_model, a.d_inner, x.dtype) != kept[1:5] or kept.buffer.device != x.device:
        raise ValueError("kept belongs to a forward pass of other sizes, dtype or device")
    a.dy = dy.data_ptr()
    a.lddy = _rows(dy, a.d_model, "dy")[1]
    a.kept = kept.buffer.data_ptr()
    shapes = ((x.shape, "dx"), (w_in.shape, "dw_in"), (w_out.shape, "dw_out"))
    grads = [_output(o, shape, x.dtype, x.device, name) if want else None
             for want, o, (shape, name) in zip(need, out, shapes)]
    a.dx, a.dw_in, a.dw_out = map(_ptr, grads)
    _run("gemm_ffn_backward", lib.gemm_ffn_workspace, lib.gemm_ffn_backward, a, x.device, 1)
    return tuple(grads)


# --------------------------------------------------- orthogonalised update --

def orthogonalize(g, steps=5, coeffs=NEWTON_SCHULZ, eps=1e-7, out=None):
    """The orthogonalised form of a matrix, by Newton-Schulz products.

    X = g / max(|g|_F, eps), then `steps` times X <- a X + (b A + c A^2) X
    with A = X X^T (on the shorter side).  g: (m, n) or a batch (b, m, n) of
    up to 65535 matrices, float32, float16 or bfloat16, rows contiguous.  The
    iterates are float16 whatever g is.  Returns bfloat16 of g's
    shape (``out`` if given): the update of a weight whose gradient or
    momentum is g.
    """
    import torch
    _on_cuda(getattr(g, "device", None), g, "g")
    lib = _lib()
    if g.dtype not in _inputs:
        raise TypeError("g must be float32, float16 or bfloat16, got %s" % g.dtype)
    if g.dim() not in (2, 3):
        raise ValueError("g must be a matrix or a batch of matrices")
    if len(coeffs) != 3:
        raise ValueError("coeffs must be (a, b, c)")
    b, m, n = (1,) * (3 - g.dim()) + tuple(g.shape)
    ld, bs = n, m * n
    if not g.is_contiguous():
        # Strides along a single row or column lead nowhere.
        ld, bs = g.stride(-2) if m > 1 else n, (g.stride(0) if g.dim() == 3 else 0)
        if (n > 1 and g.stride(-1) != 1) or ld < n or (b > 1 and bs < 0):
            raise ValueError("g must have contiguous rows")
    y = _output(out, g.shape, torch.bfloat16, g.device)
    a = OrthogonalizeArgs(batch=b, m=m, n=n, dtype=_inputs[g.dtype], g=g.data_ptr(), ldg=ld,
                          batch_stride=bs, out=y.data_ptr(), steps=int(steps), a=coeffs[0],
                          b=coeffs[1], c=coeffs[2], eps=eps)
    _run("gemm_orthogonalize", lib.gemm_orthogonalize_workspace, lib.gemm_orthogonalize, a, g.device)
    return y


# ----------------------------------------------- log probabilities of tokens --

# Per row of logits (None where not asked for): log probability of the row's
# token, entropy, log of the sum of exponentials, the best alternatives, and
# what lse's rounding to fp32 lost (for the backward pass; None: zero).
TokenLogprobs = collections.namedtuple("TokenLogprobs",
                                       "logprobs entropy lse top_logprobs top_ids lse_low",
                                       defaults=(None,))


def _logprobs_args(logits, tokens):
    import torch
    device = getattr(logits, "device", None)
    _on_cuda(device, logits, "logits")
    _lib()
    code = _inputs.get(logits.dtype)
    if code is None:
        raise TypeError("logits must be float32, float16 or bfloat16, got %s" % logits.dtype)
    shape = logits.shape
    if len(shape) < 1 or shape[-1] == 0:
        raise ValueError("logits must have at least one column")
    rows, ld = _rows(logits, shape[-1], "logits")
    if tokens is not None:
        _on_cuda(device, tokens, "tokens")
        if tokens.dtype != torch.int64:
            raise TypeError("tokens must be int64, got %s" % tokens.dtype)
        if tokens.shape != shape[:-1] or not tokens.is_contiguous():
            raise ValueError("tokens must be contiguous, one for each row of logits")
    return LogprobsArgs(rows, shape[-1], code, logits.data_ptr(), ld,
                        None if tokens is None else tokens.data_ptr())


def token_logprobs(logits, tokens=None, top_k=0):
    """Log probabilities of `tokens` under rows of logits, in fp32.

    logits: (..., vocab), float32, float16 or bfloat16, contiguous or a
    matrix of contiguous rows (a slice of a padded vocabulary); no autograd
    graph, see :func:`token_logprobs_backward`.  tokens:
    int64 (...), or None; a negative one marks a position that does not
    count (log probability 0).  top_k: how many of the best columns to
    return, at most 64, equal ones by the lowest column.

    Returns :class:`TokenLogprobs`: logprobs, entropy, lse and lse_low of
    shape (...), top_logprobs and top_ids (int64) of shape (..., top_k).  -inf masks a
    column; a row of only masked columns has entropy 0, one with NaN or +inf
    has NaN.
    """
    import torch
    a = _logprobs_args(logits, tokens)
    if not 0 <= top_k <= min(MAX_TOP_K, a.vocab):
        raise ValueError("top_k must be in [0, min(%d, columns)]" % MAX_TOP_K)
    a.top_k = top_k
    shape, dev = logits.shape[:-1], logits.device
    out = torch.empty((3 if tokens is None else 4, *shape), dtype=torch.float32, device=dev)
    logprobs = None
    if tokens is None:
        lse, entropy, lse_low = out.unbind(0)
    else:
        lse, entropy, lse_low, logprobs = out.unbind(0)
    top_lp = top_ids = None
    if top_k:
        top_lp = torch.empty((*shape, top_k), dtype=torch.float32, device=dev)
        top_ids = torch.empty((*shape, top_k), dtype=torch.int64, device=dev)
        a.top_logprobs, a.top_ids = top_lp.data_ptr(), top_ids.data_ptr()
    a.lse, a.entropy, a.lse_low = lse.data_ptr(), entropy.data_ptr(), lse_low.data_ptr()
    a.logprobs = _ptr(logprobs)
    if a.rows:
        stream = _stream(dev)
        _check(_lib().gemm_token_logprobs(_handle(dev), ctypes.byref(a), stream),
               "gemm_token_logprobs")
    return TokenLogprobs(logprobs, entropy, lse, top_lp, top_ids, lse_low)


def token_logprobs_backward(logits, tokens, result, d_logprobs=None, d_entropy=None, out=None):
    """Gradient of the logits from those of the log probabilities and the
    entropies (float32, one for each row; None: zero).

    logits, tokens: as given to :func:`token_logprobs`, and `result` what it
    returned.  out: where to write it (logits itself is allowed); a new
    contiguous tensor of logits' dtype otherwise.
    """
    import torch
    a = _logprobs_args(logits, tokens)
    if d_logprobs is not None and tokens is None:
        raise ValueError("d_logprobs needs tokens")
    for name, t in (("lse", result.lse), ("entropy", result.entropy), ("lse_low", result.lse_low),
                    ("d_logprobs", d_logprobs), ("d_entropy", d_entropy)):
        if t is None and (name.startswith("d_") or name == "lse_low"):
            continue
        _on_cuda(logits.device, t, name)
        if t.dtype != torch.float32 or t.shape != logits.shape[:-1] or not t.is_contiguous():
            raise ValueError("%s must be contiguous float32, one for each row of logits" % name)
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    _on_cuda(logits.device, out, "out")
    if out.dtype != logits.dtype or out.shape != logits.shape:
        raise ValueError("out must have the logits' shape and dtype")
    a.ldd = _rows(out, a.vocab, "out")[1]
    a.lse, a.entropy, a.lse_low, a.d_logprobs, a.d_entropy, a.d_logits = map(
        _ptr, (result.lse, result.entropy, result.lse_low, d_logprobs, d_entropy, out))
    if a.rows:
        dev = logits.device
        stream = _stream(dev)
        _check(_lib().gemm_token_logprobs_backward(_handle(dev), ctypes.byref(a), stream),
               "gemm_token_logprobs_backward")
    return out


# ------------------------------------------------ products grouped by expert --

def _grouped_args(x, w, offsets):
    import torch
    device = getattr(x, "device", None)
    _on_cuda(device, x, "x")
    _on_cuda(device, w, "w")
    _on_cuda(device, offsets, "offsets")
    _lib()
    code = _sixteen.get(x.dtype)
    if code is None:
        raise TypeError("x must be float16 or bfloat16, got %s" % x.dtype)
    if w.dtype != x.dtype:
        raise TypeError("x and w must have the same dtype")
    if w.dim() != 3 or not w.is_contiguous():
        raise ValueError("w must be a contiguous (groups, n, k) tensor")
    e, n, k = w.shape
    if n == 0 or k == 0 or not 1 <= e <= MAX_GROUPS:
        raise ValueError("w must have 1 to %d groups, and n and k at least 1" % MAX_GROUPS)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    if offsets.dtype != torch.int64:
        raise TypeError("offsets must be int64, got %s" % offsets.dtype)
    if offsets.shape != (e + 1,) or not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous, one more than there are groups")
    rows, ldx = _rows(x, k, "x")
    return GroupedArgs(rows, e, n, k, code, offsets.data_ptr(), x.data_ptr(), ldx, w.data_ptr(),
                       lddy=n)


def grouped_matmul(x, w, offsets, out=None):
    """y_r = w[e] x_r for the rows r of each group e, on the current CUDA stream.

    x: (rows, k), float16 or bfloat16, rows contiguous (with any pitch).  w:
    (groups, n, k), contiguous, of x's dtype: the experts' weights.  offsets:
    int64 (groups + 1) on the GPU: group e is x[offsets[e]:offsets[e + 1]], any
    number of rows; it is read there, so nothing synchronises.  Returns y
    (rows, n) of x's dtype (``out`` if given).

    What rows before the first group and behind the last hold reaches no
    output (they may be read, so nobody else may be writing them); in y they
    are zero, or, where ``out`` is given, left as they were.  Offsets that
    decrease or leave x are found on the GPU: nothing is then written to y and
    :func:`check_operators` raises.  No autograd graph, see
    :func:`grouped_matmul_backward`.
    """
    lib = _lib()
    a = _grouped_args(x, w, offsets)
    y = _output(out, (a.rows, a.n), x.dtype, x.device)
    a.y, a.zero_rest = y.data_ptr(), out is None
    if a.rows:
        _run("gemm_grouped_run", lib.gemm_grouped_workspace, lib.gemm_grouped_run, a, x.device, 0)
    return y


def grouped_matmul_backward(dy, x, w, offsets, need=(True, True), out=(None, None)):
    """Gradients (dx, dw) of :func:`grouped_matmul` from dy, with the same x,
    w and offsets: dx_r = w[e]^T dy_r, dw[e] = sum over its rows of dy_r x_r^T.

    dy: (rows, n), of x's dtype, rows contiguous.  need: which of the two to
    compute (None in the place of the other).  out: tensors to write them to.
    Rows of no group are zero in dx (in a given one left as they were) and
    add nothing to dw, whatever they hold; an empty group's dw is zero.
    """
    lib = _lib()
    a = _grouped_args(x, w, offsets)
    _on_cuda(x.device, dy, "dy")
    if dy.dtype != x.dtype or tuple(dy.shape) != (a.rows, a.n):
        raise ValueError("dy must be (rows, n), of x's dtype")
    a.dy, a.lddy = dy.data_ptr(), _rows(dy, a.n, "dy")[1]
    shapes = ((x.shape, "dx"), (w.shape, "dw"))
    grads = [_output(o, shape, x.dtype, x.device, name) if want else None
             for want, o, (shape, name) in zip(need, out, shapes)]
    a.dx, a.dw = map(_ptr, grads)
    a.zero_rest = out[0] is None
    if any(need):
        _run("gemm_grouped_backward", lib.gemm_grouped_workspace, lib.gemm_grouped_backward, a, x.device, 1)
    return tuple(grads)


# ----------------------------------------------------------------- layer norm --

# What a forward pass keeps for the backward pass: (3, rows) float32, each
# row's mean, what its rounding to fp32 lost, and 1 / sqrt(var + eps).
LayerNormKept = collections.namedtuple("LayerNormKept", "stats rows cols dtype")


def _layer_norm_args(x, weight, bias):
    device = getattr(x, "device", None)
    _on_cuda(device, x, "x")
    _lib()
    code = _inputs.get(x.dtype)
    if code is None:
        raise TypeError("x must be float32, float16 or bfloat16, got %s" % x.dtype)
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("x must have at least one column")
    cols = x.shape[-1]
    rows, ldx = _rows(x, cols, "x")
    wcode = code
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        _on_cuda(device, t, name)
        if t.shape != (cols,) or not t.is_contiguous():
            raise ValueError("%s must be contiguous, one for each column" % name)
        if _inputs.get(t.dtype) not in (code, 2):
            raise TypeError("%s must be of x's dtype or float32, got %s" % (name, t.dtype))
        wcode = _inputs[t.dtype]
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same dtype")
    return LayerNormArgs(rows, cols, code, wcode, x.data_ptr(), ldx, _ptr(weight), _ptr(bias))


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, save=False):
    """y = (x - mean) / sqrt(var + eps) * weight + bias over the last dimension.

    x: (..., cols), float32, float16 or bfloat16, contiguous or a matrix of
    contiguous rows.  weight, bias: (cols), of x's dtype or float32, or None
    (ones, zeros).  Returns y of x's shape and dtype (``out`` if given, which
    may be x itself), or ``(y, kept)`` with ``save=True``, kept being what
    :func:`layer_norm_backward` needs.  Sums are fp32, and the mean is kept in
    two parts, so that rows far from zero keep their differences.  No autograd
    graph, see :func:`layer_norm_backward`.
    """
    import torch
    a = _layer_norm_args(x, weight, bias)
    if not eps >= 0:
        raise ValueError("eps must be at least 0")
    a.eps = eps
    y = _output(out, x.shape, x.dtype, x.device)
    a.y = y.data_ptr()
    kept = None
    if save:
        kept = LayerNormKept(torch.empty((3, a.rows), dtype=torch.float32, device=x.device), a.rows, a.cols, x.dtype)
        a.stats = kept.stats.data_ptr()
    if a.rows:
        stream = _stream(x.device)
        _check(_lib().gemm_layer_norm(_handle(x.device), ctypes.byref(a), stream), "gemm_layer_norm")
    return (y, kept) if save else y


def layer_norm_backward(dy, x, weight, kept, need=(True, True, True), out=(None, None, None)):
    """Gradients (dx, dweight, dbias) of :func:`layer_norm` from dy and what
    the forward pass kept, with the same x and weight (None: ones).

    dy: x's shape and dtype, contiguous or a matrix of contiguous rows.
    dweight and dbias have weight's dtype (x's without a weight).  need: which
    of the three to compute (None in the place of the others).  out: tensors
    to write them to; dx may be written over dy.  The sums of a row's dy weight
    and dy weight h are fp32: where they leave its range, dx is not finite.
    """
    import torch
    if not isinstance(kept, LayerNormKept):
        raise TypeError("kept must come from layer_norm(..., save=True)")
    lib = _lib()
    a = _layer_norm_args(x, weight, None)
    _on_cuda(x.device, dy, "dy")
    if dy.dtype != x.dtype or dy.shape != x.shape:
        raise ValueError("dy must have x's shape and dtype")
    if (a.rows, a.cols, x.dtype) != kept[1:]:
        raise ValueError("kept belongs to a forward pass of other sizes or dtype")
    stats = kept.stats
    _on_cuda(x.device, stats, "kept.stats")
    if stats.dtype != torch.float32 or stats.shape != (3, a.rows) or not stats.is_contiguous():
        raise ValueError("kept.stats must be contiguous float32 (3, rows)")
    a.dy, a.lddy = dy.data_ptr(), _rows(dy, a.cols, "dy")[1]
    a.stats = stats.data_ptr()
    wdtype = x.dtype if weight is None else weight.dtype
    shapes = ((x.shape, x.dtype, "dx"), ((a.cols,), wdtype, "dweight"), ((a.cols,), wdtype, "dbias"))
    grads = [_output(o, shape, dtype, x.device, name) if want else None
             for want, o, (shape, dtype, name) in zip(need, out, shapes)]
    a.dx, a.dweight, a.dbias = map(_ptr, grads)
    _run("gemm_layer_norm_backward", lib.gemm_layer_norm_backward_workspace, lib.gemm_layer_norm_backward, a, x.device)
    return tuple(grads)


# ----------------------------------------------------------------- AdamW step --

# The states of a list of tensors: step, int64 () on the GPU, the steps made so
# far; exp_avg and exp_avg_sq, one buffer each, every tensor's elements from
# the next multiple of ADAMW_BLOCK on; scales, None (float32 states) or
# float32 (2, blocks).  In 8 bits the states are float8_e4m3fn, to be
# multiplied by their block's scale; exp_avg_sq then holds square roots.
AdamWState = collections.namedtuple("AdamWState", "step exp_avg exp_avg_sq scales")


def adamw_state(params, bits=32):
    """New (zero) states for :func:`adamw` of these tensors, in 32 or 8 bits."""
    import torch
    if bits not in (32, 8):
        raise ValueError("bits must be 32 or 8")
    if not params:
        raise ValueError("params must have at least one tensor")
    device = getattr(params[0], "device", None)
    for p in params:
        _on_cuda(device, p, "params")
    blocks = sum(-(-p.numel() // ADAMW_BLOCK) for p in params)
    size = blocks * ADAMW_BLOCK

    def state():
        return torch.zeros(size, dtype=torch.float32 if bits == 32 else torch.uint8, device=device)
    m, v = state(), state()
    scales = None
    if bits == 8:
        m, v = m.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        scales = torch.zeros((2, blocks), dtype=torch.float32, device=device)
    return AdamWState(torch.zeros((), dtype=torch.int64, device=device), m, v, scales)


@functools.lru_cache(maxsize=64)
def _table(count):
    """Packs `count` gemm_adamw_tensor_t."""
    return struct.Struct("=" + "QQQqiiif" * count)


_dtype_of, _shape_of = operator.attrgetter("dtype"), operator.attrgetter("shape")


def _adamw_list(tensors, name, index, types):
    """(pointers, type codes, shapes) of a list of tensors.  (map, not a loop: a
    step of many small tensors is bound by what the host does for each.)"""
    import torch
    t = torch.Tensor
    try:
        on = set(map(t.get_device, tensors))
        contiguous = all(map(t.is_contiguous, tensors))
        dtypes = list(map(_dtype_of, tensors))
        at, shapes = list(map(t.data_ptr, tensors)), list(map(_shape_of, tensors))
    except TypeError:
        raise ValueError("%s must be CUDA tensors" % name) from None
    if on and on != {index}:
        raise ValueError("%s must be CUDA tensors on the same device as the states" % name)
    if not contiguous:
        raise ValueError("%s must be contiguous" % name)
    if not types.keys() >= set(dtypes):
        raise TypeError("%s must be %s" % (name, " or ".join(str(d)[6:] for d in types)))
    return at, map(types.get, dtypes), shapes


def adamw(params, grads, state, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, copies=None,
          scale=None):
    """One AdamW step of many tensors, in place, on the current CUDA stream.

    With g = scale * grad, m <- b1 m + (1 - b1) g, v <- b2 v + (1 - b2) g^2 and
    p <- p - lr weight_decay p - lr m' / (sqrt(v') + eps), m' and v' being m and
    v over 1 - b^t; all in fp32.

    params, grads: lists of contiguous tensors, float32, float16 or bfloat16
    (16-bit parameters are rounded to nearest after every step, so that a step
    below half of their last bit is lost).  state: :func:`adamw_state` of
    these params; its step is on the GPU and counted there.  lr: a number, or
    a float32 tensor () on the GPU.  weight_decay: a number, or one for each
    tensor.  copies: 16-bit tensors that receive the new parameters, or None
    in the place of one or of all.  scale: float32 tensor () on the GPU that
    every gradient is multiplied by (1 / loss scale, or that of a clipped
    norm); None: 1.  eps: 0, or between 2^-126 and 2^126.  Nothing may overlap
    what is written.

    In 8 bits each block of ADAMW_BLOCK elements has a scale, its largest
    magnitude over 448.  m is rounded to nearest; sqrt(v), which moves by less
    than half a step of the format, up or down, in turns that are spread
    evenly over the steps (so results repeat bit for bit), and never to 0.
    NaN or an infinity makes its whole block NaN.  Elements of the buffers
    between tensors become zero.
    """
    import torch
    lib = _lib()
    step, m, v, scales = state
    _on_cuda(getattr(step, "device", None), step, "state")
    device = step.device
    n = len(params)
    if len(grads) != n or (copies is not None and len(copies) != n):
        raise ValueError("params, grads and copies must have the same length")
    index = device.index
    p_at, p_type, shapes = _adamw_list(params, "params", index, _inputs)
    g_at, g_type, g_shapes = _adamw_list(grads, "grads", index, _inputs)
    if shapes != g_shapes:
        raise ValueError("grads must have the shapes of params")
    c_at, c_type = itertools.repeat(0), itertools.repeat(0)
    if copies is not None:
        there = [i for i, c in enumerate(copies) if c is not None]
        at, codes, c_shapes = _adamw_list([copies[i] for i in there], "copies", index, _sixteen)
        if c_shapes != [shapes[i] for i in there]:
            raise ValueError("copies must have the shapes of params")
        c_at, c_type = [0] * n, [0] * n
        for i, a, c in zip(there, at, codes):
            c_at[i], c_type[i] = a, c
    decay = itertools.repeat(float(weight_decay)) if isinstance(weight_decay, (int, float)) else weight_decay
    if not isinstance(decay, itertools.repeat) and len(decay) != n:
        raise ValueError("weight_decay must be a number, or one for each tensor")
    sizes = list(map(torch.Size.numel, shapes))
    _on_cuda(device, m, "state")
    size = m.numel()
    if scales is None:
        want = ((m, torch.float32, (size,)), (v, torch.float32, (size,)))
    else:
        want = ((m, torch.float8_e4m3fn, (size,)), (v, torch.float8_e4m3fn, (size,)),
                (scales, torch.float32, (2, size // ADAMW_BLOCK)))
    for t, dtype, shape in want + ((step, torch.int64, ()),):
        _on_cuda(device, t, "state")
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError("state belongs to other tensors (see adamw_state)")
    rate = None
    if isinstance(lr, torch.Tensor):
        rate, lr = lr, 0.0
    for t, name in ((rate, "lr"), (scale, "scale")):
        if t is not None:
            _on_cuda(device, t, name)
            if t.dtype != torch.float32 or t.numel() != 1:
                raise ValueError("%s must be one float32" % name)
    table = _table(n).pack(*itertools.chain.from_iterable(
        zip(p_at, g_at, c_at, sizes, p_type, g_type, c_type, decay)))
    a = AdamWArgs(ctypes.cast(table, _vp), n, size, 32 if scales is None else 8, m.data_ptr(), v.data_ptr(), _ptr(scales),
                  step.data_ptr(), lr, _ptr(rate), betas[0], betas[1], eps, _ptr(scale))
    stream = _stream(device)
    _check(lib.gemm_adamw(_handle(device), ctypes.byref(a), stream), "gemm_adamw")
