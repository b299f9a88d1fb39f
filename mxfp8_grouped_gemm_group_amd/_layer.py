"""ctypes binding of the rest of the MoE block (include/gfr.h): the dense
product with its epilogue, the router's choice with the tokens in expert order,
the experts for a few tokens, the experts' products in 16 bits with their
gradients, and the dense product with an adapter per request.

Argument marshalling only, like ``_binding``: dtypes, ranks and shapes are
checked by the library, which raises GfrError here.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from . import _binding as b
from ._binding import GfrError, _need

_P = ctypes.c_void_p
_SIZE = ctypes.POINTER(ctypes.c_size_t)

# The grouped calls take no float16: their binding refuses it by itself.
DTYPES = {**b.DTYPES, torch.float16: 11}

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5}
SCORINGS = {"softmax": 0, "sigmoid": 1}
DECODE_MAX_TOKENS = 64   # GFR_DECODE_MAX_TOKENS
WORKSPACE_TOO_SMALL = 6  # GFR_ERR_WORKSPACE_TOO_SMALL

_ready = False


def _lib():
    global _ready
    lib = b.load_library()
    if not _ready:
        i = ctypes.c_int
        # descriptors and options are passed by address (_pack)
        lib.gfr_linear.argtypes = [_P] * 4 + [i] + [_P] * 3
        lib.gfr_linear_workspace_size.argtypes = [_P] * 4 + [i, _P, _SIZE]
        lib.gfr_moe_decode.argtypes = [_P] * 8 + [ctypes.c_float, _P, i, i] + [_P] * 2
        lib.gfr_moe_decode_workspace_size.argtypes = [ctypes.c_int64] * 6 + [i, i, _SIZE]
        lib.gfr_moe_route.argtypes = [_P] * 2 + [i] * 4 + [ctypes.c_float] + [_P] * 10
        lib.gfr_moe_route_workspace_size.argtypes = [ctypes.c_int64] * 3 + [_SIZE]
        lib.gfr_grouped_linear.argtypes = [_P] * 3 + [i] * 3 + [_P] * 3
        lib.gfr_grouped_linear_wgrad.argtypes = [_P] * 3 + [i] * 3 + [_P] * 3
        lib.gfr_lora_linear.argtypes = [_P] * 11
        lib.gfr_lora_linear_workspace_size.argtypes = [ctypes.c_int64] * 4 + [_SIZE]
        for f in (lib.gfr_linear, lib.gfr_linear_workspace_size, lib.gfr_moe_decode,
                  lib.gfr_moe_decode_workspace_size, lib.gfr_moe_route,
                  lib.gfr_moe_route_workspace_size, lib.gfr_grouped_linear,
                  lib.gfr_grouped_linear_wgrad, lib.gfr_lora_linear,
                  lib.gfr_lora_linear_workspace_size):
            f.restype = i
        _ready = True
    return lib


def _check(rc: int):
    if rc:
        raise GfrError(rc, b.status_string(rc))


@functools.lru_cache(maxsize=16384)
def _words(dtype, shape):
    """A gfr_tensor's 64-bit words behind its address."""
    code, n = DTYPES.get(dtype), len(shape)
    if code is None:
        raise ValueError(f"dtype {dtype} has no gfr_dtype")
    if not 1 <= n <= 4:
        raise ValueError(f"rank {n} is outside 1..4")
    return (code | n << 32, *shape, *(0,) * (4 - n))


def _pack(index, tensors, made=(), workspace=None, status=None):
    """The tensors' gfr_tensor descriptors and a gfr_options behind them in one
    array of 64-bit words, and their addresses (None for an absent tensor).  One
    array costs a fraction of a ctypes structure per tensor, and the smallest
    calls take little longer on the GPU than that.  ``made``, behind ``tensors``,
    were allocated by the caller of this and need no check.  The array has to
    outlive the call.  Raises for what the descriptors cannot carry."""
    v, at = [], []
    for t in tensors:
        if t is None:
            at.append(None)
            continue
        if t.get_device() != index:
            raise ValueError("all tensors must be on one CUDA device")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        at.append(8 * len(v))
        v.append(t.data_ptr())
        v += _words(t.dtype, t.shape)
    for t in made:
        if t is None:
            at.append(None)
            continue
        at.append(8 * len(v))
        v.append(t.data_ptr())
        v += _words(t.dtype, t.shape)
    end = 8 * len(v)
    v += (0, 0, 0, 0, 0)
    for t in (workspace, status):
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            raise ValueError("workspace and status must be contiguous and on the tensors' device")
    if workspace is not None:
        v[-4], v[-3] = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if status is not None:
        _need(status.dtype == torch.int32 and status.numel() >= 1, "status must be int32")
        v[-2] = status.data_ptr()
    words = array.array("q", v)
    base = words.buffer_info()[0]
    return words, [None if a is None else base + a for a in at], base + end


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(index: int, stream: Optional[int]):
    """A context that makes the call's device and stream current, so that what is
    allocated within belongs to the stream that uses it; None if they are."""
    if stream is not None:
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=index) if stream
                                 else torch.cuda.default_stream(index))
    return None if index == torch.cuda.current_device() else torch.cuda.device(index)


def _tracked(*tensors) -> bool:
    """Whether a result made from the tensors owes autograd a derivative: a gradient, or
    the tangent of a forward-mode level."""
    if torch.is_grad_enabled():
        for t in tensors:               # (any() takes half a microsecond more)
            if t is not None and t.requires_grad:
                return True
    return forward_ad._current_level >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _device(t, name: str) -> int:
    index = t.get_device()
    _need(index >= 0, f"{name} must be on a CUDA device")
    return index


def linear(x, w, bias=None, *, activation="none", residual=None, out_dtype=None, out=None,
           workspace=None, stream=None):
    """act(x @ w.T + bias) + residual in one pass, accumulated in FP32
    (include/gfr.h, gfr_linear); returns out.

    x [M, K] and w [N, K] bfloat16 or float16; activation "none", "relu",
    "silu", "gelu", "gelu_tanh" or "swiglu" (then w is [2N, K], gate rows
    before up rows); bias [w's rows] in x's dtype or float32; residual [M, N]
    in x's dtype (may be out); out_dtype x's (default) or float32.
    """
    lib = _lib()
    act = ACTIVATIONS.get(activation)
    _need(act is not None, f"activation must be one of {sorted(ACTIVATIONS)}")
    index = _device(x, "x")
    _need(x.dim() == 2 and w.dim() == 2, "x must be [M, K] and w [N, K]")
    _need(out is None or out_dtype is None or out.dtype == out_dtype, "out must have out_dtype")
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return linear(x, w, bias, activation=activation, residual=residual,
                          out_dtype=out_dtype, out=out, workspace=workspace)
    tensors, made = (x, w, bias, residual), ()
    if out is None:
        n = w.shape[0] // 2 if act == 5 else w.shape[0]
        out = x.new_empty((x.shape[0], n), dtype=out_dtype or x.dtype)
        made = (out,)
    else:
        tensors += (out,)
    handle = _raw_stream(index)
    words, (px, pw, pb, pr, po), opts = _pack(index, tensors, made, workspace)
    rc = lib.gfr_linear(px, pw, pb, pr, act, po, handle, opts)
    if rc == WORKSPACE_TOO_SMALL and workspace is None:
        need = ctypes.c_size_t(0)
        _check(lib.gfr_linear_workspace_size(px, pw, pb, pr, act, po, ctypes.byref(need)))
        workspace = x.new_empty(need.value, dtype=torch.uint8)
        words, (px, pw, pb, pr, po), opts = _pack(index, tensors, made, workspace)
        rc = lib.gfr_linear(px, pw, pb, pr, act, po, handle, opts)
    _check(rc)
    return out


@functools.lru_cache(maxsize=4096)
def moe_decode_workspace_size(T: int, k: int, E: int, H: int, I: int, N: int,
                              transpose_w13: bool = False, transpose_w2: bool = False) -> int:
    """Workspace bytes of a moe_decode call of these sizes."""
    need = ctypes.c_size_t(0)
    _check(_lib().gfr_moe_decode_workspace_size(
        T, k, E, H, I, N, int(bool(transpose_w13)), int(bool(transpose_w2)), ctypes.byref(need)))
    return need.value


@functools.lru_cache(maxsize=4096)
def _decode_sizes(x, w2, topk_ids, transpose_w13, transpose_w2):
    """out's shape and the workspace bytes of a call with tensors of these shapes."""
    _need(len(x) == 2 and len(w2) == 3 and len(topk_ids) == 2,
          "x must be [T, H], w2 3-D and topk_ids [T, k]")
    E, I, N = (w2[0], w2[2], w2[1]) if transpose_w2 else w2
    return (x[0], N), moe_decode_workspace_size(*topk_ids, E, x[1], I, N, transpose_w13,
                                                transpose_w2)


def moe_decode(x, w13, scale13, w2, scale2, topk_ids, topk_weights, *, transpose_w13=False,
               transpose_w2=False, shared_input=None, shared_input_weight=1.0,
               out_dtype=torch.bfloat16, out=None, workspace=None, status=None, stream=None):
    """The experts of a MoE block for at most DECODE_MAX_TOKENS tokens
    (include/gfr.h, gfr_moe_decode); returns out.

    out[t] = sum_j topk_weights[t, j] * swiglu(x[t] @ w13[e]) @ w2[e]
             + shared_input_weight * shared_input[t],   e = topk_ids[t, j]

    x bfloat16 [T, H]; w13, scale13 as gemm1_swiglu_quant's w13 and scale; w2,
    scale2 as gmm_finalize_routing's x2 and scale (float8); topk_ids int32
    [T, k] (-1: no expert), topk_weights float32 [T, k]; shared_input bfloat16
    [T, N] or None; out bfloat16 or float32 [T, N], overwritten.  ``status``
    (int32, 1 element) receives DEV_BAD_EXPERT if an id is out of range.
    ``workspace`` (uint8, moe_decode_workspace_size bytes) is allocated here if
    none is given; calls that overlap in time need one each.
    """
    lib = _lib()
    index = _device(x, "x")
    t13, t2 = int(bool(transpose_w13)), int(bool(transpose_w2))
    shape, need = _decode_sizes(x.shape, w2.shape, topk_ids.shape, t13, t2)
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return moe_decode(x, w13, scale13, w2, scale2, topk_ids, topk_weights,
                              transpose_w13=transpose_w13, transpose_w2=transpose_w2,
                              shared_input=shared_input, shared_input_weight=shared_input_weight,
                              out_dtype=out_dtype, out=out, workspace=workspace, status=status)
    tensors, made = (x, w13, scale13, w2, scale2, topk_ids, topk_weights, shared_input), ()
    if out is None:
        out = x.new_empty(shape, dtype=out_dtype)
        made = (out,)
    else:
        tensors += (out,)
    if workspace is None:
        workspace = x.new_empty(need, dtype=torch.uint8)
    words, at, opts = _pack(index, tensors, made, workspace, status)
    _check(lib.gfr_moe_decode(*at[:8], float(shared_input_weight), at[8], t13, t2,
                              _raw_stream(index), opts))
    return out


class RouteResult(NamedTuple):
    """moe_route's outputs; those after topk_weights are None without x."""
    topk_ids: torch.Tensor
    topk_weights: torch.Tensor
    xin: Optional[torch.Tensor] = None
    xin_scale: Optional[torch.Tensor] = None
    group_list: Optional[torch.Tensor] = None
    row_index: Optional[torch.Tensor] = None
    logit: Optional[torch.Tensor] = None


def moe_route(logits, top_k, *, x=None, bias=None, scoring="softmax", n_group=1, topk_group=1,
              renormalize=True, scaling=1.0, out_dtype=torch.float8_e4m3fn, workspace=None,
              stream=None) -> RouteResult:
    """A router's choice of top_k experts from its logits and, with x, the inputs
    of the grouped calls in expert order (include/gfr.h, gfr_moe_route).

    logits float32 or bfloat16 [T, E]; scoring "softmax" or "sigmoid"; bias
    float32 [E] is added to the scores for the choice only; n_group > 1 keeps
    the topk_group best of n_group equal runs of experts, by the sum of each
    run's two largest scores (with bias; not by the largest one); the weights are the
    chosen scores, summing to 1 under renormalize, times scaling.

    Returns topk_ids int32 [T, k] (-1 where a row has too few live experts),
    topk_weights float32 [T, k] and, with x bfloat16 or float16 [T, H]:
    xin out_dtype [T k, H] and xin_scale uint8 [T k, ceil(H/64), 2] (token rows
    MX-quantised, for gemm1_swiglu_quant), group_list int64 [E] (counts,
    group_list_type 1), row_index int32 [T k] and logit float32 [T k] (for
    gmm_finalize_routing).
    """
    lib = _lib()
    score = SCORINGS.get(scoring)
    _need(score is not None, f"scoring must be one of {sorted(SCORINGS)}")
    _need(logits.dim() == 2, "logits must be [T, E]")
    _need(x is None or x.dim() == 2, "x must be [T, H]")
    T, E = logits.shape
    k = int(top_k)
    _need(k >= 1, "top_k must be positive")
    index = _device(logits, "logits")
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return moe_route(logits, top_k, x=x, bias=bias, scoring=scoring, n_group=n_group,
                             topk_group=topk_group, renormalize=renormalize, scaling=scaling,
                             out_dtype=out_dtype, workspace=workspace)
    empty = logits.new_empty
    ids, weights = empty((T, k), dtype=torch.int32), empty((T, k), dtype=torch.float32)
    rows = (None,) * 5
    if x is not None:
        H, n = x.shape[1], T * k
        rows = (empty((n, H), dtype=out_dtype),
                empty((n, (H + 63) // 64, 2), dtype=torch.uint8),
                empty(E, dtype=torch.int64),
                empty(n, dtype=torch.int32),
                empty(n, dtype=torch.float32))
        if workspace is None:
            need = _route_workspace_size(T, E, k)
            if need:
                workspace = empty(need, dtype=torch.uint8)
    words, at, opts = _pack(index, (logits, bias, x), (ids, weights, *rows), workspace)
    _check(lib.gfr_moe_route(at[0], at[1], score, int(n_group), int(topk_group),
                             int(bool(renormalize)), float(scaling), at[3], at[4], at[2],
                             *at[5:], _raw_stream(index), opts))
    return RouteResult(ids, weights, *rows)


@functools.lru_cache(maxsize=4096)
def _route_workspace_size(T: int, E: int, k: int) -> int:
    need = ctypes.c_size_t(0)
    _check(_lib().gfr_moe_route_workspace_size(T, E, k, ctypes.byref(need)))
    return need.value


def _grouped(x, w, group_list, group_list_type, transpose_w, out_dtype, out, status):
    index = _device(x, "x")
    _need(x.dim() == 2 and w.dim() == 3, "x must be [M, K] and w 3-D")
    tensors, made, fill = (x, w, group_list), (), 0
    if out is None:
        n = w.shape[1] if transpose_w else w.shape[2]
        out = x.new_empty((x.shape[0], n), dtype=out_dtype or x.dtype)
        made, fill = (out,), 1
    else:
        tensors += (out,)
    words, (px, pw, pg, po), opts = _pack(index, tensors, made, None, status)
    _check(_lib().gfr_grouped_linear(px, pw, pg, group_list_type, int(bool(transpose_w)), fill, po,
                                     _raw_stream(index), opts))
    return out


def _wgrad(x, dy, group_list, group_list_type, transpose_w, out_dtype, out, accumulate, status):
    index = _device(x, "x")
    _need(x.dim() == 2 and dy.dim() == 2, "x must be [M, K] and dy [M, N]")
    tensors, made = (x, dy, group_list), ()
    if out is None:
        shape = (dy.shape[1], x.shape[1]) if transpose_w else (x.shape[1], dy.shape[1])
        out = x.new_empty((group_list.numel(), *shape), dtype=out_dtype or x.dtype)
        made = (out,)
    else:
        tensors += (out,)
    words, (px, pd, pg, po), opts = _pack(index, tensors, made, None, status)
    _check(_lib().gfr_grouped_linear_wgrad(px, pd, pg, group_list_type, int(bool(transpose_w)),
                                           int(bool(accumulate)), po, _raw_stream(index), opts))
    return out


class _GroupedLinear(torch.autograd.Function):
    """grouped_linear with its two gradients, each one launch."""

    @staticmethod
    def forward(ctx, x, w, group_list, group_list_type, transpose_w, out_dtype, status):
        # (each gradient's product takes the other operand)
        dx, dw = ctx.needs_input_grad[:2]
        ctx.save_for_backward(x if dw else None, w if dx else None, group_list)
        ctx.args = group_list_type, transpose_w, x.shape, x.dtype
        return _grouped(x, w, group_list, group_list_type, transpose_w, out_dtype, None, status)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, group_list = ctx.saved_tensors
        group_list_type, transpose_w, shape, dtype = ctx.args
        # (an FP32 result's gradient comes in FP32: the products take x's type)
        dy = dy.to(dtype).contiguous()
        if dy.data_ptr() % 16:               # (a view that begins anywhere, as cat hands on)
            dy = dy.clone()
        away = _elsewhere(dy.get_device(), None)
        with away if away is not None else contextlib.nullcontext():
            dx = dw = None
            if ctx.needs_input_grad[0]:      # (no columns: a product has to sum over some)
                dx = dy.new_zeros(shape) if dy.shape[1] == 0 else _grouped(
                    dy, w, group_list, group_list_type, not transpose_w, dtype, None, None)
            if ctx.needs_input_grad[1]:
                dw = _wgrad(x, dy, group_list, group_list_type, transpose_w, dtype, None, False,
                            None)
        return dx, dw, None, None, None, None, None


def grouped_linear(x, w, group_list, group_list_type, *, transpose_w=False, out_dtype=None,
                   out=None, status=None, stream=None):
    """Rows sorted by expert times their expert's 16-bit weights, accumulated in
    FP32 (include/gfr.h, gfr_grouped_linear); returns out.

    x bfloat16 or float16 [M, K]; w x's dtype [E, K, N], or [E, N, K] with
    transpose_w; group_list int64 [E] (0: prefix sums, 1: counts); out_dtype x's
    (default) or float32.  Rows of no expert's range are left as they were in
    ``out``, and zeros in one that the call allocates.  ``status`` (int32, 1
    element) receives DEV_BAD_GROUP_LIST.

    Differentiable by x and w (then ``out`` has to be None): their gradients have
    their dtypes; dy is rounded to x's dtype first where out_dtype is float32.
    Gradients kept in float32 take grouped_linear_wgrad.  Forward-mode derivatives are
    refused (NotImplementedError).  A step that is captured into a graph needs leaves of
    which no eager graph is alive, as every autograd function does.
    """
    index = _device(x, "x")
    _need(out is None or out_dtype is None or out.dtype == out_dtype, "out must have out_dtype")
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return grouped_linear(x, w, group_list, group_list_type, transpose_w=transpose_w,
                                  out_dtype=out_dtype, out=out, status=status)
    if _tracked(x, w):
        _need(out is None, "out must be None where a gradient is wanted")
        return _GroupedLinear.apply(x, w, group_list, int(group_list_type), bool(transpose_w),
                                    out_dtype, status)
    return _grouped(x, w, group_list, int(group_list_type), transpose_w, out_dtype, out, status)


def grouped_linear_wgrad(x, dy, group_list, group_list_type, *, transpose_w=False, out_dtype=None,
                         out=None, accumulate=False, status=None, stream=None):
    """The gradient of grouped_linear by its weights (include/gfr.h,
    gfr_grouped_linear_wgrad): out[e] = x[rows of e].T @ dy[rows of e], or its
    transpose with transpose_w; returns out.

    x bfloat16 or float16 [M, K], dy x's dtype [M, N]; out_dtype x's (default) or
    float32; ``accumulate`` adds to ``out`` (which must be given).  Not differentiable
    itself: autograd does not see the call.
    """
    index = _device(x, "x")
    _need(out is None or out_dtype is None or out.dtype == out_dtype, "out must have out_dtype")
    _need(out is not None or not accumulate, "accumulate needs an out to add to")
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return grouped_linear_wgrad(x, dy, group_list, group_list_type,
                                        transpose_w=transpose_w, out_dtype=out_dtype, out=out,
                                        accumulate=accumulate, status=status)
    return _wgrad(x, dy, group_list, int(group_list_type), transpose_w, out_dtype, out, accumulate,
                  status)


@functools.lru_cache(maxsize=4096)
def lora_linear_workspace_size(M: int, N: int, K: int, r: int) -> int:
    """Workspace bytes of a lora_linear call of these sizes."""
    need = ctypes.c_size_t(0)
    _check(_lib().gfr_lora_linear_workspace_size(M, N, K, r, ctypes.byref(need)))
    return need.value


def lora_linear(x, w, lora_a, lora_b, adapter_ids, *, scaling=None, bias=None, residual=None,
                out_dtype=None, out=None, workspace=None, status=None, stream=None):
    """x @ w.T + bias + residual and beside it the low-rank adapter of each row's own
    request (include/gfr.h, gfr_lora_linear); returns out.

    out[t] = x[t] @ w.T + bias + scaling[i] * (x[t] @ lora_a[i].T) @ lora_b[i].T
             + residual[t],   i = adapter_ids[t]

    x bfloat16 or float16 [M, K]; w [N, K], lora_a [L, r, K], lora_b [L, N, r] and
    residual [M, N] of x's dtype (residual may be out); adapter_ids int32 [M] (-1:
    no adapter), in any order; scaling float32 [L] or None (1); bias [N] in x's
    dtype or float32; out_dtype x's (default) or float32.  ``status`` (int32, 1
    element) receives DEV_BAD_ADAPTER if an id is out of range.  ``workspace``
    (uint8, lora_linear_workspace_size bytes) is allocated here if none is given;
    calls that overlap in time need one each.

    Has no gradients: where autograd wants one, the result can be used (``out`` has to be
    None), but its backward pass raises RuntimeError.  Adapters are trained over rows sorted
    by adapter, with grouped_linear.
    """
    index = _device(x, "x")
    _need(x.dim() == 2 and w.dim() == 2 and lora_a.dim() == 3,
          "x must be [M, K], w [N, K] and lora_a [L, r, K]")
    _need(out is None or out_dtype is None or out.dtype == out_dtype, "out must have out_dtype")
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return lora_linear(x, w, lora_a, lora_b, adapter_ids, scaling=scaling, bias=bias,
                               residual=residual, out_dtype=out_dtype, out=out,
                               workspace=workspace, status=status)
    operands = (x, w, bias, residual, lora_a, lora_b, adapter_ids, scaling)
    if _tracked(x, w, bias, residual, lora_a, lora_b, scaling):
        _need(out is None, "out must be None where a gradient is wanted")
        return _LoraLinear.apply(out_dtype, workspace, status, *operands)
    return _lora(index, operands, out_dtype, out, workspace, status)


def _lora(index, operands, out_dtype, out, workspace, status):
    x, w, _, _, lora_a = operands[:5]
    M, N = x.shape[0], w.shape[0]
    tensors, made = operands, ()
    if out is None:
        out = x.new_empty((M, N), dtype=out_dtype or x.dtype)
        made = (out,)
    else:
        tensors += (out,)
    if workspace is None:
        workspace = x.new_empty(lora_linear_workspace_size(M, N, x.shape[1], lora_a.shape[1]),
                                dtype=torch.uint8)
    words, at, opts = _pack(index, tensors, made, workspace, status)
    _check(_lib().gfr_lora_linear(*at, _raw_stream(index), opts))
    return out


class _LoraLinear(torch.autograd.Function):
    """lora_linear for autograd: a result whose gradient is refused, not lost."""

    @staticmethod
    def forward(ctx, out_dtype, workspace, status, *operands):
        return _lora(operands[0].get_device(), operands, out_dtype, None, workspace, status)

    @staticmethod
    def backward(ctx, dy):
        raise RuntimeError("lora_linear has no gradients: train adapters with grouped_linear")
