"""ctypes binding of the rest of the MoE block (include/gfr.h): the dense
product with its epilogue, the router's choice with the tokens in expert order,
and the experts for a few tokens.

Argument marshalling only, like ``_binding``: dtypes, ranks and shapes are
checked by the library, which raises GfrError here.
"""
from __future__ import annotations

import array
import ctypes
import functools
from typing import NamedTuple, Optional

import torch

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
        for f in (lib.gfr_linear, lib.gfr_linear_workspace_size, lib.gfr_moe_decode,
                  lib.gfr_moe_decode_workspace_size, lib.gfr_moe_route,
                  lib.gfr_moe_route_workspace_size):
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
