"""ctypes binding of the rest of the MoE block (include/gfr.h): the dense
product with its epilogue, the router's choice with the tokens in expert order,
and the experts for a few tokens.

Argument marshalling only, like ``_binding``: dtypes, ranks and shapes are
checked by the library, which raises GfrError here.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import _binding as b
from ._binding import GfrError, GfrOptions, _need, _on_device, _ref, tensor_desc

_T, _O, _P = ctypes.POINTER(b.GfrTensor), ctypes.POINTER(GfrOptions), ctypes.c_void_p
_SIZE = ctypes.POINTER(ctypes.c_size_t)

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5}
SCORINGS = {"softmax": 0, "sigmoid": 1}
DECODE_MAX_TOKENS = 64   # GFR_DECODE_MAX_TOKENS

_ready = False


def _lib():
    global _ready
    lib = b.load_library()
    if not _ready:
        lib.gfr_linear.argtypes = [_T] * 4 + [ctypes.c_int, _T, _P, _O]
        lib.gfr_linear_workspace_size.argtypes = [_T] * 4 + [ctypes.c_int, _T, _SIZE]
        lib.gfr_moe_decode.argtypes = [_T] * 8 + [ctypes.c_float, _T, ctypes.c_int, ctypes.c_int,
                                                  _P, _O]
        lib.gfr_moe_decode_workspace_size.argtypes = [ctypes.c_int64] * 6 + \
            [ctypes.c_int] * 2 + [_SIZE]
        lib.gfr_moe_route.argtypes = [_T, _T] + [ctypes.c_int] * 4 + [ctypes.c_float] + \
            [_T] * 8 + [_P, _O]
        lib.gfr_moe_route_workspace_size.argtypes = [ctypes.c_int64] * 3 + [_SIZE]
        for f in (lib.gfr_linear, lib.gfr_linear_workspace_size, lib.gfr_moe_decode,
                  lib.gfr_moe_decode_workspace_size, lib.gfr_moe_route,
                  lib.gfr_moe_route_workspace_size):
            f.restype = ctypes.c_int
        _ready = True
    return lib


def _check(rc: int):
    if rc:
        raise GfrError(rc, b.status_string(rc))


@contextlib.contextmanager
def _on_stream(dev, stream: Optional[int]):
    """The call's device and stream made current, so that what is allocated
    within belongs to the stream that uses it; gives the stream's handle."""
    if stream is None:
        with torch.cuda.device(dev):
            yield torch.cuda.current_stream(dev).cuda_stream
    else:
        s = torch.cuda.ExternalStream(stream, device=dev) if stream else \
            torch.cuda.default_stream(dev)
        with torch.cuda.stream(s):
            yield stream


def _workspace(given, need: int, dev):
    """The caller's workspace, or a new one of `need` bytes (None for none)."""
    if given is not None or need == 0:
        return given
    return torch.empty(need, dtype=torch.uint8, device=dev)


def _options(workspace, status=None):
    if workspace is None:
        return GfrOptions(0, None, 0, None if status is None else status.data_ptr(), 0, 0)
    return GfrOptions(0, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                      None if status is None else status.data_ptr(), 0, 0)


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
    dev = x.device
    _need(activation in ACTIVATIONS, f"activation must be one of {sorted(ACTIVATIONS)}")
    _need(x.dim() == 2 and w.dim() == 2, "x must be [M, K] and w [N, K]")
    _on_device([x, w, bias, residual, out, workspace], dev)
    if out is not None:
        _need(out_dtype is None or out.dtype == out_dtype, "out must have out_dtype")
    act = ACTIVATIONS[activation]
    with _on_stream(dev, stream) as handle:
        if out is None:
            n = w.shape[0] // 2 if act == 5 else w.shape[0]
            out = torch.empty((x.shape[0], n), dtype=out_dtype or x.dtype, device=dev)
        d = [tensor_desc(t) for t in (x, w, bias, residual)]
        do = tensor_desc(out)
        need = ctypes.c_size_t(0)
        _check(lib.gfr_linear_workspace_size(*map(_ref, d), act, _ref(do), ctypes.byref(need)))
        workspace = _workspace(workspace, need.value, dev)
        _check(lib.gfr_linear(*map(_ref, d), act, _ref(do), handle,
                              ctypes.byref(_options(workspace))))
    return out


def moe_decode_workspace_size(T: int, k: int, E: int, H: int, I: int, N: int,
                              transpose_w13: bool = False, transpose_w2: bool = False) -> int:
    """Workspace bytes of a moe_decode call of these sizes."""
    need = ctypes.c_size_t(0)
    _check(_lib().gfr_moe_decode_workspace_size(
        T, k, E, H, I, N, int(bool(transpose_w13)), int(bool(transpose_w2)), ctypes.byref(need)))
    return need.value


def moe_decode(x, w13, scale13, w2, scale2, topk_ids, topk_weights, *, transpose_w13=False,
               transpose_w2=False, shared_input=None, shared_input_weight=1.0,
               out_dtype=torch.bfloat16, out=None, workspace=None, status=None, stream=None):
    """The experts of a MoE block for at most DECODE_MAX_TOKENS tokens, in three
    launches (include/gfr.h, gfr_moe_decode); returns out.

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
    dev = x.device
    _need(x.dim() == 2 and w2.dim() == 3 and topk_ids.dim() == 2,
          "x must be [T, H], w2 3-D and topk_ids [T, k]")
    _on_device([x, w13, scale13, w2, scale2, topk_ids, topk_weights, shared_input, out,
                workspace, status], dev)
    T, k = topk_ids.shape
    E, I, N = w2.shape
    if transpose_w2:
        I, N = N, I
    with _on_stream(dev, stream) as handle:
        if out is None:
            out = torch.empty((x.shape[0], N), dtype=out_dtype, device=dev)
        if workspace is None:
            workspace = _workspace(None, moe_decode_workspace_size(
                T, k, E, x.shape[1], I, N, transpose_w13, transpose_w2), dev)
        d = [tensor_desc(t) for t in (x, w13, scale13, w2, scale2, topk_ids, topk_weights,
                                      shared_input, out)]
        _check(lib.gfr_moe_decode(*map(_ref, d[:8]), float(shared_input_weight), _ref(d[8]),
                                  int(bool(transpose_w13)), int(bool(transpose_w2)), handle,
                                  ctypes.byref(_options(workspace, status))))
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
    the topk_group best of n_group equal runs of experts; the weights are the
    chosen scores, summing to 1 under renormalize, times scaling.

    Returns topk_ids int32 [T, k] (-1 where a row has too few live experts),
    topk_weights float32 [T, k] and, with x bfloat16 or float16 [T, H]:
    xin out_dtype [T k, H] and xin_scale uint8 [T k, ceil(H/64), 2] (token rows
    MX-quantised, for gemm1_swiglu_quant), group_list int64 [E] (counts,
    group_list_type 1), row_index int32 [T k] and logit float32 [T k] (for
    gmm_finalize_routing).
    """
    lib = _lib()
    dev = logits.device
    _need(scoring in SCORINGS, f"scoring must be one of {sorted(SCORINGS)}")
    _need(logits.dim() == 2, "logits must be [T, E]")
    _need(x is None or x.dim() == 2, "x must be [T, H]")
    _on_device([logits, bias, x, workspace], dev)
    T, E = logits.shape
    k = int(top_k)
    _need(k >= 1, "top_k must be positive")
    with _on_stream(dev, stream) as handle:
        r = RouteResult(torch.empty((T, k), dtype=torch.int32, device=dev),
                        torch.empty((T, k), dtype=torch.float32, device=dev))
        if x is not None:
            H, n = x.shape[1], T * k
            r = RouteResult(
                r.topk_ids, r.topk_weights,
                torch.empty((n, H), dtype=out_dtype, device=dev),
                torch.empty((n, (H + 63) // 64, 2), dtype=torch.uint8, device=dev),
                torch.empty(E, dtype=torch.int64, device=dev),
                torch.empty(n, dtype=torch.int32, device=dev),
                torch.empty(n, dtype=torch.float32, device=dev))
            need = ctypes.c_size_t(0)
            _check(lib.gfr_moe_route_workspace_size(T, E, k, ctypes.byref(need)))
            workspace = _workspace(workspace, need.value, dev)
        d = [tensor_desc(t) for t in (logits, bias, r.topk_ids, r.topk_weights, x, *r[2:])]
        _check(lib.gfr_moe_route(_ref(d[0]), _ref(d[1]), SCORINGS[scoring], int(n_group),
                                 int(topk_group), int(bool(renormalize)), float(scaling),
                                 *map(_ref, d[2:]), handle, ctypes.byref(_options(workspace))))
    return r
