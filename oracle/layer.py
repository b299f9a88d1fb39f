"""CPU oracle, in float64, for the operators around the grouped products of a
MoE block: the dense product with its epilogue, the experts for a few tokens,
and the router's choice with the pairs in expert order.

TEST INFRASTRUCTURE ONLY (like the rest of this package).  Definitions as
include/gfr.h states them; the MX formats and the quantisation are
``oracle.gemm1``'s.  Besides its result each product returns the bound of what
FP32 summation in any order may be off by: a sum of K products, each exact,
rounded at most once per addition, with every partial sum at most
``mag = sum |products|``, errs by at most K 2^-23 mag (2^-23: the matrix unit
may truncate).
"""
from __future__ import annotations

import numpy as np
from scipy.special import erfc, expit

from .gemm1 import fp8_decode, mx_quantize, silu

ULP = 2.0 ** -23
SILU_SLOPE = 1.1       # |d silu / dv| <= 1.0998
GELU_SLOPE = 1.13      # of both gelu forms


def activate(v, act: str):
    if act == "none":
        return v
    if act == "relu":
        return np.where(v < 0, 0.0, v)
    if act == "silu":
        return silu(v)
    if act == "gelu":
        # erfc and expit: 1 + erf and 1 + tanh cancel below zero
        return 0.5 * v * erfc(v / -np.sqrt(2.0))
    if act == "gelu_tanh":
        return v * expit(2 * _tanh_arg(v))
    raise ValueError(act)


def _tanh_arg(v):
    return np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)


def activation_error(v, act: str):
    """What an FP32 evaluation of the activation at an exact v may be off by, relative
    to its result: a few units in the last place (16 for erfc, the bound OpenCL sets),
    and what the rounding of the function's argument makes of the result.  erfc(x)
    changes by at most 2 x^2 + 1 = v^2 + 1 times a relative change of x, here one
    product and its constant (1.5 2^-24); exp(-2u) by 2u times that of u, here six
    roundings (6 2^-24)."""
    if act in ("none", "relu"):
        return np.zeros_like(v)
    if act == "gelu":
        return 2.0 ** -19 + (v * v + 1) * 2.0 ** -23
    if act == "gelu_tanh":
        return 2.0 ** -20 + np.abs(2 * _tanh_arg(v)) * 6 * 2.0 ** -24
    return np.full_like(v, 2.0 ** -20)


def linear(x, w, bias, act: str, residual):
    """(result, bound of the FP32 computation before out's rounding)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    K = x.shape[1]
    y = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    if bias is not None:
        y = y + bias
        mag = mag + np.abs(bias)
    d = (K + 1) * ULP * mag
    if act == "swiglu":
        n = w.shape[0] // 2
        g, u, dg, du = y[:, :n], y[:, n:], d[:, :n], d[:, n:]
        out = silu(g) * u
        d = SILU_SLOPE * (np.abs(u) + du) * dg + np.abs(silu(g)) * du
    else:
        out = activate(y, act)
        d = d * (1.0 if act in ("none", "relu") else GELU_SLOPE)
    # the activation's own FP32 evaluation (2^-40: results below that are not told
    # from zero)
    if act == "swiglu":
        d = d + 2.0 ** -20 * np.abs(out) + 2.0 ** -40
    elif act != "none":
        d = d + activation_error(y, act) * np.abs(out) + 2.0 ** -40
    if residual is not None:
        out = out + residual
        d = d + ULP * np.abs(out)
    return out, d


def half_step(v, mbits: int, emin: int):
    """Half the distance between neighbours of |v| in a format with mbits
    mantissa bits and smallest normal exponent emin."""
    a = np.maximum(np.abs(v), 2.0 ** emin)
    return 2.0 ** (np.floor(np.log2(a)) - mbits - 1)


def mx_weights(codes, scale, transpose: bool, kind: int):
    """[E, K, N] values of MX weights (codes uint8 [E, K, N] or [E, N, K], scale
    uint8, shared or with a leading expert axis)."""
    v = fp8_decode(codes, kind)
    f = np.ldexp(1.0, np.asarray(scale, np.int64) - 127)
    if f.ndim == 3:
        f = f[None]
    if transpose:
        f = np.repeat(f.reshape(f.shape[0], f.shape[1], -1), 32, axis=2)[:, :, :v.shape[2]]
        return (v * f).transpose(0, 2, 1)
    f = f.transpose(0, 1, 3, 2).reshape(f.shape[0], -1, f.shape[2])
    return v * np.repeat(f, 32, axis=1)[:, :v.shape[1]]


def moe_decode(x, w13, w2, ids, weights, shared=None, shared_weight=1.0):
    """(result, bound before out's rounding).  w13 [E, H, 2I], w2 [E, I, N]
    float64.  Ids outside [0, E) are no expert.  silu(gate) * up is an FP32 value,
    summed as three bf16 terms that add up to it."""
    x = np.asarray(x, np.float64)
    T, H = x.shape
    E, I, N = w2.shape
    out, bound = np.zeros((T, N)), np.zeros((T, N))
    mags = np.zeros((T, N))
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e < 0 or e >= E:
                continue
            gu = x[t] @ w13[e]
            d = H * ULP * (np.abs(x[t]) @ np.abs(w13[e]))
            g, u, dg, du = gu[:I], gu[I:], d[:I], d[I:]
            h = silu(g) * u
            dh = SILU_SLOPE * (np.abs(u) + du) * dg + np.abs(silu(g)) * du
            dh = dh + 2.0 ** -20 * np.abs(h)
            a = np.abs(w2[e])
            wt = float(weights[t, j])
            out[t] += wt * (h @ w2[e])
            m = np.abs(wt) * (np.abs(h) @ a)
            # three terms: three times the additions
            bound[t] += np.abs(wt) * (dh @ a) + 3 * I * ULP * m
            mags[t] += m
    if shared is not None:
        s = float(shared_weight) * np.asarray(shared, np.float64)
        out += s
        mags += np.abs(s)
    # joining the pairs' sums, which come in pieces of 64 rows of I or more; weighting;
    # the shared term's product and addition
    joins = ids.shape[1] * -(-I // 64)
    return out, bound + (joins + 3) * ULP * mags


def moe_route(logits, k, bias=None, scoring="softmax", n_group=1, topk_group=1, renormalize=True,
              scaling=1.0):
    """(ids int32 [T, k], weights float64 [T, k])."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        live = z[t] > -np.inf
        if not live.any():
            continue
        if scoring == "softmax":
            e = np.where(live, np.exp(z[t] - z[t][live].max()), 0.0)
            s = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s = np.where(live, 1 / (1 + np.exp(-z[t])), 0.0)
        if bias is None and n_group == 1:
            v = np.where(live, z[t], -np.inf)
        else:
            v = s + (0.0 if bias is None else np.asarray(bias, np.float64))
            v = np.where(live & (v > -np.inf), v, -np.inf)
        if n_group > 1:
            runs = v.reshape(n_group, -1)
            best = -np.sort(-runs, axis=1)[:, :2]
            value = best[:, 0].copy()
            if best.shape[1] > 1:
                value = value + np.where(best[:, 1] > -np.inf, best[:, 1], 0.0)
            keep = np.argsort(-value, kind="stable")[:topk_group]
            mask = np.zeros(n_group, bool)
            mask[keep] = True
            v = np.where(np.repeat(mask, E // n_group), v, -np.inf)
        pick = [e for e in np.argsort(-v, kind="stable")[:k] if v[e] > -np.inf]
        ids[t, :len(pick)] = pick
        ws = s[pick]
        if renormalize:
            ws = ws / ws.sum() if ws.sum() > 0 else 0 * ws
        w[t, :len(pick)] = ws * scaling
    return ids, w


def expert_order(ids, E: int):
    """Pairs (flat indices) by expert, stable, those without one last; counts."""
    flat = np.where(ids.reshape(-1) < 0, E, ids.reshape(-1))
    return np.argsort(flat, kind="stable"), np.bincount(flat, minlength=E + 1)[:E]


def dispatched_rows(x, ids, E: int, kind: int):
    """(codes [T k, H], scale bytes [T k, ceil(H/64), 2], order, counts)."""
    order, counts = expert_order(ids, E)
    codes, scales, _ = mx_quantize(np.asarray(x, np.float64), kind)
    tok = order // ids.shape[1]
    live = (ids.reshape(-1)[order] >= 0)
    return (codes[tok] * live[:, None], scales[tok] * live[:, None, None], order, counts)
