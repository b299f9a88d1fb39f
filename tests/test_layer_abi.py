"""Host checks of gfr_linear, gfr_moe_decode and gfr_moe_route on the CPU: every
call here fails validation or is a no-op, so nothing is launched and no
pointer is dereferenced."""
import ctypes

import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from mxfp8_grouped_gemm_group_amd import _layer
from mxfp8_grouped_gemm_group_amd._binding import GfrOptions, GfrTensor

FAKE = 0x10000
E4, E5, E8M0, U8, BF16, F32, I64, I32, F16 = 0, 1, 3, 4, 5, 6, 7, 8, 11
NULL_ARG, BAD_SHAPE, UNSUPPORTED, BAD_ALIGN, WS_SMALL, BAD_ARG, BAD_DTYPE, BAD_RANK = \
    1, 2, 4, 5, 6, 7, 9, 10


def desc(dtype, *shape, data=FAKE):
    d = GfrTensor()
    d.data, d.dtype, d.ndim = data, dtype, len(shape)
    for i, n in enumerate(shape):
        d.shape[i] = n
    return d


def ref(d):
    return None if d is None else ctypes.byref(d)


def opts(ws=FAKE, n=1 << 40):
    return ctypes.byref(GfrOptions(0, ws, n, None, 0, 0))


# ---- linear -----------------------------------------------------------------


def linear(**over):
    a = dict(x=desc(BF16, 0, 64), w=desc(BF16, 32, 64), bias=None, residual=None, act=0,
             out=desc(BF16, 0, 32), opts=None)
    a.update(over)
    return _layer._lib().gfr_linear(ref(a["x"]), ref(a["w"]), ref(a["bias"]), ref(a["residual"]),
                                    a["act"], ref(a["out"]), None, a["opts"])


def test_linear_empty_is_a_no_op():
    assert linear() == 0
    assert linear(x=desc(BF16, 5, 64), w=desc(BF16, 0, 64, data=None),
                  out=desc(BF16, 5, 0, data=None)) == 0


@pytest.mark.parametrize("over, code", [
    (dict(x=None), NULL_ARG),
    (dict(x=desc(BF16, 4, 64, data=None), out=desc(BF16, 4, 32)), NULL_ARG),
    (dict(x=desc(F32, 0, 64)), BAD_DTYPE),
    (dict(w=desc(F16, 32, 64)), BAD_DTYPE),
    (dict(out=desc(F16, 0, 32)), BAD_DTYPE),
    (dict(x=desc(BF16, 0, 1, 64)), BAD_RANK),
    (dict(w=desc(BF16, 32, 128)), BAD_SHAPE),
    (dict(x=desc(BF16, 0, 0), w=desc(BF16, 32, 0)), BAD_SHAPE),
    (dict(out=desc(BF16, 0, 31)), BAD_SHAPE),
    (dict(act=5, w=desc(BF16, 33, 64)), BAD_SHAPE),
    (dict(act=5), BAD_SHAPE),                               # out must be half as wide
    (dict(act=6), BAD_ARG), (dict(act=-1), BAD_ARG),
    (dict(bias=desc(BF16, 31)), BAD_SHAPE),
    (dict(bias=desc(F16, 32)), BAD_DTYPE),
    (dict(residual=desc(F32, 0, 32)), BAD_DTYPE),
    (dict(residual=desc(BF16, 0, 16)), BAD_SHAPE),
    (dict(x=desc(BF16, 0, (1 << 21) + 8), w=desc(BF16, 32, (1 << 21) + 8)), UNSUPPORTED),
    (dict(x=desc(BF16, 1 << 31, 64), out=desc(BF16, 1 << 31, 32)), UNSUPPORTED),
    # more tiles than a grid has room for; more rows than a tile's columns count
    (dict(x=desc(BF16, 1 << 30, 64), w=desc(BF16, 2048, 64), out=desc(BF16, 1 << 30, 2048)),
     UNSUPPORTED),
    (dict(x=desc(BF16, 4, 8), w=desc(BF16, (1 << 30) + 1, 8),
          out=desc(BF16, 4, (1 << 30) + 1)), UNSUPPORTED),
    (dict(x=desc(BF16, 4, 64, data=FAKE + 8), out=desc(BF16, 4, 32)), BAD_ALIGN),
    (dict(x=desc(BF16, 4, 64), out=desc(BF16, 4, 32, data=FAKE + 4)), BAD_ALIGN),
])
def test_linear_refusals(over, code):
    assert linear(**over) == code


# ---- moe_decode -------------------------------------------------------------


def decode(T=0, H=128, I=64, N=192, E=4, k=2, **over):
    a = dict(x=desc(BF16, T, H), w13=desc(E4, E, H, 2 * I), s13=desc(E8M0, H // 64, 2 * I, 2),
             w2=desc(E4, E, I, N), s2=desc(U8, I // 64, N, 2), ids=desc(I32, T, k),
             wts=desc(F32, T, k), shared=None, out=desc(BF16, T, N), t13=0, t2=0, opts=opts())
    a.update(over)
    return _layer._lib().gfr_moe_decode(
        ref(a["x"]), ref(a["w13"]), ref(a["s13"]), ref(a["w2"]), ref(a["s2"]), ref(a["ids"]),
        ref(a["wts"]), ref(a["shared"]), 1.0, ref(a["out"]), a["t13"], a["t2"], None, a["opts"])


def test_decode_empty_is_a_no_op():
    assert decode() == 0
    assert decode(opts=None) == 0
    # both layouts, per-expert scales
    assert decode(w13=desc(E4, 4, 128, 128), s13=desc(E8M0, 4, 128, 2, 2), t13=1) == 0
    assert decode(w2=desc(E4, 4, 192, 64), s2=desc(U8, 192, 1, 2), t2=1) == 0


@pytest.mark.parametrize("over, code", [
    (dict(w2=None), NULL_ARG),
    (dict(x=desc(F32, 0, 128)), BAD_DTYPE),
    (dict(w2=desc(E5, 4, 64, 192)), BAD_DTYPE),
    (dict(ids=desc(I64, 0, 2)), BAD_DTYPE),
    (dict(out=desc(F16, 0, 192)), BAD_DTYPE),
    (dict(s13=desc(E8M0, 2, 128)), BAD_RANK),
    (dict(s13=desc(E8M0, 128, 2, 2)), BAD_SHAPE),           # the transposed layout's
    (dict(s2=desc(U8, 3, 1, 192, 2)), BAD_SHAPE),           # three experts
    (dict(w2=desc(E4, 3, 64, 192)), BAD_SHAPE),
    (dict(w2=desc(E4, 4, 128, 192)), BAD_SHAPE),            # I from w13 is 64
    (dict(wts=desc(F32, 0, 3)), BAD_SHAPE),
    (dict(out=desc(BF16, 0, 64)), BAD_SHAPE),
    (dict(shared=desc(BF16, 1, 192)), BAD_SHAPE),
    (dict(w13=desc(E4, 4, 128, 127)), BAD_SHAPE),
    (dict(t13=2), BAD_ARG),
    (dict(T=65), UNSUPPORTED),
    (dict(k=33), UNSUPPORTED),
    (dict(T=64, k=17), UNSUPPORTED),
    (dict(H=96, s13=desc(E8M0, 2, 128, 2)), UNSUPPORTED),
    (dict(I=32, s2=desc(U8, 1, 192, 2)), UNSUPPORTED),
    (dict(N=96), UNSUPPORTED),
    (dict(E=1025), UNSUPPORTED),
    (dict(H=1 << 16, I=1 << 15, w2=desc(E4, 4, 1 << 15, 192), s2=desc(U8, 512, 192, 2)),
     UNSUPPORTED),
    (dict(T=3, opts=None), WS_SMALL),
    (dict(T=3, opts=opts(n=1 << 10)), WS_SMALL),
    (dict(T=3, opts=opts(ws=FAKE + 16)), BAD_ALIGN),
    (dict(T=3, x=desc(BF16, 3, 128, data=FAKE + 2)), BAD_ALIGN),
])
def test_decode_refusals(over, code):
    assert decode(**over) == code


def test_decode_workspace_covers_its_regions():
    for T, k, E, H, I, N, t in ((1, 8, 256, 2048, 512, 2048, False),
                                (64, 3, 32, 4096, 8192, 4096, False),
                                (64, 16, 4, 64, 64, 64, True), (1, 1, 1, 64, 4096, 64, True)):
        need = gfr.moe_decode_workspace_size(T, k, E, H, I, N, t, t)
        assert need >= 4 * T * k * 2 * I + 4 * T * k * N
    with pytest.raises(gfr.GfrError):
        gfr.moe_decode_workspace_size(65, 2, 8, 64, 64, 64)


# ---- moe_route --------------------------------------------------------------


def route(T=0, E=8, k=2, H=64, with_x=True, **over):
    a = dict(logits=desc(F32, T, E), bias=None, scoring=0, n_group=1, topk_group=1, renorm=1,
             ids=desc(I32, T, k), wts=desc(F32, T, k), opts=opts())
    names = ("x", "xin", "xin_scale", "group_list", "row_index", "logit")
    # (T = 0 would still clear group_list: the no-op and refusal cases keep x away
    # or fail before that)
    a.update(x=desc(BF16, T, H), xin=desc(E4, T * k, H),
             xin_scale=desc(U8, T * k, (H + 63) // 64, 2), group_list=desc(I64, E),
             row_index=desc(I32, T * k), logit=desc(F32, T * k)) if with_x else \
        a.update({n: None for n in names})
    a.update(over)
    return _layer._lib().gfr_moe_route(
        ref(a["logits"]), ref(a["bias"]), a["scoring"], a["n_group"], a["topk_group"],
        a["renorm"], 1.0, ref(a["ids"]), ref(a["wts"]), *[ref(a[n]) for n in names], None,
        a["opts"])


def test_route_empty_is_a_no_op():
    assert route(with_x=False) == 0


@pytest.mark.parametrize("over, code", [
    (dict(logits=None), NULL_ARG),
    (dict(xin=None), NULL_ARG),
    (dict(with_x=False, logit=desc(F32, 0)), NULL_ARG),     # outputs without x
    (dict(logits=desc(F16, 0, 8)), BAD_DTYPE),
    (dict(ids=desc(I64, 0, 2)), BAD_DTYPE),
    (dict(x=desc(F32, 0, 64)), BAD_DTYPE),
    (dict(xin=desc(BF16, 0, 64)), BAD_DTYPE),
    (dict(row_index=desc(I64, 0)), BAD_DTYPE),
    (dict(bias=desc(F32, 1, 8)), BAD_RANK),
    (dict(bias=desc(F32, 7)), BAD_SHAPE),
    (dict(k=9), BAD_SHAPE),                                 # more than E
    (dict(wts=desc(F32, 0, 3)), BAD_SHAPE),
    (dict(x=desc(BF16, 1, 64)), BAD_SHAPE),
    (dict(group_list=desc(I64, 7)), BAD_SHAPE),
    (dict(xin_scale=desc(U8, 0, 2, 2)), BAD_SHAPE),
    (dict(H=48), UNSUPPORTED),
    (dict(E=1025), UNSUPPORTED),
    (dict(E=64, k=33), UNSUPPORTED),
    (dict(T=(1 << 26) + 1, k=1, with_x=False), UNSUPPORTED),
    (dict(T=1 << 26, E=64, k=32), UNSUPPORTED),             # 2^31 pairs
    (dict(scoring=2), BAD_ARG), (dict(renorm=2), BAD_ARG),
    (dict(n_group=3), BAD_ARG), (dict(n_group=0), BAD_ARG),
    (dict(n_group=4, topk_group=5), BAD_ARG), (dict(n_group=4, topk_group=0), BAD_ARG),
    (dict(E=128, n_group=128), BAD_ARG),
    (dict(T=100, opts=None), WS_SMALL),
    (dict(T=100, opts=opts(ws=FAKE + 8)), BAD_ALIGN),
    (dict(T=4, x=desc(BF16, 4, 64, data=FAKE + 8)), BAD_ALIGN),
    (dict(T=4, group_list=desc(I64, 8, data=FAKE + 4)), BAD_ALIGN),
    (dict(T=4, with_x=False, logits=desc(F32, 4, 8, data=FAKE + 2)), BAD_ALIGN),
])
def test_route_refusals(over, code):
    assert route(**over) == code


# ---- Python layer -----------------------------------------------------------


def test_python_refusals():
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gfr.linear(x, w)                                    # CPU tensors
    with pytest.raises(ValueError):
        gfr.linear(x, w, activation="tanh")
    with pytest.raises(ValueError):
        gfr.moe_route(torch.zeros(2, 4), 2, scoring="relu")
    with pytest.raises(ValueError):
        gfr.moe_route(torch.zeros(2, 4), 0)
