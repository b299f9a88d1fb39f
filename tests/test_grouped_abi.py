"""Host checks of gfr_grouped_linear and gfr_grouped_linear_wgrad on the CPU: every
call here fails validation or is a no-op, so nothing is launched and no pointer is
dereferenced."""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from mxfp8_grouped_gemm_group_amd import _layer
from tests.test_layer_abi import (BAD_ALIGN, BAD_ARG, BAD_DTYPE, BAD_RANK, BAD_SHAPE, BF16, E4,
                                  F16, F32, FAKE, I32, I64, NULL_ARG, UNSUPPORTED, desc, ref)


def grouped(M=0, K=64, N=32, E=4, **over):
    a = dict(x=desc(BF16, M, K), w=desc(BF16, E, K, N), gl=desc(I64, E), kind=1, transpose=0,
             fill=0, out=desc(BF16, M, N))
    a.update(over)
    return _layer._lib().gfr_grouped_linear(ref(a["x"]), ref(a["w"]), ref(a["gl"]), a["kind"],
                                            a["transpose"], a["fill"], ref(a["out"]), None, None)


def wgrad(M=5, K=0, N=32, E=4, **over):
    a = dict(x=desc(BF16, M, K), dy=desc(BF16, M, N), gl=desc(I64, E), kind=1, transpose=0,
             accumulate=0, out=desc(BF16, E, K, N))
    a.update(over)
    return _layer._lib().gfr_grouped_linear_wgrad(ref(a["x"]), ref(a["dy"]), ref(a["gl"]),
                                                  a["kind"], a["transpose"], a["accumulate"],
                                                  ref(a["out"]), None, None)


def test_empty_is_a_no_op():
    assert grouped() == 0
    assert grouped(w=desc(BF16, 4, 32, 64), transpose=1, kind=0, fill=1, out=desc(F32, 0, 32)) == 0
    assert grouped(M=5, N=0) == 0
    assert wgrad() == 0
    assert wgrad(K=64, N=0, out=desc(F32, 4, 0, 64), transpose=1) == 0
    assert wgrad(M=0, K=64, accumulate=1) == 0


@pytest.mark.parametrize("over, code", [
    (dict(x=None), NULL_ARG), (dict(w=None), NULL_ARG), (dict(gl=None), NULL_ARG),
    (dict(out=None), NULL_ARG),
    (dict(M=4, x=desc(BF16, 4, 64, data=None)), NULL_ARG),
    (dict(gl=desc(I64, 4, data=None)), NULL_ARG),
    (dict(x=desc(F32, 0, 64)), BAD_DTYPE), (dict(w=desc(F16, 4, 64, 32)), BAD_DTYPE),
    (dict(w=desc(E4, 4, 64, 32)), BAD_DTYPE), (dict(gl=desc(I32, 4)), BAD_DTYPE),
    (dict(out=desc(F16, 0, 32)), BAD_DTYPE),
    (dict(x=desc(BF16, 0, 64, 1)), BAD_RANK), (dict(w=desc(BF16, 64, 32)), BAD_RANK),
    (dict(gl=desc(I64, 4, 1)), BAD_RANK), (dict(out=desc(BF16, 0)), BAD_RANK),
    (dict(transpose=1), BAD_SHAPE), (dict(w=desc(BF16, 4, 128, 32)), BAD_SHAPE),
    (dict(gl=desc(I64, 3)), BAD_SHAPE), (dict(out=desc(BF16, 0, 31)), BAD_SHAPE),
    (dict(out=desc(BF16, 1, 32)), BAD_SHAPE), (dict(K=0), BAD_SHAPE),
    (dict(kind=2), BAD_ARG), (dict(kind=-1), BAD_ARG), (dict(fill=2), BAD_ARG),
    (dict(E=0), UNSUPPORTED), (dict(E=1025), UNSUPPORTED),
    (dict(M=(1 << 30) + 1), UNSUPPORTED), (dict(K=(1 << 21) + 8), UNSUPPORTED),
    (dict(N=(1 << 21) + 8), UNSUPPORTED),
    (dict(x=desc(BF16, 0, 64, data=FAKE + 8)), BAD_ALIGN),
    (dict(w=desc(BF16, 4, 64, 32, data=FAKE + 2)), BAD_ALIGN),
    (dict(out=desc(BF16, 0, 32, data=FAKE + 8)), BAD_ALIGN),
    (dict(gl=desc(I64, 4, data=FAKE + 4)), BAD_ALIGN),
])
def test_grouped_refusals(over, code):
    assert grouped(**over) == code


def test_transpose_has_to_be_a_flag():
    assert grouped(transpose=2, w=desc(BF16, 4, 32, 64)) == BAD_ARG
    assert wgrad(transpose=-1, K=32) == BAD_ARG


@pytest.mark.parametrize("over, code", [
    (dict(x=None), NULL_ARG), (dict(dy=None), NULL_ARG), (dict(gl=None), NULL_ARG),
    (dict(out=None), NULL_ARG), (dict(K=64, out=desc(BF16, 4, 64, 32, data=None)), NULL_ARG),
    (dict(x=desc(F32, 5, 0)), BAD_DTYPE), (dict(dy=desc(F16, 5, 32)), BAD_DTYPE),
    (dict(out=desc(F16, 4, 0, 32)), BAD_DTYPE), (dict(gl=desc(I32, 4)), BAD_DTYPE),
    (dict(dy=desc(BF16, 5, 32, 1)), BAD_RANK), (dict(out=desc(BF16, 0, 32)), BAD_RANK),
    (dict(dy=desc(BF16, 4, 32)), BAD_SHAPE), (dict(out=desc(BF16, 4, 32, 0)), BAD_SHAPE),
    (dict(transpose=1), BAD_SHAPE), (dict(gl=desc(I64, 5)), BAD_SHAPE),
    (dict(kind=3), BAD_ARG), (dict(accumulate=2), BAD_ARG),
    (dict(E=0), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(M=(1 << 30) + 1), UNSUPPORTED),
    (dict(K=(1 << 21) + 8), UNSUPPORTED), (dict(N=(1 << 21) + 8), UNSUPPORTED),
    (dict(dy=desc(BF16, 5, 32, data=FAKE + 8)), BAD_ALIGN),
    (dict(out=desc(F32, 4, 0, 32, data=FAKE + 8)), BAD_ALIGN),
])
def test_wgrad_refusals(over, code):
    assert wgrad(**over) == code


@pytest.mark.gpu
def test_python_refusals():
    dev = "cuda:0"
    x = torch.zeros(6, 64, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(2, 64, 32, dtype=torch.bfloat16, device=dev)
    dy = torch.zeros(6, 32, dtype=torch.bfloat16, device=dev)
    gl = torch.tensor([2, 4], device=dev)
    for bad in [lambda: gfr.grouped_linear(x.cpu(), w, gl, 1),
                lambda: gfr.grouped_linear(x, w.cpu(), gl, 1),
                lambda: gfr.grouped_linear(x, w, gl.cpu(), 1),
                lambda: gfr.grouped_linear(x, w.transpose(1, 2), gl, 1, transpose_w=True),
                lambda: gfr.grouped_linear(x[0], w, gl, 1),
                lambda: gfr.grouped_linear(x, w[0], gl, 1),
                lambda: gfr.grouped_linear(x, w, gl, 1, out=dy, out_dtype=torch.float32),
                lambda: gfr.grouped_linear(x, w, gl, 1, status=torch.zeros(1, device=dev)),
                lambda: gfr.grouped_linear_wgrad(x, dy[0], gl, 1),
                lambda: gfr.grouped_linear_wgrad(x, dy, gl, 1, accumulate=True)]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: gfr.grouped_linear(x, w.half(), gl, 1),
                lambda: gfr.grouped_linear(x.float(), w.float(), gl, 1),
                lambda: gfr.grouped_linear(x, w, gl.int(), 1),
                lambda: gfr.grouped_linear(x, w, gl, 2),
                lambda: gfr.grouped_linear(x, w, gl, 1, transpose_w=True),
                lambda: gfr.grouped_linear_wgrad(x, dy[:5], gl, 1)]:
        with pytest.raises(gfr.GfrError):
            bad()
