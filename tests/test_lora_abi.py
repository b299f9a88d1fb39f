"""Host checks of gfr_lora_linear on the CPU: every call here fails validation or is a
no-op, so nothing is launched and no pointer is dereferenced."""
import ctypes

import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from mxfp8_grouped_gemm_group_amd import _layer
from tests.test_layer_abi import (BAD_ALIGN, BAD_DTYPE, BAD_RANK, BAD_SHAPE, BF16, F16, F32, FAKE,
                                  I32, I64, NULL_ARG, UNSUPPORTED, WS_SMALL, desc, opts, ref)


def lora(M=0, N=32, K=64, L=4, r=8, **over):
    a = dict(x=desc(BF16, M, K), w=desc(BF16, N, K), bias=None, residual=None,
             la=desc(BF16, L, r, K), lb=desc(BF16, L, N, r), ids=desc(I32, M), scaling=None,
             out=desc(BF16, M, N), opts=opts())
    a.update(over)
    return _layer._lib().gfr_lora_linear(
        ref(a["x"]), ref(a["w"]), ref(a["bias"]), ref(a["residual"]), ref(a["la"]), ref(a["lb"]),
        ref(a["ids"]), ref(a["scaling"]), ref(a["out"]), None, a["opts"])


def test_empty_is_a_no_op():
    assert lora() == 0
    assert lora(opts=None) == 0
    assert lora(M=5, N=0) == 0
    assert lora(out=desc(F32, 0, 32), bias=desc(F32, 32), scaling=desc(F32, 4)) == 0


@pytest.mark.parametrize("over, code", [
    (dict(x=None), NULL_ARG), (dict(la=None), NULL_ARG), (dict(lb=None), NULL_ARG),
    (dict(ids=None), NULL_ARG), (dict(out=None), NULL_ARG),
    (dict(M=4, ids=desc(I32, 4, data=None)), NULL_ARG),
    (dict(x=desc(F32, 0, 64)), BAD_DTYPE), (dict(la=desc(F16, 4, 8, 64)), BAD_DTYPE),
    (dict(lb=desc(F32, 4, 32, 8)), BAD_DTYPE), (dict(ids=desc(I64, 0)), BAD_DTYPE),
    (dict(scaling=desc(BF16, 4)), BAD_DTYPE), (dict(residual=desc(F32, 0, 32)), BAD_DTYPE),
    (dict(la=desc(BF16, 8, 64)), BAD_RANK), (dict(lb=desc(BF16, 4, 32)), BAD_RANK),
    (dict(ids=desc(I32, 0, 1)), BAD_RANK), (dict(scaling=desc(F32, 4, 1)), BAD_RANK),
    (dict(la=desc(BF16, 4, 8, 32)), BAD_SHAPE), (dict(lb=desc(BF16, 4, 8, 32)), BAD_SHAPE),
    (dict(lb=desc(BF16, 3, 32, 8)), BAD_SHAPE), (dict(ids=desc(I32, 1)), BAD_SHAPE),
    (dict(scaling=desc(F32, 3)), BAD_SHAPE), (dict(bias=desc(BF16, 31)), BAD_SHAPE),
    (dict(out=desc(BF16, 0, 31)), BAD_SHAPE),
    (dict(r=0), UNSUPPORTED), (dict(r=257), UNSUPPORTED), (dict(L=0), UNSUPPORTED),
    (dict(L=(1 << 20) + 1), UNSUPPORTED), (dict(M=(1 << 26) + 1), UNSUPPORTED),
    (dict(K=(1 << 21) + 8), UNSUPPORTED),
    (dict(la=desc(BF16, 4, 8, 64, data=FAKE + 8)), BAD_ALIGN),
    (dict(lb=desc(BF16, 4, 32, 8, data=FAKE + 2)), BAD_ALIGN),
    (dict(M=4, ids=desc(I32, 4, data=FAKE + 2)), BAD_ALIGN),
    (dict(scaling=desc(F32, 4, data=FAKE + 2)), BAD_ALIGN),
    (dict(M=4, opts=None), WS_SMALL), (dict(M=4, opts=opts(n=4)), WS_SMALL),
    (dict(M=4, opts=opts(ws=FAKE + 64)), BAD_ALIGN),
])
def test_refusals(over, code):
    assert lora(**over) == code


def test_workspace_size():
    size = lambda *a: gfr.lora_linear_workspace_size(*a)
    assert size(0, 32, 64, 8) == 0 and size(4, 0, 64, 8) == 0
    assert size(4, 32, 64, 8) >= 4 * 4 * 8
    for bad in [(4, 32, 0, 8), (4, 32, 64, 0), (4, 32, 64, 257), (-1, 32, 64, 8)]:
        with pytest.raises(gfr.GfrError):
            size(*bad)
    assert _layer._lib().gfr_lora_linear_workspace_size(4, 32, 64, 8, None) == NULL_ARG
    n = ctypes.c_size_t(0)
    assert _layer._lib().gfr_lora_linear_workspace_size(4, 32, 64, 8, ctypes.byref(n)) == 0


@pytest.mark.gpu
def test_python_refusals():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda:0")
    x, w, a, b = z(6, 64), z(32, 64), z(2, 8, 64), z(2, 32, 8)
    ids = torch.zeros(6, dtype=torch.int32, device="cuda:0")
    for bad in [lambda: gfr.lora_linear(x.cpu(), w, a, b, ids),
                lambda: gfr.lora_linear(x, w, a.cpu(), b, ids),
                lambda: gfr.lora_linear(x, w, a, b, ids.cpu()),
                lambda: gfr.lora_linear(x, w, a.transpose(1, 2), b, ids),
                lambda: gfr.lora_linear(x, w, a[0], b, ids),
                lambda: gfr.lora_linear(x, w, a, b, ids, out=z(6, 32), out_dtype=torch.float32)]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: gfr.lora_linear(x, w, a, b, ids.long()),
                lambda: gfr.lora_linear(x, w, a.half(), b, ids),
                lambda: gfr.lora_linear(x, w, a, b[:1], ids),
                lambda: gfr.lora_linear(x, w, a, b, ids[:5])]:
        with pytest.raises(gfr.GfrError):
            bad()
