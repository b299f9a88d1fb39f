"""lora_linear has no gradients, and says so where one is asked for."""
import pytest
import torch
from torch.autograd import forward_ad

import mxfp8_grouped_gemm_group_amd as gfr
from tests.test_lora_linear_gpu import BF, DEV, integers

pytestmark = pytest.mark.gpu


def operands():
    a = integers(9, 40, 64, 3, 16, BF, bias=BF, residual=True)
    return {k: v.to(DEV) for k, v in a.items()}


def call(d, **over):
    return gfr.lora_linear(d["x"], d["w"], d["a"], d["b"], d["ids"], scaling=d["scaling"],
                           bias=d["bias"], residual=d["residual"], **over)


@pytest.mark.parametrize("wanted", ["x", "w", "a", "b", "scaling", "bias", "residual"])
def test_a_gradient_is_refused_not_lost(wanted):
    d = operands()
    plain = call(d)
    leaf = d[wanted].requires_grad_(True)
    y = call(d)
    assert torch.equal(y.detach(), plain) and y.requires_grad
    with pytest.raises(RuntimeError, match="no gradients"):
        y.sum().backward()
    assert leaf.grad is None
    with pytest.raises(ValueError):
        call(d, out=torch.empty_like(plain))
    with torch.no_grad():
        out = torch.empty_like(plain)
        assert call(d, out=out) is out and torch.equal(out, plain)
        assert not call(d).requires_grad
    d[wanted] = leaf.detach()
    assert not call(d).requires_grad


def test_forward_mode_is_refused():
    d = operands()
    with forward_ad.dual_level():
        d["x"] = forward_ad.make_dual(d["x"], torch.ones_like(d["x"]))
        with pytest.raises(NotImplementedError):
            call(d)


def test_on_another_stream():
    d = operands()
    plain = call(d)
    d["a"].requires_grad_(True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = call(d, stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y.detach(), plain) and y.requires_grad
