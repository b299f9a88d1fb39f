"""grouped_linear under autograd, as torch's other functions hand it gradients and as its
results are asked for derivatives."""
import pytest
import torch
from torch.autograd import forward_ad

import mxfp8_grouped_gemm_group_amd as gfr
from tests import grouped_inputs as gi
from tests.test_grouped_linear_grad_gpu import COUNTS, DEV, setup

pytestmark = pytest.mark.gpu


def gradients_are(xd, wd, x, w, dy, rng, transpose):
    torch.cuda.synchronize()
    assert torch.equal(xd.grad.cpu(), gi.forward(dy, w, rng, not transpose).to(x.dtype))
    assert torch.equal(wd.grad.cpu(), gi.wgrad(x, dy, rng, transpose).to(x.dtype))


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("K, N, ahead", [(67, 33, 3), (72, 136, 1), (264, 40, 0)])
def test_gradients_that_begin_anywhere(K, N, ahead, transpose):
    """Behind other rows (cat along rows) and behind other elements (a flat cat)."""
    x, w, dy, xd, wd, dyd, gl, rng = setup(K, N, transpose)
    y = gfr.grouped_linear(xd, wd, gl, 1, transpose_w=transpose)
    z = torch.zeros(ahead, N, dtype=y.dtype, device=DEV)
    torch.cat([z, y]).backward(torch.cat([z, dyd]))
    gradients_are(xd, wd, x, w, dy, rng, transpose)
    xd.grad = wd.grad = None
    y = gfr.grouped_linear(xd, wd, gl, 1, transpose_w=transpose)
    five = torch.zeros(5, dtype=y.dtype, device=DEV)
    torch.cat([five, y.flatten()]).backward(torch.cat([five, dyd.flatten()]))
    gradients_are(xd, wd, x, w, dy, rng, transpose)


def test_a_captured_gradient_that_begins_anywhere():
    x, w, dy, xd, wd, dyd, gl, rng = setup(67, 33, False)
    five = torch.zeros(5, dtype=dyd.dtype, device=DEV)

    def step():
        y = torch.cat([five, gfr.grouped_linear(xd, wd, gl, 1).flatten()])
        return torch.autograd.grad(y, (xd, wd), torch.cat([five, dyd.flatten()]))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, dw = step()
    torch.cuda.synchronize()
    for i in range(4):
        x, w, dy = gi.integers(COUNTS, x.shape[0], 67, 33, torch.bfloat16, seed=i)
        with torch.no_grad():
            xd.copy_(x), wd.copy_(w), dyd.copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx.cpu(), gi.forward(dy, w, rng, True).bfloat16())
        assert torch.equal(dw.cpu(), gi.wgrad(x, dy, rng, False).bfloat16())
        torch.randn(256, 256, device=DEV).relu_()


def test_forward_mode_is_refused():
    """A tangent is not dropped; without one the call is as ever."""
    *_, xd, wd, dyd, gl, _ = setup(72, 136, False, requires=False)
    plain = gfr.grouped_linear(xd, wd, gl, 1)
    with forward_ad.dual_level():
        for args in [(forward_ad.make_dual(xd, torch.ones_like(xd)), wd),
                     (xd, forward_ad.make_dual(wd, torch.ones_like(wd)))]:
            with pytest.raises(NotImplementedError):
                gfr.grouped_linear(*args, gl, 1)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                gfr.grouped_linear(*args, gl, 1)
            with pytest.raises(ValueError):
                gfr.grouped_linear(*args, gl, 1, out=torch.empty_like(plain))
        assert torch.equal(gfr.grouped_linear(xd, wd, gl, 1), plain)
    with pytest.raises(Exception):
        torch.func.jvp(lambda a: gfr.grouped_linear(a, wd, gl, 1), (xd,), (torch.ones_like(xd),))


@pytest.mark.parametrize("transpose", [False, True])
def test_only_what_a_gradient_takes_is_kept(transpose):
    """With frozen weights x may change, and is freed, before the backward pass; with
    frozen rows the weights may."""
    x, w, dy, xd, wd, dyd, gl, rng = setup(72, 136, transpose, requires=False)
    xd.requires_grad_(True)
    rows = xd * 1
    before = torch.cuda.memory_allocated()
    y = gfr.grouped_linear(rows, wd, gl, 1, transpose_w=transpose)
    rows.zero_()
    del rows
    assert torch.cuda.memory_allocated() < before + y.numel() * y.element_size()
    y.backward(dyd)
    assert torch.equal(xd.grad.cpu(), gi.forward(dy, w, rng, not transpose).bfloat16())
    xd, wd = xd.detach(), wd.requires_grad_(True)
    copy = wd * 1
    y = gfr.grouped_linear(xd, copy, gl, 1, transpose_w=transpose)
    copy.zero_()
    y.backward(dyd)
    assert torch.equal(wd.grad.cpu(), gi.wgrad(x, dy, rng, transpose).bfloat16())
    # what it takes is guarded
    wd = wd.detach()
    y = gfr.grouped_linear(xd.requires_grad_(True), wd, gl, 1, transpose_w=transpose)
    wd.zero_()
    with pytest.raises(RuntimeError):
        y.backward(dyd)
