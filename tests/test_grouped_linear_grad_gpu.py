"""grouped_linear under autograd: against the formula's gradients in 64 bits and
against differences; which tensors get one, captured steps, streams."""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from tests import grouped_inputs as gi

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
COUNTS = [40, 0, 130, 7]


def setup(K, N, transpose, dtype=torch.bfloat16, rest=6, requires=True):
    M = sum(COUNTS) + rest
    x, w, dy = gi.integers(COUNTS, M, K, N, dtype, transpose)
    gl = torch.tensor(COUNTS, dtype=torch.int64, device=DEV)
    xd, wd = x.to(DEV).requires_grad_(requires), w.to(DEV).requires_grad_(requires)
    return x, w, dy, xd, wd, dy.to(DEV), gl, gi.ranges(COUNTS, 1, M)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("K, N", [(72, 136), (67, 33)])
def test_gradients_equal_the_formulas(dtype, transpose, K, N):
    x, w, dy, xd, wd, dyd, gl, rng = setup(K, N, transpose, dtype)
    y = gfr.grouped_linear(xd, wd, gl, 1, transpose_w=transpose)
    y.backward(dyd)
    torch.cuda.synchronize()
    dx = gi.forward(dy, w, rng, not transpose)
    assert torch.equal(y.detach().cpu(), gi.forward(x, w, rng, transpose).to(dtype))
    assert torch.equal(xd.grad.cpu(), dx.to(dtype))
    assert torch.equal(wd.grad.cpu(), gi.wgrad(x, dy, rng, transpose).to(dtype))


@pytest.mark.parametrize("transpose", [False, True])
def test_gradient_against_differences(transpose):
    """The loss sum(c * y), linear in x and in w: the difference over a whole step is
    the gradient's product with the step, on integers exactly."""
    x, w, c, xd, wd, cd, gl, _ = setup(72, 40, transpose)

    def loss(a, b):
        y = gfr.grouped_linear(a, b, gl, 1, transpose_w=transpose, out_dtype=torch.float32)
        return (y.double() * cd.double()).sum()

    base = loss(xd, wd)
    base.backward()
    g = torch.Generator().manual_seed(3)
    for t, other in ((xd, wd), (wd, xd)):
        step = torch.randint(-1, 2, t.shape, generator=g).to(DEV)
        with torch.no_grad():
            moved = (t.double() + step).to(t.dtype)
            high = loss(moved, wd) if t is xd else loss(xd, moved)
        # (the gradient's own rounding to 16 bits: half a step, 2^-8, of each element)
        want = (t.grad.double() * step).sum()
        slack = 2.0 ** -8 * t.grad.double().abs().sum()
        assert abs((high - base) - want) <= slack


def test_only_wanted_gradients():
    *_, xd, wd, dyd, gl, _ = setup(72, 136, False, requires=False)
    assert not gfr.grouped_linear(xd, wd, gl, 1).requires_grad
    xd.requires_grad_(True)
    gfr.grouped_linear(xd, wd, gl, 1).backward(dyd)
    assert xd.grad is not None and wd.grad is None
    xd.requires_grad_(False)
    wd.requires_grad_(True)
    xd.grad = None
    gfr.grouped_linear(xd, wd, gl, 1).backward(dyd)
    assert xd.grad is None and wd.grad is not None
    with torch.no_grad():
        assert not gfr.grouped_linear(xd, wd, gl, 1).requires_grad
    with pytest.raises(ValueError):
        gfr.grouped_linear(xd, wd, gl, 1, out=torch.empty_like(dyd))


def test_broadcast_and_strided_gradients():
    x, w, dy, xd, wd, dyd, gl, rng = setup(72, 136, False)
    y = gfr.grouped_linear(xd, wd, gl, 1)
    y.sum().backward()                      # one element, expanded
    ones = torch.ones_like(dy)
    assert torch.equal(xd.grad.cpu(), gi.forward(ones, w, rng, True).bfloat16())
    xd.grad = wd.grad = None
    gfr.grouped_linear(xd, wd, gl, 1).t().backward(dyd.t())
    assert torch.equal(wd.grad.cpu(), gi.wgrad(x, dy, rng, False).bfloat16())


def test_float32_result_and_second_use():
    x, w, dy, xd, wd, dyd, gl, rng = setup(72, 136, True)
    y = gfr.grouped_linear(xd, wd, gl, 1, transpose_w=True, out_dtype=torch.float32)
    y.backward(dyd.float())
    assert torch.equal(xd.grad.cpu(), gi.forward(dy, w, rng, False).bfloat16())
    with pytest.raises(RuntimeError):
        y.backward(dyd.float())             # saved tensors are gone
    xd.grad = None
    y = gfr.grouped_linear(xd, wd, gl, 1, transpose_w=True)
    (g,) = torch.autograd.grad(y, xd, dyd, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()                  # differentiable once


def test_side_stream():
    x, w, dy, xd, wd, dyd, gl, rng = setup(264, 520, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = gfr.grouped_linear(xd, wd, gl, 1, stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    dx, dw = torch.autograd.grad(y, (xd, wd), dyd)
    torch.cuda.synchronize()
    assert torch.equal(y.detach().cpu(), gi.forward(x, w, rng, False).bfloat16())
    assert torch.equal(dx.cpu(), gi.forward(dy, w, rng, True).bfloat16())
    assert torch.equal(dw.cpu(), gi.wgrad(x, dy, rng, False).bfloat16())


@pytest.mark.parametrize("K, N", [(264, 520), (67, 33)])
def test_training_step_under_graph(K, N):
    """A captured step replays on new rows, groups and gradients."""
    x, w, dy, xd, wd, dyd, gl, _ = setup(K, N, False)
    M = x.shape[0]

    def step():
        y = gfr.grouped_linear(xd, wd, gl, 1)
        return (y, *torch.autograd.grad(y, (xd, wd), dyd))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx, dw = step()
    torch.cuda.synchronize()
    for i, counts in enumerate([COUNTS, [0, 90, 3, 80], [177, 0, 0, 0], [1, 1, 1, 1], COUNTS]):
        x, w, dy = gi.integers(COUNTS, M, K, N, torch.bfloat16, seed=i)
        rng = gi.ranges(counts, 1, M)
        with torch.no_grad():
            xd.copy_(x), wd.copy_(w), dyd.copy_(dy)
            gl.copy_(torch.tensor(counts))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.detach().cpu(), gi.forward(x, w, rng, False).bfloat16())
        assert torch.equal(dx.cpu(), gi.forward(dy, w, rng, True).bfloat16())
        assert torch.equal(dw.cpu(), gi.wgrad(x, dy, rng, False).bfloat16())
        torch.randn(256, 256, device=DEV).relu_()


@pytest.mark.gpu
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("M, N", [(0, 24), (5, 0), (0, 0)])
def test_gradients_without_rows_or_columns(M, N, transpose):
    x = torch.ones(M, 16, dtype=torch.bfloat16, device="cuda:0", requires_grad=True)
    w = torch.ones(2, *((N, 16) if transpose else (16, N)), dtype=torch.bfloat16, device="cuda:0",
                   requires_grad=True)
    counts = torch.tensor([M, 0], device="cuda:0")
    y = gfr.grouped_linear(x, w, counts, 1, transpose_w=transpose)
    assert y.shape == (M, N)
    y.backward(torch.ones_like(y))
    assert x.grad.shape == x.shape and not x.grad.any()
    assert w.grad.shape == w.shape and not w.grad.any()
