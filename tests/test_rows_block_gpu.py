"""The products chosen by the row as a MoE block uses them: 16-bit experts behind the
router, forward and backward, adapters on the shared expert, LoRA training over rows
sorted by adapter; under a graph and on two streams at once.

The block: router logits (linear) -> moe_route(x) -> the rows in its order ->
grouped_linear (gate and up) -> silu(gate) * up -> grouped_linear (down) -> the
weighted sum over each token's experts, plus the shared expert's lora_linear pair.
"""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E, K, H, I, SI, L, R = 16, 4, 256, 192, 320, 5, 16
BF = torch.bfloat16


def weights(seed=0, device=DEV):
    g = torch.Generator().manual_seed(seed)
    w = lambda *s, k: (torch.randn(*s, generator=g) / k ** 0.5).to(BF).to(device)
    return dict(router=w(E, H, k=H), w13=w(E, 2 * I, H, k=H), w2=w(E, I, H, k=I),
                up=w(2 * SI, H, k=H), down=w(H, SI, k=SI),
                up_a=w(L, R, H, k=H), up_b=w(L, 2 * SI, R, k=4 * R),
                down_a=w(L, R, SI, k=SI), down_b=w(L, H, R, k=4 * R))


def tokens(T, seed=1):
    return torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).to(BF).to(DEV)


def route(b, x):
    logits = gfr.linear(x, b["router"], out_dtype=torch.float32)
    return gfr.moe_route(logits, K, x=x)


def experts(x, w13, w2, r):
    """[T, H] float32: the weighted sum over each token's experts."""
    rows = x[r.row_index.long()]
    gu = gfr.grouped_linear(rows, w13, r.group_list, 1, transpose_w=True)
    h = torch.nn.functional.silu(gu[:, :I].float()) * gu[:, I:].float()
    y = gfr.grouped_linear(h.to(BF), w2, r.group_list, 1)
    return torch.zeros(x.shape, device=x.device).index_add(
        0, r.row_index.long(), y.float() * r.logit[:, None])


def shared(b, x, ids):
    gu = gfr.lora_linear(x, b["up"], b["up_a"], b["up_b"], ids)
    h = (torch.nn.functional.silu(gu[:, :SI].float()) * gu[:, SI:].float()).to(BF)
    return gfr.lora_linear(h, b["down"], b["down_a"], b["down_b"], ids)


def experts64(x, w13, w2, r):
    out = torch.zeros(x.shape, dtype=torch.float64)
    rows, logit = r.row_index.long().cpu(), r.logit.double().cpu()
    at = 0
    for e, n in enumerate(r.group_list.tolist()):
        t = rows[at:at + n]
        gu = x[t] @ w13[e].T
        y = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ w2[e]
        out = out.index_add(0, t, y * logit[at:at + n, None])
        at += n
    return out


def off(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("T", [1, 24, 300])
def test_experts_forward_and_backward(T):
    """Relative to the norms.  A rounding to bf16 is 2^-8 at most.  Forward: gate, up (both
    in one product's result), h, y.  Backward: dy, dh, the gradient of gate and up, each
    with the forward's roundings of what it multiplies, and the result's own."""
    b = weights()
    x = tokens(T).requires_grad_(True)
    w13, w2 = b["w13"].requires_grad_(True), b["w2"].requires_grad_(True)
    with torch.no_grad():
        r = route(b, x)
    y = experts(x, w13, w2, r)
    c = torch.randn(y.shape, generator=torch.Generator().manual_seed(2))
    y.backward(c.to(DEV))
    x64, w1364, w264 = (t.detach().double().cpu().requires_grad_(True) for t in (x, w13, w2))
    want = experts64(x64, w1364, w264, r)
    want.backward(c.double())
    step = 2.0 ** -8
    assert off(y.detach(), want.detach()) <= 4 * step
    assert off(w2.grad, w264.grad) <= 6 * step
    assert off(w13.grad, w1364.grad) <= 8 * step
    assert off(x.grad, x64.grad) <= 9 * step
    empty = (r.group_list == 0).nonzero().flatten()
    assert (w13.grad[empty] == 0).all() and (w2.grad[empty] == 0).all()


@pytest.mark.parametrize("T", [1, 48, 700])
def test_block_with_adapters(T):
    """As above; the shared expert's pair has the same roundings."""
    b = weights()
    x = tokens(T)
    ids = torch.randint(-1, L, (T,), generator=torch.Generator().manual_seed(3),
                        dtype=torch.int32).to(DEV)
    r = route(b, x)
    got = experts(x, b["w13"], b["w2"], r) + shared(b, x, ids).float()
    d = {k: v.double().cpu() for k, v in b.items()}
    x64, i64 = x.double().cpu(), ids.cpu()

    def lora(v, w, a, bb):
        y = v @ w.T
        for i in range(L):
            t = (i64 == i).nonzero().flatten()
            y[t] += v[t] @ a[i].T @ bb[i].T
        return y

    gu = lora(x64, d["up"], d["up_a"], d["up_b"])
    h = torch.nn.functional.silu(gu[:, :SI]) * gu[:, SI:]
    want = experts64(x64, d["w13"], d["w2"], r) + lora(h, d["down"], d["down_a"], d["down_b"])
    assert off(got, want) <= 4 * 2.0 ** -8


def test_lora_training_by_grouped_products():
    """Rows sorted by adapter: two grouped products are the adapters' forward and, with
    their gradients, their training."""
    b = weights()
    counts = torch.tensor([30, 0, 77, 1, 20])
    x = tokens(int(counts.sum()))
    gl = counts.to(DEV)
    a, bb = b["up_a"].requires_grad_(True), b["up_b"].requires_grad_(True)
    inner = gfr.grouped_linear(x, a, gl, 1, transpose_w=True)
    y = gfr.grouped_linear(inner, bb, gl, 1, transpose_w=True, out_dtype=torch.float32)
    c = torch.randn(y.shape, generator=torch.Generator().manual_seed(2)).to(BF)
    y.backward(c.float().to(DEV))
    a64, b64 = (t.detach().double().cpu().requires_grad_(True) for t in (a, bb))
    rows = x.double().cpu().split(counts.tolist())
    want = torch.cat([v @ a64[i].T @ b64[i].T for i, v in enumerate(rows)])
    want.backward(c.double())
    assert off(y.detach(), want.detach()) <= 2.0 ** -8
    assert off(bb.grad, b64.grad) <= 2 * 2.0 ** -8
    assert off(a.grad, a64.grad) <= 2 * 2.0 ** -8
    # the serving call on the same rows and adapters
    ids = torch.arange(L, dtype=torch.int32).repeat_interleave(counts).to(DEV)
    zero = torch.zeros(2 * SI, H, dtype=BF, device=DEV)
    served = gfr.lora_linear(x, zero, a.detach(), bb.detach(), ids, out_dtype=torch.float32)
    assert off(served, want.detach()) <= 2.0 ** -15


@pytest.mark.parametrize("T", [8, 300])
def test_training_step_of_the_block_under_graph(T):
    b = weights()
    w13, w2 = b["w13"].requires_grad_(True), b["w2"].requires_grad_(True)
    x, c = tokens(T).requires_grad_(True), torch.ones(T, H, device=DEV)

    def step():
        with torch.no_grad():
            r = route(b, x)
        y = experts(x, w13, w2, r)
        return (y, *torch.autograd.grad(y, (x, w13, w2), c))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    torch.cuda.synchronize()
    for i in range(4):
        with torch.no_grad():
            x.copy_(tokens(T, seed=10 + i))
            c.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in out]
        want = [t.detach() for t in step()]
        torch.cuda.synchronize()
        # (index_add sums a token's rows, and the gradient of x's gather its rows', by
        # atomics: K = 4 FP32 additions of either order, then a rounding to bf16 in dx)
        assert off(got[0], want[0].double().cpu()) <= 4 * 2.0 ** -23
        assert off(got[1], want[1].double().cpu()) <= 2 * 4 * 2.0 ** -8
        assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])


def test_two_calls_at_once_on_two_streams():
    b = weights()
    xs = [tokens(T, T) for T in (300, 40, 700, 64)]
    rs = [route(b, x) for x in xs]
    want = []
    for x, r in zip(xs, rs):
        rows = x[r.row_index.long()]
        y = gfr.grouped_linear(rows, b["w13"], r.group_list, 1, transpose_w=True)
        want.append((rows, r, y, gfr.grouped_linear_wgrad(rows, y, r.group_list, 1,
                                                          transpose_w=True)))
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = [(gfr.grouped_linear(rows, b["w13"], r.group_list, 1, transpose_w=True,
                                   stream=s.cuda_stream),
                gfr.grouped_linear_wgrad(rows, y, r.group_list, 1, transpose_w=True,
                                         stream=s.cuda_stream))
               for (rows, r, y, _), s in zip(want, streams)]
    torch.cuda.synchronize()
    for (_, _, y, w), (gy, gw) in zip(want, got):
        assert torch.equal(y, gy) and torch.equal(w, gw)
