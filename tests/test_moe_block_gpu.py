"""The operators of a MoE block used together, under HIP graphs, on other
streams, and two calls at once.

The block: router logits (linear) -> moe_route -> the experts -> out, with the
shared expert's two dense products.  Few tokens take moe_decode; more take
moe_route's sorted, quantised rows through gemm1_swiglu_quant and
gmm_finalize_routing.
"""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E, K, H, I, SI = 16, 4, 512, 256, 384       # experts, top-k, widths, shared expert's width


def block(seed=0):
    g = torch.Generator().manual_seed(seed)
    code = lambda *s: torch.randn(*s, generator=g).to(torch.float8_e4m3fn).to(DEV)
    scale = lambda *s: torch.randint(119, 122, s, generator=g, dtype=torch.uint8).to(DEV)
    w = lambda n, k: (torch.randn(n, k, generator=g) / k ** 0.5).bfloat16().to(DEV)
    return dict(router=w(E, H), bias=(0.1 * torch.randn(E, generator=g)).to(DEV),
                w13=code(E, H, 2 * I), s13=scale(H // 64, 2 * I, 2), w2=code(E, I, H),
                s2=scale(I // 64, H, 2), up=w(2 * SI, H), down=w(H, SI))


def tokens(T, seed=1):
    return torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)


ROUTER = dict(scoring="sigmoid", n_group=4, topk_group=2, scaling=1.5)


def few(b, x):
    logits = gfr.linear(x, b["router"], out_dtype=torch.float32)
    r = gfr.moe_route(logits, K, bias=b["bias"], **ROUTER)
    shared = gfr.linear(gfr.linear(x, b["up"], activation="swiglu"), b["down"])
    return gfr.moe_decode(x, b["w13"], b["s13"], b["w2"], b["s2"], r.topk_ids, r.topk_weights,
                          shared_input=shared)


def many(b, x):
    logits = gfr.linear(x, b["router"], out_dtype=torch.float32)
    r = gfr.moe_route(logits, K, x=x, bias=b["bias"], **ROUTER)
    shared = gfr.linear(gfr.linear(x, b["up"], activation="swiglu"), b["down"])
    x1, s1 = gfr.gemm1_swiglu_quant(r.xin, b["w13"], b["s13"], r.xin_scale, r.group_list, 1)
    out = torch.zeros(x.shape[0], H, device=DEV)
    return gfr.gmm_finalize_routing(x1, b["w2"], b["s2"], s1, r.group_list, 1, r.logit,
                                    r.row_index, shared, 1.0, 0, out, deterministic=True)


def reference(b, x):
    """float64 from the block's definition, no intermediate rounded."""
    h = lambda t: t.detach().double().cpu().numpy()
    u8 = lambda t: t.contiguous().view(torch.uint8).cpu().numpy()
    xs = h(x)
    ids, w = layer.moe_route(np.float32(xs @ h(b["router"]).T), K, h(b["bias"]), **ROUTER)
    gu = xs @ h(b["up"]).T
    shared = (layer.silu(gu[:, :SI]) * gu[:, SI:]) @ h(b["down"]).T
    w13 = layer.mx_weights(u8(b["w13"]), u8(b["s13"]), False, 0)
    w2 = layer.mx_weights(u8(b["w2"]), u8(b["s2"]), False, 0)
    out, _ = layer.moe_decode(xs, w13, w2, ids, w, shared, 1.0)
    return out


def test_block_few_and_many_tokens_agree_with_the_definition():
    """Relative to the block's norm: bf16 roundings of the shared expert's hidden
    row, its result and the output (2^-8 each at most, in the 2-norm), plus, in
    the grouped chain, two MXFP8 quantisations (half an E4M3 step, 2^-4, of each
    element at most: of x and of silu(gate) * up; gate and up both carry x's)."""
    b = block()
    x = tokens(24)
    want = reference(b, x)
    norm = np.linalg.norm(want)
    a = few(b, x).double().cpu().numpy()
    c = many(b, x).double().cpu().numpy()
    assert np.linalg.norm(a - want) <= 3 * 2.0 ** -8 * norm
    assert np.linalg.norm(c - want) <= (3 * 2.0 ** -4 + 2 * 2.0 ** -8) * norm


def test_one_token_equals_its_row_of_a_batch_in_the_choice():
    b = block()
    x = tokens(40)
    logits = gfr.linear(x, b["router"], out_dtype=torch.float32)
    r = gfr.moe_route(logits, K, x=x, bias=b["bias"], **ROUTER)
    one = gfr.moe_route(logits[7:8].contiguous(), K, x=x[7:8].contiguous(), bias=b["bias"],
                        **ROUTER)
    torch.cuda.synchronize()
    assert torch.equal(r.topk_ids[7:8], one.topk_ids)
    assert torch.equal(r.topk_weights[7:8], one.topk_weights)
    rows = (r.row_index == 7).nonzero().flatten()
    assert torch.equal(r.xin.view(torch.uint8)[rows], one.xin.view(torch.uint8))


@pytest.mark.parametrize("run, T", [(few, 1), (few, 24), (few, 64), (many, 24), (many, 300)])
def test_block_under_graph(run, T):
    b = block()
    x, y = tokens(T), tokens(T, 2)
    want_x, want_y = run(b, x).clone(), run(b, y).clone()
    static = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(b, static)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(b, static)
    torch.cuda.synchronize()
    noise = torch.randn(512, 512, device=DEV)
    for i in range(5):
        static.copy_(y if i % 2 else x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_y if i % 2 else want_x), f"replay {i}"
        _ = (noise @ noise).sum().item()
        run(b, y)                                # eager calls between the replays
    del g


def test_two_graphs_and_eager_calls_share_nothing():
    b = block()
    x, y = tokens(9), tokens(9, 2)
    want_x, want_y = few(b, x).clone(), few(b, y).clone()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in (x, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(few(b, t))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = few(b, x)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want_x) and torch.equal(outs[1], want_y)
        assert torch.equal(eager, want_x)


def test_two_streams_at_once():
    b = block()
    x, y = tokens(24), tokens(24, 2)
    want = [f(b, t).clone() for f in (few, many) for t in (x, y)]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(6):
        with torch.cuda.stream(s):
            a, c = few(b, x), many(b, x)
        with torch.cuda.stream(t):
            d, e = few(b, y), many(b, y)
        torch.cuda.synchronize()
        for got, w in zip((a, d, c, e), want):
            assert torch.equal(got, w)


def test_explicit_stream_owns_what_it_allocates():
    """stream= runs the call, and allocates its output and workspace, on that
    stream: a slow stream's result is not handed to later work of the current
    one's allocator."""
    b = block()
    x = tokens(24)
    want = few(b, x).clone()
    logits = gfr.linear(x, b["router"], out_dtype=torch.float32)
    r = gfr.moe_route(logits, K, bias=b["bias"], **ROUTER)
    shared = gfr.linear(gfr.linear(x, b["up"], activation="swiglu"), b["down"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=DEV)
    for _ in range(3):
        with torch.cuda.stream(s):
            for _ in range(4):
                big = big @ big * 1e-3
        out = gfr.moe_decode(x, b["w13"], b["s13"], b["w2"], b["s2"], r.topk_ids,
                             r.topk_weights, shared_input=shared, stream=s.cuda_stream)
        lg = gfr.linear(x, b["router"], out_dtype=torch.float32, stream=s.cuda_stream)
        rt = gfr.moe_route(logits, K, bias=b["bias"], stream=s.cuda_stream, **ROUTER)
        junk = [torch.full((1 << 16,), float("nan"), device=DEV) for _ in range(8)]
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(lg, logits)
        assert torch.equal(rt.topk_ids, r.topk_ids)
        del junk
    assert torch.equal(gfr.linear(x, b["router"], out_dtype=torch.float32,
                                  stream=torch.cuda.default_stream().cuda_stream), logits)
    torch.cuda.synchronize()


def test_refusals_on_the_device():
    b = block()
    x = tokens(4)
    with pytest.raises(ValueError):
        gfr.linear(x.t(), b["router"].t())                       # not contiguous
    with pytest.raises(ValueError):
        gfr.linear(x, b["router"].cpu())
    with pytest.raises(gfr.GfrError):
        gfr.linear(x, b["router"].float())
    with pytest.raises(gfr.GfrError):
        gfr.linear(x, b["router"][:, :256].contiguous())
    with pytest.raises(gfr.GfrError):
        gfr.moe_route(torch.zeros(4, 8, device=DEV), 9)
    with pytest.raises(gfr.GfrError):
        gfr.moe_route(torch.zeros(4, 8, device=DEV), 2, n_group=3)
    with pytest.raises(gfr.GfrError):
        gfr.moe_route(torch.zeros(4, 8, device=DEV), 2, x=x[:, :40].contiguous())
    ids = torch.zeros(65, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(gfr.GfrError):
        gfr.moe_decode(tokens(65), b["w13"], b["s13"], b["w2"], b["s2"], ids,
                       torch.ones(65, 2, device=DEV))
    with pytest.raises(gfr.GfrError):
        gfr.moe_decode(x, b["w13"], b["s13"], b["w2"], b["s2"], ids[:4].long(),
                       torch.ones(4, 2, device=DEV))
