"""lora_linear on integer inputs whose sums FP32 holds exactly: equal to the 64-bit
definition (rounded once, where out is 16 bits wide); random ones within the bound of
FP32 sums and of an inner row of 16 bits."""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


def ids_of(M, L, mix, seed=0):
    """Adapters of the rows: one for all, runs, a row's own, with and without gaps."""
    g = torch.Generator().manual_seed(seed + M)
    if mix == "one":
        return torch.full((M,), L - 1, dtype=torch.int32)
    if mix == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if mix == "runs":
        lengths = torch.randint(1, 90, (M,), generator=g)
        which = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
        return which.repeat_interleave(lengths)[:M].contiguous()
    return torch.randint(-1 if mix == "gaps" else 0, L, (M,), generator=g, dtype=torch.int32)


def integers(M, N, K, L, r, dtype, mix="gaps", bias=None, residual=False, scaling=True, seed=0):
    """CPU arguments.  The sums of magnitudes: the dense one at most 16 K, inner at most
    2 * 2 * 4 * 32 = 512 (a row of lora_a has at most 32 non-zeros), its products with
    lora_b at most 256 * 512 * 4 = 2^19, bias and residual 200: below 2^24 for K <= 2^19."""
    g = torch.Generator().manual_seed(seed + 7919 * M + 31 * N + K + r)
    draw = lambda high, *s: torch.randint(-high, high + 1, s, generator=g, dtype=torch.int8)
    a = torch.zeros(L, r, K)
    where = torch.randint(0, K, (L, r, 32), generator=g)
    a.scatter_(2, where, torch.randint(-2, 3, where.shape, generator=g).float())
    return dict(x=draw(4, M, K).to(dtype), w=draw(4, N, K).to(dtype), a=a.to(dtype),
                b=draw(4, L, N, r).to(dtype), ids=ids_of(M, L, mix, seed),
                scaling=(2.0 ** torch.randint(-1, 2, (L,), generator=g)).float()
                if scaling else None,
                bias=None if bias is None else draw(100, N).to(bias),
                residual=draw(100, M, N).to(dtype) if residual else None)


def definition(a):
    x = a["x"].double()
    y = x @ a["w"].double().T
    for i in range(a["a"].shape[0]):
        t = torch.nonzero(a["ids"] == i).flatten()
        if len(t):
            inner = x[t] @ a["a"][i].double().T
            if a["scaling"] is not None:
                inner = inner * a["scaling"][i].double()
            y[t] += inner @ a["b"][i].double().T
    for extra in ("bias", "residual"):
        if a[extra] is not None:
            y += a[extra].double()
    return y


def call(a, **over):
    d = {k: None if v is None else v.to(DEV) for k, v in a.items()}
    return gfr.lora_linear(d["x"], d["w"], d["a"], d["b"], d["ids"],
                           **{**dict(scaling=d["scaling"], bias=d["bias"],
                                     residual=d["residual"]), **over})


def same(got, want, what=""):
    torch.cuda.synchronize()
    got, want = got.cpu(), want.to(got.dtype)
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at " \
                          f"{bad.nonzero()[:3].tolist()}"


def check(M, N, K, L, r, dtype=BF, out_dtype=F32, **kw):
    what = f"M {M} N {N} K {K} L {L} r {r} {dtype} {kw}"
    print(what, flush=True)
    a = integers(M, N, K, L, r, dtype, **kw)
    y = call(a, out_dtype=out_dtype)
    assert y.shape == (M, N) and y.dtype == (out_dtype or dtype)
    same(y, definition(a), what)


@pytest.mark.parametrize("M", [1, 2, 15, 17, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("N, K, r", [(8, 8, 8), (64, 64, 16), (136, 72, 64), (320, 264, 24),
                                     (264, 520, 128)])
def test_sizes_aligned(M, N, K, r):
    check(M, N, K, 5, r, BF)
    check(M, N, K, 3, r, HF, bias=HF, residual=True, mix="runs")


@pytest.mark.parametrize("M", [1, 5, 31, 64, 97, 290])
@pytest.mark.parametrize("N, K, r", [(1, 1, 1), (17, 63, 3), (33, 65, 12), (130, 131, 20),
                                     (515, 264, 7), (67, 72, 8), (72, 67, 16), (40, 72, 100)])
def test_sizes_unaligned(M, N, K, r):
    check(M, N, K, 4, r, HF)
    check(M, N, K, 6, r, BF, bias=BF, residual=True, mix="runs")


@pytest.mark.parametrize("M", [3, 64, 200, 700])
@pytest.mark.parametrize("mix", ["one", "none", "runs", "gaps", "random"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_mixes(M, mix, dtype):
    check(M, 264, 136, 40, 16, dtype, mix=mix, bias=F32)
    check(M, 264, 136, 7, 40, dtype, mix=mix, out_dtype=None, residual=True, scaling=False)


@pytest.mark.parametrize("r", [1, 2, 4, 8, 16, 32, 48, 64, 65, 96, 128, 200, 256])
@pytest.mark.parametrize("M", [4, 300])
def test_ranks(M, r):
    check(M, 136, 264, 3, r)


@pytest.mark.parametrize("M, N, K, L, r", [(700, 2056, 520, 9, 16), (1100, 600, 72, 300, 8),
                                           (64, 72, 4104, 64, 16), (257, 1032, 1096, 2, 64),
                                           (2100, 264, 264, 3, 32), (1, 4104, 2056, 4, 64)])
def test_shapes(M, N, K, L, r):
    check(M, N, K, L, r, bias=BF, residual=True, mix="runs")
    check(M, N, K, L, r, mix="random", out_dtype=None)


def test_inner_row_keeps_its_bits():
    """Inner values up to 2^15: no rounding to the inputs' type."""
    M, N, K, L, r = 300, 72, 264, 3, 16
    a = integers(M, N, K, L, r, BF, mix="runs")
    a["a"] = a["a"] * 64
    a["scaling"][:] = 1
    for rows in (M, 40):
        b = {**a, "x": a["x"][:rows], "ids": a["ids"][:rows]}
        inner = max((b["x"].double() @ a["a"][i].double().T).abs().max() for i in range(L))
        assert 2 ** 12 < inner < 2 ** 16
        same(call(b, out_dtype=F32), definition(b))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M, mix", [(5, "random"), (64, "gaps"), (300, "runs"), (300, "random")])
def test_random_values_within_the_bound(dtype, M, mix):
    """Of FP32 sums (K and r additions, 2^-23 of the sum of magnitudes each) and an inner
    row of 16 bits (2^-16), plus, with F16, its spacing at zero, 2^-24."""
    N, K, L, r = 200, 520, 6, 24
    g = torch.Generator().manual_seed(M)
    f = lambda *s: torch.randn(*s, generator=g)
    a = dict(x=f(M, K).to(dtype), w=(f(N, K) / K ** 0.5).to(dtype),
             a=(f(L, r, K) / K ** 0.5).to(dtype), b=(0.1 * f(L, N, r)).to(dtype),
             ids=ids_of(M, L, mix), scaling=(0.5 + f(L).abs()), bias=f(N).to(dtype),
             residual=f(M, N).to(dtype))
    want = definition(a)
    h = lambda t: t.double().abs()
    bound = (K + 2) * 2.0 ** -23 * (h(a["x"]) @ h(a["w"]).T + h(a["bias"]) + h(a["residual"]))
    for i in range(L):
        t = torch.nonzero(a["ids"] == i).flatten()
        if len(t) == 0:
            continue
        inner = h(a["x"])[t] @ h(a["a"][i]).T * a["scaling"][i].double()
        mag = inner @ h(a["b"][i]).T
        bound[t] += ((K + r + 4) * 2.0 ** -23 + 2.0 ** -16) * mag
        bound[t] += 2.0 ** -24 * h(a["b"][i]).sum(1)
    for out_dtype in (F32, None):
        got = call(a, out_dtype=out_dtype).double().cpu()
        tol = bound
        if out_dtype is None:
            tol = tol + torch.from_numpy(layer.half_step(
                (want.abs() + bound).numpy(), *((7, -126) if dtype == BF else (10, -14))))
        assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("M, mix", [(6, "random"), (64, "random"), (300, "runs"),
                                    (300, "random")])
@pytest.mark.parametrize("K, r", [(72, 16), (67, 5)])
def test_nan_stays_with_its_adapter_and_row(M, mix, K, r):
    N, L = 136, 4
    a = integers(M, N, K, L, r, BF, mix=mix)
    a["ids"][:4] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    clean = definition(a)
    for t, i in (("a", 1), ("b", 2)):
        for bad in (NAN, float("inf")):
            b = {**a, t: a[t].clone()}
            b[t][i] = bad
            y = call(b, out_dtype=F32)
            torch.cuda.synchronize()
            rest = a["ids"] != i
            same(y.cpu()[rest], clean[rest], f"{t} {i} {bad}")
            if bad != bad:
                assert y.cpu()[~rest].isnan().all()
    b = {**a, "x": a["x"].clone()}
    b["x"][2] = NAN
    y = call(b, out_dtype=F32).cpu()
    rest = torch.arange(M) != 2
    same(y[rest], clean[rest], "row")
    assert y[2].isnan().all()
    # scaling of another adapter
    b = {**a, "scaling": a["scaling"].clone()}
    b["scaling"][3] = NAN
    rest = a["ids"] != 3
    same(call(b, out_dtype=F32).cpu()[rest], clean[rest], "scaling")


@pytest.mark.parametrize("M", [4, 300])
def test_ids_out_of_range_have_no_adapter_and_are_flagged(M):
    a = integers(M, 72, 136, 5, 16, BF, mix="random")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    same(call(a, out_dtype=F32, status=status), definition(a))
    assert status.item() == 0
    a["ids"][1] = 5
    a["ids"][2] = -2
    a["ids"][3] = 2 ** 31 - 1
    want = definition({**a, "ids": torch.where((a["ids"] < 5) & (a["ids"] >= 0), a["ids"], -1)})
    same(call(a, out_dtype=F32, status=status), want)
    assert status.item() == gfr.DEV_BAD_ADAPTER


@pytest.mark.parametrize("M, N, K", [(3, 33, 100), (64, 136, 72), (300, 257, 136), (300, 264, 136)])
def test_residual_in_place_workspace_of_the_caller_and_nothing_outside_out(M, N, K):
    a = integers(M, N, K, 4, 16, BF, residual=True)
    want = definition(a).to(BF)
    buf = torch.full((M * N + 128,), 7.0, dtype=BF, device=DEV)
    out = buf[64:64 + M * N].view(M, N)
    out.copy_(a["residual"])
    need = gfr.lora_linear_workspace_size(M, N, K, 16)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)       # NaN sums
    got = call(a, residual=out, out=out, workspace=ws[:need])
    assert got is out
    same(out, want)
    assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all() and (ws[need:] == 255).all()
    if need:
        with pytest.raises(gfr.GfrError):
            call(a, workspace=ws[:need - 1])


@pytest.mark.parametrize("M, K", [(1, 2056), (64, 264), (300, 520), (300, 67)])
def test_same_bits_twice(M, K):
    g = torch.Generator().manual_seed(1)
    a = integers(M, 264, K, 4, 16, BF)
    a["x"], a["a"] = torch.randn(M, K, generator=g).to(BF), torch.randn(4, 16, K, generator=g).to(BF)
    one, two = call(a, out_dtype=F32), call(a, out_dtype=F32)
    torch.cuda.synchronize()
    assert torch.equal(one, two)


def test_empty():
    a = integers(4, 8, 64, 2, 8, BF)
    d = {k: v.to(DEV) for k, v in a.items() if v is not None}
    assert gfr.lora_linear(d["x"][:0], d["w"], d["a"], d["b"], d["ids"][:0]).shape == (0, 8)
    assert gfr.lora_linear(d["x"], d["w"][:0], d["a"], d["b"][:, :0].contiguous(),
                           d["ids"]).shape == (4, 0)


@pytest.mark.parametrize("M, N, K", [(1, 264, 520), (48, 136, 264), (300, 264, 264)])
def test_under_graph_with_other_ids(M, N, K):
    a = integers(M, N, K, 5, 16, BF, mix="random", bias=BF)
    d = {k: v.to(DEV) for k, v in a.items() if v is not None}
    run = lambda: gfr.lora_linear(d["x"], d["w"], d["a"], d["b"], d["ids"], scaling=d["scaling"],
                                  bias=d["bias"], out_dtype=F32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    torch.cuda.synchronize()
    for i in range(5):
        b = integers(M, N, K, 5, 16, BF, mix=["runs", "none", "one", "gaps", "random"][i], bias=BF,
                     seed=i)
        for k in ("x", "ids", "bias", "scaling"):
            a[k] = b[k]
            d[k].copy_(b[k])
        graph.replay()
        same(y, definition(a), str(i))
        torch.randn(256, 256, device=DEV).relu_()


def test_two_calls_at_once_on_two_streams():
    sets = [integers(M, 264, 520, 5, 16, BF, seed=M) for M in (64, 300, 40, 700)]
    want = [definition(a) for a in sets]
    dev = [{k: v.to(DEV) for k, v in a.items() if v is not None} for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    out = []
    for _ in range(3):
        out = [gfr.lora_linear(d["x"], d["w"], d["a"], d["b"], d["ids"], scaling=d["scaling"],
                               out_dtype=F32, stream=s.cuda_stream)
               for d, s in zip(dev, streams)]
    torch.cuda.synchronize()
    for y, z in zip(out, want):
        same(y, z)


# ---- whole tiles, which expand in their epilogue: 128 of them or more -----------------


TILED = dict(M=4300, N=2056, K=72)


def test_tiles_are_taken():
    from tests import dispatch_rows
    assert dispatch_rows.lora(4300, 2056, 72, 16) and dispatch_rows.lora(4300, 2056, 72, 200)
    for M, N, K, r in [(4300, 2056, 71, 16), (4300, 2055, 72, 16), (4300, 2056, 72, 12),
                       (256, 2056, 72, 16)]:
        assert not dispatch_rows.lora(M, N, K, r)


@pytest.mark.parametrize("mix", ["one", "none", "runs", "gaps", "random"])
@pytest.mark.parametrize("dtype, r", [(BF, 16), (HF, 40)])
def test_tiles_mixes(mix, dtype, r):
    check(**TILED, L=9, r=r, dtype=dtype, mix=mix, bias=F32)
    check(**TILED, L=40, r=r, dtype=dtype, mix=mix, out_dtype=None, residual=True, scaling=False)
    check(**TILED, L=9, r=r, dtype=dtype, mix=mix, out_dtype=None, residual=True, bias=dtype)


@pytest.mark.parametrize("r", [8, 24, 64, 72, 128, 200, 256])
def test_tiles_ranks(r):
    check(**TILED, L=3, r=r, mix="runs")


@pytest.mark.parametrize("M, N, K", [(4097, 2048, 8), (3900, 2312, 136), (4200, 1800, 520),
                                     (32800, 264, 64), (100, 32776, 64), (4290, 2056, 264)])
def test_tiles_shapes(M, N, K):
    # a last tile of 1, 32, 64, 100 (one), 104 and 192 rows or so; few and many columns
    check(M, N, K, 5, 16, mix="runs", bias=BF, residual=True, out_dtype=None)


def test_tiles_inner_row_keeps_its_bits():
    a = integers(**TILED, L=3, r=16, dtype=BF, mix="runs")
    a["a"] = a["a"] * 64
    a["scaling"][:] = 1
    same(call(a, out_dtype=F32), definition(a))


@pytest.mark.parametrize("mix", ["runs", "random"])
def test_tiles_nan_stays_with_its_adapter_and_row(mix):
    L = 4
    a = integers(**TILED, L=L, r=16, dtype=BF, mix=mix)
    a["ids"][:4] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    clean = definition(a)
    for t, i in (("a", 1), ("b", 2)):
        for bad in (NAN, float("inf")):
            b = {**a, t: a[t].clone()}
            b[t][i] = bad
            y = call(b, out_dtype=F32).cpu()
            rest = a["ids"] != i
            same(y[rest], clean[rest], f"{t} {i} {bad}")
            if bad != bad:
                assert y[~rest].isnan().all()
    b = {**a, "x": a["x"].clone()}
    b["x"][2] = NAN
    y = call(b, out_dtype=F32).cpu()
    rest = torch.arange(TILED["M"]) != 2
    same(y[rest], clean[rest], "row")
    assert y[2].isnan().all()


def test_tiles_in_place_flags_and_nothing_outside_out():
    M, N, K = TILED.values()
    a = integers(**TILED, L=4, r=16, dtype=BF, residual=True, mix="random")
    a["ids"][1], a["ids"][M - 1] = 4, -2
    want = definition({**a, "ids": torch.where((a["ids"] < 4) & (a["ids"] >= 0), a["ids"], -1)})
    buf = torch.full((M * N + 128,), 7.0, dtype=BF, device=DEV)
    out = buf[64:64 + M * N].view(M, N)
    out.copy_(a["residual"])
    need = gfr.lora_linear_workspace_size(M, N, K, 16)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)       # NaN terms
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert call(a, residual=out, out=out, workspace=ws[:need], status=status) is out
    same(out, want)
    assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all() and (ws[need:] == 255).all()
    assert status.item() == gfr.DEV_BAD_ADAPTER


def test_tiles_same_bits_twice_and_under_graph():
    a = integers(**TILED, L=5, r=16, dtype=BF, mix="runs", bias=BF)
    d = {k: v.to(DEV) for k, v in a.items() if v is not None}
    run = lambda: gfr.lora_linear(d["x"], d["w"], d["a"], d["b"], d["ids"], scaling=d["scaling"],
                                  bias=d["bias"], out_dtype=F32)
    assert torch.equal(run(), run())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    torch.cuda.synchronize()
    for i in range(3):
        a["ids"] = ids_of(TILED["M"], 5, ["random", "one", "runs"][i], i)
        d["ids"].copy_(a["ids"])
        graph.replay()
        same(y, definition(a), str(i))
        torch.randn(256, 256, device=DEV).relu_()


# few columns or ranks in fours alone, many rows: the shrink by tiles ahead of rows' expansion
@pytest.mark.parametrize("M, N, K, r", [(4400, 72, 2056, 128), (4000, 71, 1096, 36),
                                        (3000, 75, 2056, 20)])
@pytest.mark.parametrize("mix", ["runs", "gaps"])
def test_shrink_by_tiles_and_rows_expanded(M, N, K, r, mix):
    assert 2 * M * r * K > 2e8
    check(M, N, K, 5, r, mix=mix, bias=BF)
    check(M, N, K, 5, r, dtype=HF, mix=mix, residual=True, out_dtype=None)


@pytest.mark.parametrize("M, N, K", [(5, 136, 72), (300, 136, 264), (4300, 2056, 72)])
@pytest.mark.parametrize("r", [8, 5])
def test_infinities_as_the_definition_has_them(M, N, K, r):
    """An infinite inner value gives infinities (and NaN for a zero beside it), not NaN all
    over: x, an adapter's row and a scaling that are infinite."""
    a = integers(M, N, K, 3, r, BF, mix="random")
    a["ids"][:3] = torch.tensor([0, 1, 2], dtype=torch.int32)
    a["b"][a["b"] == 0] = 1
    for change in ("x", "a", "scaling"):
        b = {**a, change: a[change].clone()}
        if change == "x":
            b["x"][1, K - 1] = float("inf")
        elif change == "a":
            b["a"][1, r - 1, 3] = float("-inf")
            b["x"][:, 3] = 2
        else:
            b["scaling"][2] = float("inf")
        same(call(b, out_dtype=F32), definition(b), change)
