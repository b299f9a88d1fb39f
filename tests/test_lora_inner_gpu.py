"""lora_linear keeps its inner row in 32 bits: integer inputs whose inner values need up to
21 bits (and lie beyond F16's range), while every sum stays exact in FP32; infinities in
lora_b as the definition has them, whatever the rank; a row's bits are its own."""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from tests import dispatch_rows
from tests.test_lora_linear_gpu import BF, DEV, F32, HF, call, definition, ids_of, integers, same

pytestmark = pytest.mark.gpu

INF = float("inf")
FEW = [(5, 136, 264), (64, 72, 520), (300, 264, 136), (331, 67, 133)]
MANY = [(4300, 2056, 136)]


def wide(M, N, K, L, r, dtype, mix):
    """CPU arguments: |inner| up to about 2^20, each column of an adapter's B with two
    non-zeros."""
    g = torch.Generator().manual_seed(M + 31 * N + K + r)

    def signed(low, high, *s):
        return torch.randint(low, high + 1, s, generator=g) * \
            (2 * torch.randint(0, 2, s, generator=g) - 1)

    a = integers(M, N, K, L, r, dtype, mix=mix)
    a["x"] = signed(64, 127, M, K).to(dtype)
    low = signed(128, 255, L, r, K)
    low[..., 128:] = 0
    a["a"] = low.to(dtype)
    b = torch.zeros(L, N, r)
    b.scatter_(2, torch.randint(0, r, (L, N, 2), generator=g), signed(1, 1, L, N, 2).float())
    a["b"] = b.to(dtype)
    a["scaling"][:] = 1
    return a


def inner_of(a):
    """All adapters' inner rows in 64 bits, and the most that a sum of the call can reach."""
    x, low = a["x"].double(), a["a"].double()
    inner = torch.einsum("mk,lrk->lmr", x, low)
    most = max((torch.einsum("mk,lrk->lmr", x.abs(), low.abs())).max().item(),
               2 * inner.abs().max().item())
    return inner, most + (x.abs() @ a["w"].double().abs().T).max().item()


def check(M, N, K, L, r, dtype, mix):
    print(M, N, K, L, r, dtype, mix, flush=True)
    a = wide(M, N, K, L, r, dtype, mix)
    inner, most = inner_of(a)
    # (sums of halves and quarters of them are exact too)
    assert most < 2 ** 22
    high = inner.to(BF).double()
    lost = high + (inner - high).to(BF).double() != inner
    assert lost.double().mean() > 0.03 and inner.abs().max() > 65504
    same(call(a, out_dtype=F32), definition(a))
    same(call(a, out_dtype=BF if dtype == BF else F32), definition(a))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("mix", ["one", "runs", "gaps"])
@pytest.mark.parametrize("r", [3, 4, 16, 24, 65, 72, 256])
@pytest.mark.parametrize("M, N, K", FEW)
def test_few_rows_keep_the_inner_row(M, N, K, r, mix, dtype):
    check(M, N, K, 5, r, dtype, mix)


@pytest.mark.parametrize("M, N, K, r", [(4400, 72, 1032, 128), (3000, 75, 2056, 20)])
def test_a_shrink_by_tiles_keeps_the_inner_row(M, N, K, r):
    assert 2 * M * r * K > 2e8
    check(M, N, K, 5, r, BF, "runs")
    check(M, N, K, 5, r, HF, "gaps")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("mix", ["one", "runs", "gaps"])
@pytest.mark.parametrize("r", [8, 16, 72, 256])
@pytest.mark.parametrize("M, N, K", MANY)
def test_whole_tiles_keep_the_inner_row(M, N, K, r, mix, dtype):
    assert dispatch_rows.lora(M, N, K, r)
    check(M, N, K, 3, r, dtype, mix)


def infinities(M, N, K, r, dtype, mix="random"):
    """One infinity of either sign in an adapter's B, and inner values of every kind
    beside it: large, of few bits, zero."""
    a = integers(M, N, K, 4, r, dtype, mix=mix)
    a["ids"][:4] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    for i, bad in ((1, INF), (2, -INF)):
        b = {**a, "b": a["b"].clone()}
        b["b"][i, N - 1, r - 1] = bad
        b["b"][i, 2, 0] = bad
        want = definition(b)
        assert want.isinf().any()
        same(call(b, out_dtype=F32), want, f"{r} {bad}")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("r", [5, 8, 12, 16, 72])
@pytest.mark.parametrize("M, N, K", FEW)
def test_infinities_in_b(M, N, K, r, dtype):
    infinities(M, N, K, r, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("r", [8, 72])
@pytest.mark.parametrize("mix", ["random", "runs"])
@pytest.mark.parametrize("M, N, K", MANY)
def test_infinities_in_b_of_whole_tiles(M, N, K, mix, r, dtype):
    infinities(M, N, K, r, dtype, mix)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("mix", ["one", "random"])
def test_whole_tiles_of_all_kinds_of_inner_values(mix, dtype):
    """A rank's inner value of 24 bits or few, of either sign, large, small or zero: its
    product with a power of two of B is exact."""
    M, N, K = MANY[0]
    a = integers(M, N, K, 3, 8, dtype, mix=mix)
    a["x"] = torch.zeros(M, K).to(dtype)
    a["w"][:, 0] = 0
    a["a"], a["b"] = torch.zeros(3, 8, K).to(dtype), torch.zeros(3, N, 8).to(dtype)
    power = torch.arange(M) % 26 - 12                      # 2^-12 .. 2^13, of either sign
    a["x"][:, 0] = (2.0 ** power * torch.where(torch.arange(M) % 2 == 0, 1, -1)).to(dtype)
    a["b"][:, :, 3] = (2.0 ** (torch.arange(N) % 20 - 8)).to(dtype)
    for scale in (1.0, 1.0 + 2.0 ** -23, 2.0 ** 60, 2.0 ** -60, 0.0):
        a["scaling"][:] = scale
        factors = [1.0, 2.0, 0.125] if scale % 2.0 ** -20 else [1.0, 3.0, 255.0]
        a["a"][:, 3, 0] = torch.tensor(factors).to(dtype)
        want = definition(a)
        assert torch.equal(want.float().double(), want)
        same(call(a, out_dtype=F32), want, str(scale))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("r", [8, 16, 40, 64, 200])
@pytest.mark.parametrize("M, N, K", [(40, 136, 264), (300, 264, 520), *MANY])
def test_a_row_keeps_its_bits_whatever_its_neighbours_ids(M, N, K, r, dtype):
    """One id changes in blocks of one adapter, another's in blocks of none."""
    g = torch.Generator().manual_seed(r + M)
    f = lambda *s: torch.randn(*s, generator=g)
    ids = torch.arange(M, dtype=torch.int32) // 128 % 4 - 1
    a = dict(x=f(M, K).to(dtype), w=(f(N, K) / K ** 0.5).to(dtype),
             a=(f(3, r, K) / K ** 0.5).to(dtype), b=f(3, N, r).to(dtype), ids=ids,
             scaling=0.5 + f(3).abs(), bias=f(N).to(dtype), residual=f(M, N).to(dtype))
    other = ids.clone()
    other[5::64] = (other[5::64] + 2) % 3
    same_id = other == ids
    assert 0 < (~same_id).sum() <= M / 32
    one, two = (call({**a, "ids": i}, out_dtype=F32) for i in (ids, other))
    torch.cuda.synchronize()
    assert torch.equal(one.cpu()[same_id], two.cpu()[same_id])
    assert not torch.equal(one, two)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_offsets_beyond_32_bits(dtype):
    """Sums that wait beyond 4 GiB, results beyond 2 GiB: the first and last rows are right."""
    M, N, K, L, r = 300000, 4096, 64, 3, 64
    assert dispatch_rows.lora(M, N, K, r)
    a = integers(M, N, K, L, r, dtype, mix="runs")
    ends = torch.cat([torch.arange(300), torch.arange(M - 300, M)])
    a["ids"][ends] = torch.arange(600, dtype=torch.int32) // 40 % 4 - 1
    y = call(a)
    part = {**a, "x": a["x"][ends], "ids": a["ids"][ends]}
    same(y[ends.to(y.device)], definition(part).to(dtype))


def tiled_f16(mix, **kw):
    assert dispatch_rows.lora(*MANY[0], 16)
    return integers(*MANY[0], 4, 16, HF, mix=mix, **kw)


@pytest.mark.parametrize("mix", ["one", "runs", "random"])
def test_f16_tiles_keep_nan_with_its_adapter_and_row(mix):
    a = tiled_f16(mix)
    a["ids"][:4] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    clean = definition(a)
    nan = float("nan")
    for t, i, value in (("a", 1, nan), ("b", 2, nan), ("b", 3, INF), ("scaling", 0, nan)):
        b = {**a, t: a[t].clone()}
        b[t][i] = value
        y, rest = call(b, out_dtype=F32).cpu(), a["ids"] != i
        same(y[rest], clean[rest], f"{t} {i}")
        if value != value:
            assert y[~rest].isnan().all()
    b = {**a, "x": a["x"].clone()}
    b["x"][2] = nan
    y, rest = call(b, out_dtype=F32).cpu(), torch.arange(a["x"].shape[0]) != 2
    same(y[rest], clean[rest], "row")
    assert y[2].isnan().all()


def test_f16_tiles_in_place_flags_and_nothing_outside():
    M, N, K = MANY[0]
    a = tiled_f16("random", residual=True)
    a["ids"][1], a["ids"][M - 1] = 4, -2
    want = definition({**a, "ids": torch.where((a["ids"] < 4) & (a["ids"] >= 0), a["ids"], -1)})
    buf = torch.full((M * N + 128,), 7.0, dtype=HF, device=DEV)
    out = buf[64:64 + M * N].view(M, N)
    out.copy_(a["residual"])
    need = gfr.lora_linear_workspace_size(M, N, K, 16)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert call(a, residual=out, out=out, workspace=ws[:need], status=status) is out
    same(out, want)
    assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all() and (ws[need:] == 255).all()
    assert status.item() == gfr.DEV_BAD_ADAPTER


def test_f16_tiles_under_graph_and_on_two_streams():
    a = tiled_f16("runs", bias=HF)
    d = {k: v.to(DEV) for k, v in a.items() if v is not None}
    run = lambda **kw: gfr.lora_linear(d["x"], d["w"], d["a"], d["b"], d["ids"],
                                       scaling=d["scaling"], bias=d["bias"], out_dtype=F32, **kw)
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
    for i, mix in enumerate(["random", "none", "one", "runs"]):
        a["ids"] = ids_of(MANY[0][0], 4, mix, i)
        d["ids"].copy_(a["ids"])
        graph.replay()
        same(y, definition(a), mix)
        torch.randn(256, 256, device=DEV).relu_()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        out = [run(stream=s.cuda_stream) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, out[0]) for o in out)
    same(out[0], definition(a))
