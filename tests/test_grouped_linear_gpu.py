"""grouped_linear and grouped_linear_wgrad on integer inputs, whose sums FP32 holds
exactly: equal to the 64-bit definition (rounded once, where out is 16 bits wide).  A
row of a neighbouring group, a lost tail or step, and sums in fewer bits all show."""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from tests import grouped_inputs as gi

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


def dev(*tensors):
    return [t.to(DEV) for t in tensors]


def groups(counts, kind):
    return torch.tensor(gi.as_list(counts, kind), dtype=torch.int64, device=DEV)


def same(got, want, what):
    torch.cuda.synchronize()
    got, want = got.cpu(), want.to(got.dtype)
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at " \
                          f"{bad.nonzero()[:3].tolist()}"


def check(counts, K, N, dtype=BF, transpose=False, out_dtype=F32, kind=1, rest=0, ops="fw"):
    M = sum(counts) + rest
    what = f"counts {counts} rest {rest} K {K} N {N} {dtype} transpose {transpose} {out_dtype}"
    print(what, flush=True)
    x, w, dy = gi.integers(counts, M, K, N, dtype, transpose)
    rng = gi.ranges(counts, 1, M)
    gl = groups(counts, kind)
    xd, wd, dyd = dev(x, w, dy)
    if "f" in ops:
        y = gfr.grouped_linear(xd, wd, gl, kind, transpose_w=transpose, out_dtype=out_dtype)
        assert y.shape == (M, N) and y.dtype == (out_dtype or dtype)
        same(y, gi.forward(x, w, rng, transpose), "forward " + what)
    if "w" in ops:
        g = gfr.grouped_linear_wgrad(xd, dyd, gl, kind, transpose_w=transpose,
                                     out_dtype=out_dtype)
        assert g.shape == w.shape
        same(g, gi.wgrad(x, dy, rng, transpose), "wgrad " + what)


LISTS = [[1], [0, 1, 0], [3, 0, 5, 1], [17, 130, 0, 64, 1, 31], [255, 256, 257, 0, 2]]


@pytest.mark.parametrize("counts", LISTS)
@pytest.mark.parametrize("K, N", [(8, 8), (64, 64), (72, 136), (264, 320), (200, 520)])
@pytest.mark.parametrize("transpose", [False, True])
def test_sizes_aligned(counts, K, N, transpose):
    check(counts, K, N, BF, transpose)
    check(counts, K, N, HF, transpose, kind=0, rest=5)


@pytest.mark.parametrize("counts", LISTS)
@pytest.mark.parametrize("K, N", [(1, 1), (3, 129), (63, 65), (130, 7), (257, 515), (136, 33),
                                  (67, 128)])
@pytest.mark.parametrize("transpose", [False, True])
def test_sizes_unaligned(counts, K, N, transpose):
    check(counts, K, N, HF, transpose)
    check(counts, K, N, BF, transpose, kind=0, rest=3)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("K, N", [(264, 320), (130, 257)])
def test_sixteen_bit_results(dtype, transpose, K, N):
    check([40, 0, 300, 7], K, N, dtype, transpose, out_dtype=None, rest=9)


# rows of every kind of rest over whole blocks, long sums, many small experts, one
# expert that has everything, sums over many rows, one row to an expert
@pytest.mark.parametrize("counts, K, N", [
    ([700, 33, 1, 520, 96, 65], 1096, 776), ([3000], 520, 264), ([2] * 300 + [0] * 724, 64, 40),
    ([0] * 1023 + [77], 64, 48), ([5000, 1, 0, 900], 136, 264), ([1] * 64, 2056, 264),
    ([16] * 5, 4104, 72), ([33, 64, 48], 72, 4104), ([130] * 9, 520, 1032)])
@pytest.mark.parametrize("transpose", [False, True])
def test_shapes(counts, K, N, transpose):
    check(counts, K, N, BF, transpose)


@pytest.mark.parametrize("transpose", [False, True])
def test_no_rows(transpose):
    check([0, 0, 0], 72, 40, transpose=transpose)
    check([0, 0], 72, 40, transpose=transpose, rest=6)
    x, w, dy = dev(*gi.integers([0, 0], 0, 64, 0, BF, transpose))
    gl = groups([0, 0], 1)
    assert gfr.grouped_linear(x, w, gl, 1, transpose_w=transpose).shape == (0, 0)
    assert gfr.grouped_linear_wgrad(x, dy, gl, 1, transpose_w=transpose).shape == w.shape


@pytest.mark.parametrize("kind, lists", [
    (1, [[4, -3, 9], [4, 400, 9], [70, 70, 70], [2 ** 62, 1, 2 ** 62], [-2 ** 62, 5, 5]]),
    (0, [[9, 4, 30], [4, 400, 500], [-5, 10, 20], [2 ** 62, 2 ** 62, 2 ** 62]])])
@pytest.mark.parametrize("K, N", [(72, 264), (67, 33)])
def test_bad_lists_are_clamped_and_flagged(kind, lists, K, N):
    M = 100
    x, w, dy = gi.integers([0] * 3, M, K, N, BF)
    xd, wd, dyd = dev(x, w, dy)
    for values in lists:
        print(kind, values, flush=True)
        gl = torch.tensor(values, dtype=torch.int64, device=DEV)
        rng = gi.ranges(values, kind, M)
        for call, args, want in [
                (gfr.grouped_linear, (xd, wd), gi.forward(x, w, rng, False)),
                (gfr.grouped_linear_wgrad, (xd, dyd), gi.wgrad(x, dy, rng, False))]:
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            same(call(*args, gl, kind, out_dtype=F32, status=status), want, str(values))
            assert status.item() == gfr.DEV_BAD_GROUP_LIST
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gfr.grouped_linear(xd, wd, groups([30, 0, 70], kind), kind, status=status)
    gfr.grouped_linear_wgrad(xd, dyd, groups([30, 0, 70], kind), kind, status=status)
    assert status.item() == 0


@pytest.mark.parametrize("counts", [[40, 0, 300, 7], [3, 0, 5, 2]])
@pytest.mark.parametrize("K, N", [(72, 264), (67, 33), (264, 256)])
@pytest.mark.parametrize("transpose", [False, True])
def test_rows_of_no_group_stay_and_nothing_outside_out(counts, K, N, transpose):
    M = sum(counts) + 20
    x, w, dy = gi.integers(counts, M, K, N, BF, transpose)
    rng = gi.ranges(counts, 1, M)
    want = gi.forward(x, w, rng, transpose, rest=-5.0)
    for dtype in (BF, F32):
        buf = torch.full((M * N + 128,), -5.0, dtype=dtype, device=DEV)
        out = buf[64:64 + M * N].view(M, N)
        xd, wd, dyd = dev(x, w, dy)
        got = gfr.grouped_linear(xd, wd, groups(counts, 1), 1, transpose_w=transpose, out=out)
        assert got is out
        same(out, want.to(dtype), "kept rows")
        assert (buf[:64] == -5).all() and (buf[64 + M * N:] == -5).all()
        size = w.numel()
        buf = torch.full((size + 128,), -5.0, dtype=dtype, device=DEV)
        out = buf[64:64 + size].view(w.shape)
        gfr.grouped_linear_wgrad(xd, dyd, groups(counts, 1), 1, transpose_w=transpose, out=out)
        same(out, gi.wgrad(x, dy, rng, transpose).to(dtype), "wgrad in a buffer")
        assert (buf[:64] == -5).all() and (buf[64 + size:] == -5).all()


@pytest.mark.parametrize("K, N", [(72, 264), (67, 33), (128, 256)])
@pytest.mark.parametrize("transpose", [False, True])
def test_accumulate(K, N, transpose):
    counts = [40, 0, 300, 7]
    M = sum(counts) + 5
    x, w, dy = gi.integers(counts, M, K, N, BF, transpose)
    want = gi.wgrad(x, dy, gi.ranges(counts, 1, M), transpose)
    xd, dyd = dev(x, dy)
    for dtype in (F32, BF):
        old = torch.randint(-100, 100, want.shape).to(dtype)
        out = old.to(DEV)
        got = gfr.grouped_linear_wgrad(xd, dyd, groups(counts, 1), 1, transpose_w=transpose,
                                       out=out, accumulate=True)
        assert got is out
        # (16 bits: the FP32 sum of both, rounded once)
        same(out, (old.double() + want).to(dtype), "accumulate")


@pytest.mark.parametrize("counts", [[40, 0, 300, 7], [3, 0, 5, 2]])
@pytest.mark.parametrize("K, N", [(72, 264), (67, 33), (256, 520), (200, 40)])
@pytest.mark.parametrize("transpose", [False, True])
def test_nan_stays_where_it_belongs(counts, K, N, transpose):
    """NaN in rows behind the last group, in another group's rows, and in the weights
    of an expert without rows reaches nothing else."""
    M = sum(counts) + 20
    x, w, dy = gi.integers(counts, M, K, N, BF, transpose)
    rng = gi.ranges(counts, 1, M)
    x[sum(counts):], dy[sum(counts):] = NAN, NAN
    w[1] = NAN
    gl = groups(counts, 1)
    xd, wd, dyd = dev(x, w, dy)
    y = gfr.grouped_linear(xd, wd, gl, 1, transpose_w=transpose, out_dtype=F32)
    same(y, gi.forward(x, w, rng, transpose), "clean rows")
    g = gfr.grouped_linear_wgrad(xd, dyd, gl, 1, transpose_w=transpose, out_dtype=F32)
    same(g, gi.wgrad(x, dy, rng, transpose), "clean groups")
    # the third group's rows and its weights
    a, b = rng[2]
    x[a:b], w[2] = NAN, float("inf")
    xd, wd = dev(x, w)
    y = gfr.grouped_linear(xd, wd, gl, 1, transpose_w=transpose, out_dtype=F32)
    same(y, gi.forward(x, w, rng, transpose), "rows of the others")
    g = gfr.grouped_linear_wgrad(xd, dyd, gl, 1, transpose_w=transpose, out_dtype=F32)
    same(g, gi.wgrad(x, dy, rng, transpose), "gradients of the others")
    # one element: its row, and its row or column of the gradient
    x, w, dy = gi.integers(counts, M, K, N, BF, transpose)
    x[a + 1, K - 1] = NAN
    dy[a, N - 1] = NAN
    xd, wd, dyd = dev(x, w, dy)
    y = gfr.grouped_linear(xd, wd, gl, 1, transpose_w=transpose, out_dtype=F32)
    same(y, gi.forward(x, w, rng, transpose), "one row")
    g = gfr.grouped_linear_wgrad(xd, dyd, gl, 1, transpose_w=transpose, out_dtype=F32)
    same(g, gi.wgrad(x, dy, rng, transpose), "one row and column")


@pytest.mark.parametrize("counts, K, N", [([40, 0, 300, 7], 264, 520), ([3, 0, 5, 2], 1032, 264),
                                          ([40, 0, 300, 7], 67, 33)])
@pytest.mark.parametrize("transpose", [False, True])
def test_same_bits_twice(counts, K, N, transpose):
    M = sum(counts)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=g).bfloat16().to(DEV)
    dy = torch.randn(M, N, generator=g).bfloat16().to(DEV)
    w = torch.randn(4, *((N, K) if transpose else (K, N)), generator=g).bfloat16().to(DEV)
    gl = groups(counts, 1)
    one, two = (gfr.grouped_linear(x, w, gl, 1, transpose_w=transpose, out_dtype=F32)
                for _ in range(2))
    three, four = (gfr.grouped_linear_wgrad(x, dy, gl, 1, transpose_w=transpose, out_dtype=F32)
                   for _ in range(2))
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(three, four)


@pytest.mark.parametrize("K, N", [(264, 520), (67, 33)])
@pytest.mark.parametrize("transpose", [False, True])
def test_a_row_keeps_its_bits_whatever_the_group_sizes(K, N, transpose):
    """A row's sum depends on the sizes of the call alone: moving other rows between
    groups leaves its bits."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(400, K, generator=g).bfloat16().to(DEV)
    w = torch.randn(4, *((N, K) if transpose else (K, N)), generator=g).bfloat16().to(DEV)
    one = gfr.grouped_linear(x, w, groups([100, 100, 100, 100], 1), 1, transpose_w=transpose,
                             out_dtype=F32)
    two = gfr.grouped_linear(x, w, groups([3, 197, 7, 193], 1), 1, transpose_w=transpose,
                             out_dtype=F32)
    torch.cuda.synchronize()
    for a, b in [(0, 3), (100, 200), (200, 207), (300, 400)]:
        assert torch.equal(one[a:b], two[a:b])
