"""The direct kernel of the 16-bit grouped products (whole pieces straight to LDS), on
integer inputs: equal to the definition.  The sizes are asserted to take it."""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from tests import dispatch_rows
from tests import grouped_inputs as gi
from tests.test_grouped_linear_gpu import BF, DEV, F32, HF, NAN, check, dev, groups, same

# Groups that end in every tile shape (up to 32, 64, 128, 192 and 256 rows) and one behind
# each of their ends.
RESTS = [300, 520, 700, 33, 65, 0, 97, 161, 225, 1, 32, 64, 129, 193, 256]
# (counts, K, N): steps that end early, columns that do, few rows of a long sum
FEW = [([5, 0, 40, 64, 1], 4104, 264), ([1], 5000, 1032)]      # (the general kernel's)
FORWARD = [([5, 0, 40, 64, 1], 4104, 8200), ([1], 5000, 40008), ([100, 128, 0, 90], 392, 8200),
           (RESTS, 136, 4104), (RESTS, 200, 2568), ([2000], 1096, 2056), ([7] * 200, 72, 1032),
           ([3, 0] * 300, 1000, 264)]
WGRAD = [(RESTS, 520, 4104), (RESTS, 1032, 1544), ([5, 0, 40, 64, 1] * 4, 1000, 648),
         ([64, 65, 0, 63] * 6, 264, 2056), ([1] * 60, 1000, 648), ([700, 0, 1500], 2056, 2056)]


def test_the_sizes_take_the_direct_kernel():
    for counts, K, N in FORWARD:
        for t in (False, True):
            assert dispatch_rows.grouped(sum(counts), len(counts), K, N, False, t) == "direct"
    for counts, K, N in WGRAD:
        assert dispatch_rows.grouped(sum(counts), len(counts), K, N, True) == "direct"
        assert dispatch_rows.grouped(sum(counts), len(counts), N, K, True) == "direct"
    assert dispatch_rows.grouped(2000, 1, 1096, 2051, False, True) == "direct"


def test_the_other_kernels_are_taken_too():
    take = dispatch_rows.grouped
    assert take(512, 1, 2048, 1024) == "64" and take(512, 1, 2048, 1024, True) == "64"
    assert take(16384, 8, 2051, 4096) == "128" and take(16384, 8, 4096, 2051, True) == "128"
    assert take(2000, 1, 1096, 2051) == "64"                 # rows of w begin anywhere
    assert take(2001, 1, 2056, 4107, True) == "128" and take(2001, 4, 1097, 2056, True) == "128"
    assert take(0, 4, 64, 64) in ("64", "direct") and take(0, 4, 64, 64, True) in ("64", "direct")


@pytest.mark.gpu
@pytest.mark.parametrize("counts, K, N", FEW + FORWARD)
@pytest.mark.parametrize("transpose", [False, True])
def test_forward(counts, K, N, transpose):
    check(counts, K, N, BF, transpose, ops="f")
    check(counts, K, N, HF, transpose, out_dtype=None, kind=0, rest=70, ops="f")


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [F32, None])
def test_forward_with_rows_of_out_that_begin_anywhere(out_dtype):
    check([2000], 1096, 2051, BF, True, out_dtype=out_dtype, rest=9, ops="f")
    check(RESTS, 136, 4099, HF, True, out_dtype=out_dtype, ops="f")


@pytest.mark.gpu
@pytest.mark.parametrize("counts, K, N", WGRAD)
@pytest.mark.parametrize("transpose", [False, True])
def test_wgrad(counts, K, N, transpose):
    check(counts, K, N, BF, transpose, ops="w")
    check(counts, K, N, HF, transpose, out_dtype=None, kind=0, rest=70, ops="w")


@pytest.mark.gpu
def test_general_tiles_of_128():
    check([5000, 0, 3000, 8384], 131, 1032, BF, True, ops="f")
    check([1000, 0, 1000, 1], 1097, 2056, BF, False, ops="w")
    check([2001], 2056, 4107, HF, True, out_dtype=None, ops="w")


# Long sums of few tiles: steps that do not share out evenly among four groups of waves,
# rows that begin anywhere, more tiles than CUs (groups of one row), groups without steps.
LONG = [([5, 0, 40, 64, 1], 1281, 99), ([70], 2051, 515), ([1, 0, 3], 1344, 64),
        ([1] * 39 + [2521], 1288, 384), ([300, 7], 5000, 1032)]
LONG_WGRAD = [([1300, 0, 1, 4000], 130, 259), ([4097], 72, 1032), ([9, 1281, 2600], 64, 64),
              ([30, 0] * 8 + [8000, 9000, 12000], 136, 200)]


def test_long_sums_of_few_tiles_take_four_groups():
    for counts, K, N in LONG + FEW:
        for t in (False, True):
            assert dispatch_rows.grouped(sum(counts), len(counts), K, N, False, t,
                                         long=True) == "64 long"
    for counts, K, N in LONG_WGRAD:
        assert dispatch_rows.grouped(sum(counts), len(counts), K, N, True, long=True) == "64 long"
    # the same steps of more tiles; fewer steps
    assert dispatch_rows.grouped(1024, 2, 2048, 2048, long=True) == "64"
    assert dispatch_rows.grouped(1024, 1, 1024, 1024, long=True) == "64"


@pytest.mark.gpu
@pytest.mark.parametrize("counts, K, N", LONG)
@pytest.mark.parametrize("transpose", [False, True])
def test_long_sums(counts, K, N, transpose):
    check(counts, K, N, BF, transpose, ops="f")
    check(counts, K, N, HF, transpose, out_dtype=None, kind=0, rest=70, ops="f")


@pytest.mark.gpu
@pytest.mark.parametrize("counts, K, N", LONG_WGRAD)
@pytest.mark.parametrize("transpose", [False, True])
def test_long_sums_of_wgrad(counts, K, N, transpose):
    check(counts, K, N, BF, transpose, ops="w")
    check(counts, K, N, HF, transpose, out_dtype=None, kind=0, rest=70, ops="w")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_long_sums_add_up_keep_their_bits_and_their_place(dtype):
    counts, K, N = [1300, 0, 1, 4000], 130, 259
    M = sum(counts) + 5
    x, w, dy = gi.integers(counts, M, K, N, BF, False)
    want = gi.wgrad(x, dy, gi.ranges(counts, 1, M), False)
    old = torch.randint(-100, 100, want.shape).to(dtype)
    buf = torch.full((want.numel() + 128,), -5.0, dtype=dtype, device=DEV)
    out = buf[64:64 + want.numel()].view(want.shape)
    out.copy_(old)
    gfr.grouped_linear_wgrad(*dev(x, dy), groups(counts, 1), 1, out=out, accumulate=True)
    same(out, (old.double() + want).to(dtype), "accumulate")
    assert (buf[:64] == -5).all() and (buf[64 + want.numel():] == -5).all()
    x = torch.randn(300, 2051, device=DEV).bfloat16()
    w = torch.randn(3, 2051, 515, device=DEV).bfloat16()
    call = lambda c: gfr.grouped_linear(x, w, groups(c, 1), 1, out_dtype=dtype)
    one, two, three = call([100] * 3), call([100] * 3), call([30, 170, 100])
    assert torch.equal(one, two)
    for a, b in [(0, 30), (100, 300)]:
        assert torch.equal(one[a:b], three[a:b])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("transpose", [False, True])
def test_accumulate_and_nothing_outside(dtype, transpose):
    counts, K, N = [5, 0, 40, 64, 1] * 4, 1000, 648
    M = sum(counts) + 5
    x, w, dy = gi.integers(counts, M, K, N, BF, transpose)
    want = gi.wgrad(x, dy, gi.ranges(counts, 1, M), transpose)
    xd, dyd = dev(x, dy)
    old = torch.randint(-100, 100, want.shape).to(dtype)
    buf = torch.full((want.numel() + 128,), -5.0, dtype=dtype, device=DEV)
    out = buf[64:64 + want.numel()].view(want.shape)
    out.copy_(old)
    gfr.grouped_linear_wgrad(xd, dyd, groups(counts, 1), 1, transpose_w=transpose, out=out,
                             accumulate=True)
    same(out, (old.double() + want).to(dtype), "accumulate")
    gfr.grouped_linear_wgrad(xd, dyd, groups(counts, 1), 1, transpose_w=transpose, out=out)
    same(out, want.to(dtype), "overwrite")
    assert (buf[:64] == -5).all() and (buf[64 + want.numel():] == -5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [4104, 4099])
def test_rows_of_no_group_stay_and_nothing_outside(dtype, N):
    M = sum(RESTS) + 300
    x, w, _ = gi.integers(RESTS, M, 136, N, BF, True)
    want = gi.forward(x, w, gi.ranges(RESTS, 1, M), True, rest=-5.0)
    buf = torch.full((M * N + 128,), -5.0, dtype=dtype, device=DEV)
    out = buf[64:64 + M * N].view(M, N)
    xd, wd = dev(x, w)
    gfr.grouped_linear(xd, wd, groups(RESTS, 1), 1, transpose_w=True, out=out)
    same(out, want.to(dtype), "kept rows")
    assert (buf[:64] == -5).all() and (buf[64 + M * N:] == -5).all()
    fresh = gfr.grouped_linear(xd, wd, groups(RESTS, 1), 1, transpose_w=True, out_dtype=dtype)
    same(fresh, gi.forward(x, w, gi.ranges(RESTS, 1, M), True).to(dtype), "cleared rows")


@pytest.mark.gpu
@pytest.mark.parametrize("transpose", [False, True])
def test_nan_stays_where_it_belongs(transpose):
    K, N = 136, 4104
    M = sum(RESTS) + 20
    x, w, dy = gi.integers(RESTS, M, K, N, BF, transpose)
    rng = gi.ranges(RESTS, 1, M)
    x[sum(RESTS):] = NAN
    w[5] = NAN                                   # the expert without rows
    a, b = rng[3]
    x[a:b], w[3] = NAN, float("inf")
    x[rng[7][0] + 1, K - 1] = NAN
    w[9, 5 if transpose else K - 1, K - 1 if transpose else 5] = NAN
    y = gfr.grouped_linear(*dev(x, w), groups(RESTS, 1), 1, transpose_w=transpose, out_dtype=F32)
    same(y, gi.forward(x, w, rng, transpose), "forward")
    counts, K, N = [5, 0, 40, 64, 1] * 4, 1000, 648
    M = sum(counts) + 20
    x, w, dy = gi.integers(counts, M, K, N, BF, transpose)
    rng = gi.ranges(counts, 1, M)
    x[sum(counts):], dy[sum(counts):] = NAN, NAN
    x[rng[2][0]:rng[2][1]] = NAN
    dy[rng[8][0] + 3, N - 1] = float("inf")
    g = gfr.grouped_linear_wgrad(*dev(x, dy), groups(counts, 1), 1, transpose_w=transpose,
                                 out_dtype=F32)
    same(g, gi.wgrad(x, dy, rng, transpose), "wgrad")


@pytest.mark.gpu
@pytest.mark.parametrize("transpose", [False, True])
def test_bits(transpose):
    """Two calls give the same bits, and a row keeps its own whatever the groups."""
    g = torch.Generator().manual_seed(1)
    K, N = 1096, 2056
    x = torch.randn(2000, K, generator=g).bfloat16().to(DEV)
    w = torch.randn(4, *((N, K) if transpose else (K, N)), generator=g).bfloat16().to(DEV)
    call = lambda c: gfr.grouped_linear(x, w, groups(c, 1), 1, transpose_w=transpose,
                                        out_dtype=F32)
    one, two, three = call([500] * 4), call([500] * 4), call([30, 970, 17, 983])
    torch.cuda.synchronize()
    assert torch.equal(one, two)
    for a, b in [(0, 30), (500, 1000), (1000, 1017), (1500, 2000)]:
        assert torch.equal(one[a:b], three[a:b])


@pytest.mark.gpu
@pytest.mark.parametrize("kind, values", [(1, [700, -3, 9, 5000]), (0, [2000, 30, 2500, 2100])])
def test_bad_lists(kind, values):
    K, N, M = 1096, 2056, 2050
    x, w, dy = gi.integers([0] * 4, M, K, N, BF)
    gl = torch.tensor(values, dtype=torch.int64, device=DEV)
    rng = gi.ranges(values, kind, M)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = gfr.grouped_linear(*dev(x, w), gl, kind, out_dtype=F32, status=status)
    same(y, gi.forward(x, w, rng, False), "forward")
    assert status.item() == gfr.DEV_BAD_GROUP_LIST
    g = gfr.grouped_linear_wgrad(*dev(x, dy), gl, kind, out_dtype=F32)
    same(g, gi.wgrad(x, dy, rng, False), "wgrad")


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Weights of 5 GiB and rows behind the 2 GiB mark: the last expert and row are right."""
    E, K, N = 330, 2048, 4096
    w = torch.zeros(E, K, N, dtype=BF, device=DEV)
    x = torch.zeros(700000, K, dtype=BF, device=DEV)
    w[E - 1, K - 1] = torch.arange(N, device=DEV).remainder(200).to(BF)
    w[0, 0] = 3
    x[-300:, K - 1] = 2
    x[:300, 0] = 1
    counts = torch.zeros(E, dtype=torch.int64, device=DEV)
    counts[0], counts[E - 1] = 699700, 300
    y = torch.empty(700000, N, dtype=BF, device=DEV)
    gfr.grouped_linear(x, w, counts, 1, out=y)
    assert (y[:300] == 3).all() and (y[300:699700].abs().amax() == 0)
    assert torch.equal(y[-300:], (2 * w[E - 1, K - 1])[None].expand(300, N))
    g = gfr.grouped_linear_wgrad(x, y, counts, 1, out=torch.empty_like(w))
    want = (600 * y[-1].float()).to(BF)
    assert torch.equal(g[E - 1, K - 1], want) and (g[E - 1, :K - 1] == 0).all()
    assert (g[0, 0] == 900).all() and (g[1:E - 1] == 0).all()
