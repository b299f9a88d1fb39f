"""GPU parity of gfr.linear against the float64 oracle (oracle.layer.linear).

Tolerance: the oracle's bound of the FP32 computation (each of the K additions
rounds once, by at most 2^-23 of the largest possible partial sum, carried
through the activation's slope), plus half a step of out's type.
"""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
# mantissa bits and smallest normal exponent
FORMATS = {torch.bfloat16: (7, -126), torch.float16: (10, -14), torch.float32: (23, -126)}


def make(M, N, K, dtype, act="none", bias=None, residual=False, seed=0):
    g = torch.Generator().manual_seed(seed + 7919 * M + 31 * N + K)
    rows = 2 * N if act == "swiglu" else N
    r = lambda *s: torch.randn(*s, generator=g)
    return dict(x=r(M, K).to(dtype).to(DEV), w=(r(rows, K) / K ** 0.5).to(dtype).to(DEV),
                bias=None if bias is None else r(rows).to(bias).to(DEV),
                residual=r(M, N).to(dtype).to(DEV) if residual else None)


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(out, a, act, what):
    want, bound = layer.linear(host(a["x"]), host(a["w"]), host(a["bias"]), act,
                               host(a["residual"]))
    got = host(out)
    tol = bound + layer.half_step(np.abs(want) + bound, *FORMATS[out.dtype])
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, worst "
                           f"{np.nanmax(err / tol):.3g} of the tolerance at "
                           f"{np.argwhere(bad)[:3].tolist()}")


def run(M, N, K, dtype=torch.bfloat16, act="none", bias=None, residual=False, out_dtype=None):
    what = f"M {M} N {N} K {K} {dtype} {act} bias {bias} residual {residual} out {out_dtype}"
    print(what, flush=True)
    a = make(M, N, K, dtype, act, bias, residual)
    out = gfr.linear(a["x"], a["w"], a["bias"], activation=act, residual=a["residual"],
                     out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert out.shape == (M, N) and out.dtype == (out_dtype or dtype)
    check(out, a, act, what)


# one row to the edges of the row kernel's fragments, the tile kernel from 65;
# K below one step, whole steps, tails of whole and of broken eights; N below a
# fragment, odd
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("N, K", [(1, 8), (16, 64), (17, 72), (50, 520), (96, 1024), (67, 136)])
def test_sizes_aligned(M, N, K):
    run(M, N, K, out_dtype=torch.float32)


@pytest.mark.parametrize("M", [1, 5, 16, 31, 64, 97, 129])
@pytest.mark.parametrize("N, K", [(3, 1), (17, 63), (33, 65), (48, 130), (51, 263), (64, 515)])
def test_sizes_unaligned(M, N, K):
    run(M, N, K, dtype=torch.float16, out_dtype=torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("M, N, K", [(3, 48, 256), (40, 35, 192), (150, 130, 320)])
def test_epilogues(dtype, act, M, N, K):
    run(M, N, K, dtype, act, bias=dtype, residual=True)
    run(M, N, K, dtype, act, bias=torch.float32, residual=False)
    run(M, N, K, dtype, act, bias=None, residual=True, out_dtype=torch.float32)


@pytest.mark.parametrize("M, N, K", [(9, 23, 77), (70, 45, 131), (300, 129, 67)])
def test_swiglu_odd_rows(M, N, K):
    # odd N and K: the up rows begin at an odd element
    run(M, N, K, torch.bfloat16, "swiglu", bias=torch.bfloat16, residual=True)


@pytest.mark.parametrize("M, N, K, act", [(2048, 6144, 192, "none"), (4100, 4099, 136, "silu"),
                                          (1500, 5000, 200, "swiglu"), (700, 2304, 131, "gelu"),
                                          (8200, 257, 264, "relu")])
def test_large_tiles(M, N, K, act):
    run(M, N, K, torch.bfloat16, act, bias=torch.bfloat16, residual=True)


# few tiles of a long K: the K split and its joining launch, rows that begin
# anywhere and aligned ones, two split halves under swiglu
@pytest.mark.parametrize("M, N, K, act", [(100, 72, 4104, "silu"), (100, 75, 4107, "none"),
                                          (700, 600, 4104, "none"), (200, 264, 2056, "swiglu"),
                                          (200, 259, 2051, "swiglu"), (50, 72, 4104, "relu"),
                                          (331, 4099, 1544, "gelu"), (450, 2056, 2059, "none"),
                                          (450, 1032, 1544, "swiglu"),
                                          (450, 1029, 1549, "swiglu")])
def test_split_k(M, N, K, act):
    run(M, N, K, torch.bfloat16, act, bias=torch.bfloat16, residual=True)
    run(M, N, K, torch.float16, act, out_dtype=torch.float32)


# tiles of 256 x 128, aligned columns and not
@pytest.mark.parametrize("M, N, K, act", [(2100, 2050, 72, "none"), (2100, 1032, 136, "swiglu"),
                                          (2600, 1041, 200, "swiglu")])
def test_oblong_tiles(M, N, K, act):
    run(M, N, K, torch.float16, act, bias=torch.float32, residual=True)


def test_split_k_in_place_and_workspace_of_the_caller():
    from mxfp8_grouped_gemm_group_amd import _layer
    M, N, K = 100, 72, 4104
    a = make(M, N, K, torch.bfloat16, residual=True)
    want = gfr.linear(a["x"], a["w"], residual=a["residual"])
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)      # NaN sums
    out = a["residual"].clone()
    gfr.linear(a["x"], a["w"], residual=out, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(gfr.GfrError) as e:
        gfr.linear(a["x"], a["w"], workspace=ws[:256])
    assert e.value.code == _layer.WORKSPACE_TOO_SMALL


def test_long_k():
    run(4, 64, 28672, torch.bfloat16, out_dtype=torch.float32)
    run(100, 64, 28680, torch.float16)


def test_infinities_and_nan_reach_their_rows_alone():
    a = make(6, 40, 200, torch.bfloat16)
    want = gfr.linear(a["x"], a["w"], activation="relu")
    x = a["x"].clone()
    x[2, 7] = float("nan")
    x[4, 199] = float("inf")
    got = gfr.linear(x, a["w"], activation="relu")
    torch.cuda.synchronize()
    assert torch.isnan(got[2]).all()
    assert torch.isinf(got[4][a["w"][:, 199] > 0]).all()
    assert (got[4][a["w"][:, 199] < 0] == 0).all()
    rest = [0, 1, 3, 5]
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("M", [5, 100, 300])
def test_values_behind_k_are_not_read(M):
    """K ends inside a step and the next row begins right behind it: NaN there
    must not reach this row."""
    K = 72
    a = make(M, 40, K, torch.bfloat16)
    want = gfr.linear(a["x"], a["w"])
    x = a["x"].clone()
    x[1:] = float("nan")
    got = gfr.linear(x, a["w"])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.isnan(got[1:]).all()
    w = a["w"].clone()
    w[1:] = float("nan")
    got = gfr.linear(a["x"], w)
    torch.cuda.synchronize()
    assert torch.equal(got[:, 0], want[:, 0]) and torch.isnan(got[:, 1:]).all()


@pytest.mark.parametrize("M, N, K", [(3, 33, 100), (77, 50, 96), (260, 300, 128)])
def test_residual_in_place_and_nothing_outside_out(M, N, K):
    a = make(M, N, K, torch.bfloat16, residual=True)
    want = gfr.linear(a["x"], a["w"], residual=a["residual"])
    buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[32:32 + M * N].view(M, N)
    out.copy_(a["residual"])
    got = gfr.linear(a["x"], a["w"], residual=out, out=out)
    torch.cuda.synchronize()
    assert got is out and torch.equal(out, want)
    assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()


@pytest.mark.parametrize("M, N, K", [(1, 256, 2048), (48, 100, 1000), (331, 515, 1032)])
def test_same_bits_twice(M, N, K):
    a = make(M, N, K, torch.bfloat16, "silu", bias=torch.bfloat16)
    one = gfr.linear(a["x"], a["w"], a["bias"], activation="silu")
    two = gfr.linear(a["x"], a["w"], a["bias"], activation="silu")
    torch.cuda.synchronize()
    assert torch.equal(one, two)


def test_empty():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.randn(8, 64, device=DEV).bfloat16()
    assert gfr.linear(x, w).shape == (0, 8)
    assert gfr.linear(w, x).shape == (8, 0)
