"""GPU results of gfr.moe_decode on inputs whose sums FP32 holds exactly
(exact_inputs): equal to the definition, not near it, in every variant of the two
products (test_dispatch asserts on the CPU that the sizes take the variants named
here)."""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr

from . import exact_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def check(*sizes, **kw):
    print(sizes, kw, flush=True)
    args, want, _ = exact_inputs.decode_case(*sizes, **kw)
    args = {n: v.to(DEV) if torch.is_tensor(v) else v for n, v in args.items()}
    out = gfr.moe_decode(**args, out_dtype=torch.float32).double().cpu()
    torch.cuda.synchronize()
    bad = (out != torch.from_numpy(want)).nonzero()
    assert len(bad) == 0, f"{len(bad)} of {want.size} differ, first {bad[:3].tolist()}"


# silu(gate) * up, here of 18 to 23 bits, goes into the down product whole: formed by
# its blocks (below 32 pairs) and once ahead of them
@pytest.mark.parametrize("t13, t2", [(False, False), (True, True), (True, False), (False, True)])
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("T, k, E, H, I, N, spread", [
    (1, 2, 4, 128, 512, 512, 1), (9, 2, 8, 192, 320, 384, 1), (16, 2, 3, 128, 1024, 1024, 1),
    (40, 2, 3, 128, 128, 64, 2), (64, 4, 16, 256, 576, 640, 1)])
def test_silu_times_up_is_not_rounded(T, k, E, H, I, N, spread, fp8, t13, t2):
    check(T, k, E, H, I, N, fp8, t13, t2, per_expert=T % 2 == 0, spread=spread)


# T, k, E, H, I, N, and of each product: waves of a block, whether these share a tile
# and whether a wave takes several tiles.  Weights [K, N] and [N, K].
KN = [
    (1, 8, 128, 768, 256, 512, (4, 1, 0), (4, 1, 0)),
    (2, 3, 5, 4160, 448, 1344, (4, 1, 0), (4, 1, 0)),
    (3, 8, 8, 64, 1024, 6400, (4, 1, 0), (4, 0, 0)),
    (8, 6, 8, 1088, 3200, 192, (4, 0, 0), (4, 1, 0)),
    (16, 16, 128, 1088, 64, 192, (4, 0, 0), (4, 1, 0)),
    (16, 8, 128, 512, 512, 512, (4, 1, 0), (4, 1, 0)),
    (24, 8, 64, 64, 64, 6400, (4, 1, 0), (4, 0, 0)),
    (48, 16, 256, 64, 64, 3264, (4, 1, 0), (4, 0, 1)),
    (24, 16, 256, 64, 2048, 192, (4, 0, 1), (4, 0, 0)),
    (16, 16, 64, 64, 3200, 192, (8, 0, 0), (4, 1, 0)),
    (33, 16, 128, 64, 3200, 192, (8, 0, 1), (4, 0, 0)),
    (16, 16, 64, 64, 64, 6400, (4, 1, 0), (8, 0, 0)),
    (33, 16, 128, 64, 64, 6400, (4, 1, 0), (8, 0, 1)),
    (17, 1, 1, 320, 192, 192, (4, 0, 0), (4, 0, 0)),
    (48, 16, 64, 64, 2048, 192, (8, 0, 0), (4, 0, 0)),
    (48, 16, 64, 64, 64, 6400, (4, 0, 0), (8, 0, 0)),
    (64, 8, 8, 64, 3200, 6400, (4, 0, 0), (8, 0, 1)),
]
NK = [
    (1, 8, 256, 512, 192, 320, (4, 0, 0), (4, 0, 0)),
    (3, 6, 8, 64, 3200, 6400, (4, 0, 0), (4, 0, 1)),
    (16, 8, 128, 512, 256, 512, (4, 0, 0), (4, 0, 0)),
    (17, 6, 32, 64, 3200, 192, (4, 0, 1), (4, 0, 0)),
    (8, 16, 16, 64, 3200, 192, (8, 0, 0), (4, 0, 0)),
    (8, 16, 32, 64, 3200, 192, (8, 0, 1), (4, 0, 0)),
    (8, 16, 16, 64, 64, 6400, (4, 0, 0), (8, 0, 0)),
    (8, 16, 32, 64, 64, 6400, (4, 0, 0), (8, 0, 1)),
    (17, 1, 1, 320, 192, 192, (4, 0, 0), (4, 0, 0)),
    (64, 16, 16, 1088, 2048, 192, (4, 0, 1), (4, 0, 0)),
    (64, 16, 16, 64, 3200, 192, (8, 0, 0), (4, 0, 0)),
    (48, 16, 64, 64, 2048, 192, (8, 0, 1), (4, 0, 0)),
    (48, 16, 16, 64, 320, 6400, (4, 0, 0), (4, 0, 1)),
    (64, 16, 16, 64, 64, 6400, (4, 0, 0), (8, 0, 0)),
    (48, 16, 64, 64, 64, 6400, (4, 0, 0), (8, 0, 1)),
]


@pytest.mark.parametrize("T, k, E, H, I, N, gate_up, down", KN)
def test_weights_kn(T, k, E, H, I, N, gate_up, down):
    check(T, k, E, H, I, N, "e4m3" if T % 3 else "e5m2", False, False, per_expert=T % 2 == 0)


@pytest.mark.parametrize("T, k, E, H, I, N, gate_up, down", NK)
def test_weights_nk(T, k, E, H, I, N, gate_up, down):
    check(T, k, E, H, I, N, "e4m3" if T % 3 else "e5m2", True, True, per_expert=T % 2 == 0)


# E8M0's ends: code 0 is 2^-127, and a weight is exact while it is a multiple of 2^-133,
# bf16's smallest value (any code times 2^-124 for E4M3, 2^-117 for E5M2)
@pytest.mark.parametrize("t", [False, True])
@pytest.mark.parametrize("fp8, exact_from, values", [
    ("e4m3", 3, [1.0, 1.875, 448.0, 2.0 ** -6, 1.75 * 2.0 ** -6, 1.5 * 2.0 ** -8, 2.0 ** -9]),
    ("e5m2", 10, [1.0, 1.75, 57344.0, 2.0 ** -14, 1.5 * 2.0 ** -15, 2.0 ** -16])])
def test_smallest_and_largest_scales(fp8, exact_from, values, t):
    x = torch.zeros(1, 64)
    x[0, 0], x[0, 1] = 2.0 ** 60, 2.0 ** 50       # gate and up: h = 2^110
    w13 = torch.zeros(1, 64, 128)
    w13[0, 0, :64] = w13[0, 1, 64:] = 1
    s13 = torch.full((1, 128, 2), 127, dtype=torch.uint8)
    flip = lambda v, *dims: (v.permute(*dims) if t else v).contiguous().to(DEV)
    for value in values:
        w2 = torch.zeros(1, 64, 64)
        w2[0, 0] = value
        # h * weight stays below 2^128 (codes in order, then up to 2^4)
        codes = torch.tensor([*range(40), *range(100, 124)], dtype=torch.uint8)
        for s in (codes, codes + 8 if value <= 1 else codes):
            s2 = torch.full((1, 64, 2), 127, dtype=torch.uint8)
            s2[0, :, 0] = s
            out = gfr.moe_decode(
                x.bfloat16().to(DEV), flip(w13.to(exact_inputs.FP8[fp8]), 0, 2, 1),
                flip(s13, 1, 0, 2), flip(w2.to(exact_inputs.FP8[fp8]), 0, 2, 1),
                flip(s2, 1, 0, 2), torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                torch.ones(1, 1, device=DEV), transpose_w13=t, transpose_w2=t,
                out_dtype=torch.float32).double().cpu()[0]
            want = value * 2.0 ** (110.0 + s.double() - 127)
            assert want.max() < 2.0 ** 128
            smallest = value * 2.0 ** (s.double() - 127)
            whole = (smallest / 2.0 ** -133) % 1 == 0
            assert torch.equal(out[whole], want[whole]), (fp8, value)
            assert whole[s >= exact_from].all()
            # below, off by at most one such step
            assert ((out - want).abs() <= 2.0 ** (110 - 133)).all()
