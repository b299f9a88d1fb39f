"""GPU results of gfr.moe_decode on inputs whose sums FP32 holds exactly
(exact_inputs): equal to the definition, not near it."""
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
