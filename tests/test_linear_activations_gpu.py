"""gfr.linear's activations at exact sums (one product of a row by a power of two):
relative to the result also where it is small.

Tolerance: oracle.layer.activation_error relative to the result, plus half a step of
out's type.
"""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
FORMATS = {torch.bfloat16: (7, -126), torch.float16: (10, -14), torch.float32: (23, -126)}


# the row kernel, tiles, K splits with rows that begin at 16 bytes and anywhere
@pytest.mark.parametrize("M, N, K", [(40, 16, 8), (700, 16, 8), (700, 17, 9), (100, 72, 4104),
                                     (100, 75, 4107)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_small_results_below_zero(M, N, K, act):
    v = torch.linspace(-9, 9, M).bfloat16()
    powers = 2.0 ** -(torch.arange(N) % 4)
    for dtype in (torch.bfloat16, torch.float16):
        x, w = torch.zeros(M, K, dtype=dtype), torch.zeros(N, K, dtype=dtype)
        x[:, K // 2], w[:, K // 2] = v.to(dtype), powers.to(dtype)
        y = x[:, K // 2].double()[:, None].numpy() * powers.double().numpy()
        want = layer.activate(y, act)
        for out_dtype in (dtype, torch.float32):
            print(M, N, K, act, dtype, out_dtype, flush=True)
            out = gfr.linear(x.to(DEV), w.to(DEV), activation=act, out_dtype=out_dtype)
            torch.cuda.synchronize()
            bound = layer.activation_error(y, act) * np.abs(want)
            tol = bound + layer.half_step(np.abs(want) + bound, *FORMATS[out_dtype])
            err = np.abs(out.double().cpu().numpy() - want)
            bad = np.argwhere(~(err <= tol))
            assert len(bad) == 0, (f"{len(bad)} off, worst {np.max(err / tol):.3g} of the "
                                   f"tolerance at y {y[tuple(bad[0])]}")
