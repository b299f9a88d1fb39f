"""GPU results of gfr.linear on inputs whose sums FP32 holds exactly (exact_inputs):
equal to the definition, in every kernel, K split and epilogue (test_dispatch
asserts on the CPU that the sizes take the kernels named here)."""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr

from . import exact_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"

# M, N, K, activation, the kernel they take, whether it splits K.  N a multiple of 8:
# out's rows are whole 16 bytes.  K a multiple of 8: the rows of x and w are.
CASES = [
    # one, two and four fragments of 16 rows
    (1, 33, 200, "none", "rows", False), (5, 264, 1544, "relu", "rows", False),
    (16, 75, 203, "none", "rows", False), (7, 40, 264, "swiglu", "rows", False),
    (3, 33, 131, "swiglu", "rows", False), (17, 75, 264, "none", "rows", False),
    (31, 264, 267, "relu", "rows", False), (32, 72, 520, "swiglu", "rows", False),
    (29, 33, 131, "swiglu", "rows", False), (33, 33, 72, "none", "rows", False),
    (64, 600, 203, "none", "rows", False), (33, 75, 200, "swiglu", "rows", False),
    (61, 259, 203, "swiglu", "rows", False),
    # 64 x 64 tiles
    (65, 33, 328, "none", "64x64", False), (130, 72, 203, "relu", "64x64", False),
    (65, 33, 200, "swiglu", "64x64", False), (130, 72, 195, "swiglu", "64x64", False),
    (100, 72, 4104, "none", "64x64", True), (100, 75, 4107, "relu", "64x64", True),
    (1, 33, 4104, "none", "64x64", True), (200, 264, 2056, "swiglu", "64x64", True),
    (200, 259, 2051, "swiglu", "64x64", True),
    # 128 x 128 tiles
    (200, 4099, 264, "relu", "128x128", False), (200, 4104, 203, "none", "128x128", False),
    (200, 4099, 195, "swiglu", "128x128", False), (200, 4104, 200, "swiglu", "128x128", False),
    (65, 4099, 2056, "none", "128x128", True), (65, 4104, 2059, "none", "128x128", True),
    (65, 2051, 4107, "swiglu", "128x128", True), (4100, 16, 4104, "swiglu", "128x128", True),
    # 256 x 128 and 256 x 256 tiles
    (1000, 4099, 136, "none", "256x128", False), (1000, 4104, 264, "relu", "256x128", False),
    (450, 4099, 136, "swiglu", "256x128", False), (450, 4104, 264, "swiglu", "256x128", False),
    (4100, 2051, 136, "none", "256x256", False), (4100, 2048, 328, "relu", "256x256", False),
    (2600, 1500, 136, "swiglu", "256x256", False), (1000, 4104, 264, "swiglu", "256x256", False),
    # a long K
    (4, 64, 28672, "none", "64x64", True), (100, 64, 28680, "none", "64x64", True),
]


@pytest.mark.parametrize("M, N, K, act, kernel, split", CASES)
def test_equal_to_the_definition(M, N, K, act, kernel, split):
    for dtype, bias, residual in ((torch.bfloat16, torch.float32, True),
                                  (torch.float16, None, False)):
        print(M, N, K, act, dtype, bias, residual, flush=True)
        args, want, _ = exact_inputs.linear_case(M, N, K, act, dtype, bias, residual)
        args = {n: v.to(DEV) if torch.is_tensor(v) else v for n, v in args.items()}
        out = gfr.linear(**args, out_dtype=torch.float32)
        torch.cuda.synchronize()
        bad = (out.double().cpu() != torch.from_numpy(want)).nonzero()
        assert len(bad) == 0, f"{len(bad)} of {want.size} differ, first {bad[:3].tolist()}"
