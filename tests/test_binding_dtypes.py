"""Which torch dtypes the Python layer hands to the library, and how it refuses the
others."""
import pytest
import torch

from mxfp8_grouped_gemm_group_amd import _binding, _layer


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.bool])
def test_grouped_calls_refuse_by_value_error(dtype):
    """Callers catch ValueError for a dtype that no grouped call takes."""
    with pytest.raises(ValueError):
        _binding.tensor_desc(torch.zeros(4, dtype=dtype))


def test_layer_calls_take_float16():
    assert _layer._words(torch.float16, (4, 8)) == (11 | 2 << 32, 4, 8, 0, 0)
    assert _layer._words(torch.bfloat16, (4, 8)) == (5 | 2 << 32, 4, 8, 0, 0)
    with pytest.raises(ValueError):
        _layer._words(torch.float64, (4, 8))


@pytest.mark.gpu
def test_grouped_product_refuses_float16_by_value_error():
    import mxfp8_grouped_gemm_group_amd as gfr
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device="cuda:0")
    f8 = lambda *s: z(*s).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        gfr.gmm_finalize_routing(f8(2, 64), f8(1, 64, 64), z(1, 64, 2), z(2, 1, 2),
                                 z(1, dtype=torch.int64), 1, z(2, dtype=torch.float16),
                                 z(2, dtype=torch.int64), None, 1.0, 0,
                                 z(2, 64, dtype=torch.float32))
