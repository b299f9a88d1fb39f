"""gfr_lora_linear's limit on rows and ranks, on both sides, without a device."""
import pytest

import mxfp8_grouped_gemm_group_amd as gfr
from tests.test_lora_abi import BF16, UNSUPPORTED, desc, lora


@pytest.mark.parametrize("r", [1, 4, 5, 8, 13, 16, 256])
def test_rows_times_ranks_in_fours(r):
    """M times r, rounded up to a multiple of four, up to 2^27 (and M up to 2^26)."""
    fours = (r + 3) // 4 * 4
    most = min(2 ** 27 // fours, 2 ** 26)
    assert gfr.lora_linear_workspace_size(most, 8, 64, r) >= 4 * most * r
    with pytest.raises(gfr.GfrError) as e:
        gfr.lora_linear_workspace_size(most + 1, 8, 64, r)
    assert e.value.code == UNSUPPORTED
    assert lora(M=most + 1, N=8, r=r, residual=desc(BF16, most + 1, 8)) == UNSUPPORTED
