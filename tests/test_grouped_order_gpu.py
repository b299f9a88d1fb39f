"""grouped_linear_wgrad: M, E, K, N and a range's own rows fix its bits, in every kernel."""
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from tests import dispatch_rows
from tests.test_grouped_linear_gpu import BF, DEV, F32, groups

# (kernel, K, N, two lists of the same rows with the same first and third range)
CASES = [("direct", 1032, 1544, [400, 900, 300, 400], [400, 900, 300, 0]),
         ("64", 264, 520, [130, 70, 200, 100], [130, 70, 200, 99]),
         ("64 long", 136, 264, [1500, 2000, 1600, 900], [1500, 2000, 1600, 0]),
         ("128", 1097, 2056, [700, 500, 600, 201], [700, 500, 600, 200])]


def sizes(one):
    return sum(one), len(one)


def test_the_cases_take_their_kernels():
    for kernel, K, N, one, two in CASES:
        M, E = sizes(one)
        assert dispatch_rows.grouped(M, E, K, N, True, long=True) == kernel, (kernel, K, N)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel, K, N, one, two", CASES)
def test_a_range_keeps_its_bits_whatever_the_others(kernel, K, N, one, two):
    M, _ = sizes(one)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(M, K, generator=g).to(BF).to(DEV)
    dy = torch.randn(M, N, generator=g).to(BF).to(DEV)
    call = lambda counts, a=x, b=dy: gfr.grouped_linear_wgrad(a, b, groups(counts, 1), 1,
                                                              out_dtype=F32)
    first, second = call(one), call(two)
    torch.cuda.synchronize()
    assert torch.equal(first[:3], second[:3])
    # the first range's rows at another place, behind those of another expert
    n, shift = one[0], one[1]
    order = torch.cat([torch.arange(n, n + shift), torch.arange(n), torch.arange(n + shift, M)])
    moved = call([one[1], one[0], *one[2:]], x[order.to(DEV)], dy[order.to(DEV)])
    torch.cuda.synchronize()
    assert torch.equal(first[0], moved[1]) and torch.equal(first[1], moved[0])
