"""gfr.moe_route's weights where no bias or runs take part: computed in FP64 and
rounded once, so within half an FP32 step of the float64 oracle's (2^-24 of the
value; 2^-44 beside it for the FP64 evaluation's own few units of 2^-53 and the
oracle's)."""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
REL = 2.0 ** -24 + 2.0 ** -44


def check(z, k, with_x, **kw):
    print(tuple(z.shape), k, with_x, kw, flush=True)
    x = torch.ones(z.shape[0], 32).bfloat16().to(DEV) if with_x else None
    r = gfr.moe_route(z.to(DEV), k, x=x, **kw)
    torch.cuda.synchronize()
    ids, w = layer.moe_route(z.double().numpy(), k, **kw)
    assert np.array_equal(r.topk_ids.cpu().numpy(), ids)
    got = r.topk_weights.double().cpu().numpy()
    err = np.abs(got - w) / np.maximum(np.abs(w), 2.0 ** -126)
    assert err.max() <= REL, f"{err.max() / REL:.3g} of the tolerance"


ROUTERS = [dict(scoring=s, renormalize=r, scaling=c)
           for s in ("softmax", "sigmoid") for r in (True, False) for c in (1.0, 2.5)]


@pytest.mark.parametrize("kw", ROUTERS)
@pytest.mark.parametrize("with_x", [False, True])
@pytest.mark.parametrize("T, E, k", [(1, 8, 2), (16, 60, 4), (5, 128, 8), (70, 256, 8),
                                     (33, 384, 6), (7, 1024, 32)])
def test_weights_are_rounded_once(T, E, k, with_x, kw):
    z = 2 * torch.randn(T, E, generator=torch.Generator().manual_seed(T + E + k))
    check(z, k, with_x, **kw)


@pytest.mark.parametrize("kw", ROUTERS)
@pytest.mark.parametrize("base", [-80.0, 0.0, 30.0])
def test_choices_far_below_the_largest(base, kw):
    """Logits tens apart: the rounding of their FP32 difference alone would change
    the smaller weights by some 2^-19."""
    g = torch.Generator().manual_seed(3)
    z = base - 11.0 * torch.rand(12, 16, generator=g) * torch.arange(16)
    z = z[:, torch.randperm(16, generator=g)].clamp_min(base - 60)
    z = z + 0.01 * torch.randn(12, 16, generator=g)
    if kw["scoring"] == "sigmoid" and not kw["renormalize"]:
        z = z.clamp_min(-60)             # (weights above FP32's smallest normal)
        z = z - 0.001 * torch.arange(16)
    check(z, 6, False, **kw)
