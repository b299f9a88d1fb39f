"""GPU parity of gfr.moe_route with rows for few tokens (one launch, a wave per token
in every block) over many experts, against the float64 oracle.

Ids, counts, order, codes and scale bytes have to be equal; weights within 2^-20
(test_moe_route_gpu's tolerance).
"""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("kw", [dict(), dict(scoring="sigmoid"),
                                dict(n_group=4, topk_group=2, renormalize=False),
                                dict(scoring="sigmoid", n_group=8, topk_group=3, scaling=2.5)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T, E, k, H", [(1, 128, 8, 96), (15, 128, 6, 64), (16, 256, 8, 1056),
                                        (2, 256, 8, 2048), (7, 384, 5, 64), (16, 384, 8, 32),
                                        (3, 1024, 32, 64), (16, 1024, 17, 160)])
def test_rows(T, E, k, H, bias, kw):
    print(f"T {T} E {E} k {k} H {H} bias {bias} {kw}", flush=True)
    g = torch.Generator().manual_seed(T + E + k + H)
    z = 2 * torch.randn(T, E, generator=g)
    z = z.masked_fill(torch.rand(T, E, generator=g) < 0.05, -float("inf"))
    b = 0.2 * torch.randn(E, generator=g) if bias else None
    x = torch.randn(T, H, generator=g).bfloat16()
    r = gfr.moe_route(z.to(DEV), k, x=x.to(DEV), bias=b.to(DEV) if bias else None, **kw)
    torch.cuda.synchronize()
    ids, w = layer.moe_route(z.numpy(), k, b.numpy() if bias else None, **kw)
    assert np.array_equal(r.topk_ids.cpu().numpy(), ids)
    got = r.topk_weights.cpu().numpy()
    assert (np.abs(got - w) <= 2.0 ** -20 * np.abs(w)).all()
    codes, scales, order, counts = layer.dispatched_rows(x.double().numpy(), ids, E, 0)
    assert np.array_equal(r.group_list.cpu().numpy(), counts)
    assert np.array_equal(r.row_index.cpu().numpy(), order // k)
    assert np.array_equal(r.logit.cpu().numpy(), got.reshape(-1)[order])
    assert np.array_equal(r.xin_scale.cpu().numpy(), scales)
    assert np.array_equal(r.xin.view(torch.uint8).cpu().numpy(), codes)
