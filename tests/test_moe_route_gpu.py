"""GPU parity of gfr.moe_route against the float64 oracle (oracle.layer).

Ids, counts, order, codes and scale bytes have to be equal.  Weights: the
scores and their sum are FP32 or better with expf's few units in the last
place, so 2^-20 relative.
"""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from oracle import gemm1, layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
REL = 2.0 ** -20


def make(T, E, dtype=torch.float32, bias=False, seed=0, masked=0.0):
    g = torch.Generator().manual_seed(seed + 13 * T + E)
    z = 2 * torch.randn(T, E, generator=g)
    if masked:
        z = z.masked_fill(torch.rand(T, E, generator=g) < masked, -float("inf"))
    return (z.to(dtype).to(DEV),
            (0.2 * torch.randn(E, generator=g)).to(DEV) if bias else None)


def check_choice(r, logits, k, bias, **kw):
    ids, w = layer.moe_route(logits.double().cpu().numpy(), k,
                             None if bias is None else bias.double().cpu().numpy(), **kw)
    got, gw = r.topk_ids.cpu().numpy(), r.topk_weights.double().cpu().numpy()
    bad = np.argwhere(got != ids)
    assert bad.size == 0, f"{len(bad)} ids differ, first {bad[:3].tolist()}"
    assert (np.abs(gw - w) <= REL * np.abs(w)).all()
    return ids, w


def check_rows(r, x, ids, E, dtype):
    kind = 0 if dtype == torch.float8_e4m3fn else 1
    codes, scales, order, counts = layer.dispatched_rows(x.double().cpu().numpy(), ids, E, kind)
    assert np.array_equal(r.group_list.cpu().numpy(), counts)
    assert np.array_equal(r.row_index.cpu().numpy(), order // ids.shape[1])
    assert np.array_equal(r.logit.cpu().numpy(), r.topk_weights.cpu().numpy().reshape(-1)[order])
    assert np.array_equal(r.xin_scale.cpu().numpy(), scales)
    assert np.array_equal(r.xin.view(torch.uint8).cpu().numpy(), codes)


ROUTERS = [dict(), dict(scoring="sigmoid"), dict(renormalize=False, scaling=2.5),
           dict(scoring="sigmoid", renormalize=False),
           dict(n_group=4, topk_group=2), dict(scoring="sigmoid", n_group=2, topk_group=1)]


@pytest.mark.parametrize("kw", ROUTERS)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T, E, k", [(1, 8, 2), (5, 64, 6), (33, 60, 4), (40, 128, 8),
                                     (17, 256, 8), (9, 384, 5), (6, 1024, 32)])
def test_choice(T, E, k, bias, kw):
    print(f"T {T} E {E} k {k} bias {bias} {kw}", flush=True)
    for dtype in (torch.float32, torch.bfloat16):
        logits, b = make(T, E, dtype, bias)
        r = gfr.moe_route(logits, k, bias=b, **kw)
        torch.cuda.synchronize()
        assert r.xin is None and r.group_list is None
        check_choice(r, logits, k, b, **kw)


@pytest.mark.parametrize("fp8", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T, E, k, H", [
    (1, 8, 2, 32), (3, 16, 4, 96), (32, 24, 3, 128), (33, 24, 3, 1056), (64, 40, 5, 64),
    (65, 40, 5, 64), (100, 64, 6, 64),
    (49, 256, 8, 1024), (300, 7, 7, 160)])
def test_rows(T, E, k, H, xdt, fp8):
    print(f"T {T} E {E} k {k} H {H} {xdt} {fp8}", flush=True)
    logits, _ = make(T, E)
    x = (torch.randn(T, H) * torch.exp(2 * torch.randn(T, H))).to(xdt).to(DEV)
    x[0, :32] = 0
    r = gfr.moe_route(logits, k, x=x, out_dtype=fp8)
    torch.cuda.synchronize()
    ids, _ = check_choice(r, logits, k, None)
    check_rows(r, x, ids, E, fp8)


@pytest.mark.parametrize("T", [4, 64, 2500])
@pytest.mark.parametrize("kw", [dict(), dict(scoring="sigmoid", n_group=4, topk_group=2)])
def test_masked_experts_and_padded_tokens(T, kw):
    logits, b = make(T, 16, bias=True, masked=0.6)
    logits[T // 2] = -float("inf")
    logits[-1] = float("nan")
    logits[0, 3] = float("nan")
    b[5] = -float("inf")
    x = torch.randn(T, 64).bfloat16().to(DEV)
    r = gfr.moe_route(logits, 6, x=x, bias=b, **kw)
    torch.cuda.synchronize()
    ids, _ = check_choice(r, logits, 6, b, **kw)
    assert (ids[T // 2] == -1).all() and (ids[-1] == -1).all() and (ids < 0).any()
    check_rows(r, x, ids, 16, torch.float8_e4m3fn)


@pytest.mark.parametrize("E", [16, 256])
@pytest.mark.parametrize("shift", [-60.0, -95.0, -300.0, 95.0])
def test_far_logits_keep_their_weights(E, shift):
    """A row's scores may all be too small for FP32 (sigmoid of -95); their ratios
    are not."""
    logits, _ = make(6, E)
    logits = logits + shift
    for scoring in ("sigmoid", "softmax"):
        r = gfr.moe_route(logits, 4, scoring=scoring)
        torch.cuda.synchronize()
        check_choice(r, logits, 4, None, scoring=scoring)


def test_ties_go_to_the_lower_index():
    for E in (16, 64, 200, 256, 1000):
        for T in (2, 80):
            g = torch.Generator().manual_seed(E)
            logits = torch.randint(0, 3, (T, E), generator=g).float().to(DEV)
            logits[0] = 0
            n = 4 if E % 4 == 0 else 1
            for kw in (dict(), dict(scoring="sigmoid", n_group=n, topk_group=max(1, n // 2))):
                for b in (None, torch.zeros(E, device=DEV)):
                    r = gfr.moe_route(logits, 8, bias=b, **kw)
                    torch.cuda.synchronize()
                    check_choice(r, logits, 8, b, **kw)


def test_neighbouring_scores_are_told_apart():
    """Sigmoids that FP32 rounds to one value still differ in FP64."""
    E = 64
    z = torch.full((2, E), -3.0)
    z[:, 10], z[:, 50] = 17.0, 17.5          # 1 - 4.1e-8 and 1 - 2.5e-8
    logits = z.to(DEV)
    r = gfr.moe_route(logits, 2, scoring="sigmoid", bias=torch.zeros(E, device=DEV))
    torch.cuda.synchronize()
    assert r.topk_ids.tolist() == [[50, 10], [50, 10]]


def test_all_16_bit_values_quantise_as_the_oracle():
    """Every bf16 and f16 bit pattern but infinities, NaN and (where the product
    by a power of two is subnormal in FP32) none: codes and scales are equal."""
    for xdt in (torch.bfloat16, torch.float16):
        bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(xdt)
        x = torch.where(torch.isfinite(bits), bits, torch.zeros_like(bits))
        perm = torch.randperm(1 << 16, generator=torch.Generator().manual_seed(1))
        for order in (torch.arange(1 << 16), perm):
            xx = x[order].view(64, 1024).contiguous().to(DEV)
            logits = torch.zeros(64, 1, device=DEV)
            for fp8 in (torch.float8_e4m3fn, torch.float8_e5m2):
                r = gfr.moe_route(logits, 1, x=xx, out_dtype=fp8)
                torch.cuda.synchronize()
                check_rows(r, xx, np.zeros((64, 1), np.int32), 1, fp8)


def test_infinite_and_nan_elements():
    x = torch.randn(2, 64).bfloat16()
    x[0, 3], x[0, 40] = float("inf"), float("nan")
    x[1, 10] = -float("inf")
    r = gfr.moe_route(torch.zeros(2, 1, device=DEV), 1, x=x.to(DEV))
    torch.cuda.synchronize()
    q = r.xin.float().cpu()
    assert q[0, 3] == 448 and q[1, 10] == -448 and torch.isnan(q[0, 40])
    assert torch.isfinite(q[0, :40]).all() and torch.isfinite(q[1]).all()
    # the NaN does not enter its block's maximum
    want = x.clone()
    want[0, 40] = 0
    _, s, _ = gemm1.mx_quantize(want[:1, 32:].double().numpy(), 0)
    assert r.xin_scale[0, 0, 1].item() == s[0, 0, 0]


def test_infinite_logits():
    z = torch.randn(3, 8)
    z[1, 2] = float("inf")
    r = gfr.moe_route(z.to(DEV), 2)
    s = gfr.moe_route(z.to(DEV), 2, scoring="sigmoid")
    torch.cuda.synchronize()
    assert r.topk_ids[1, 0] == 2 and torch.isnan(r.topk_weights[1]).all()
    assert torch.isfinite(r.topk_weights[[0, 2]]).all()
    assert s.topk_ids[1, 0] == 2 and torch.isfinite(s.topk_weights).all()


def test_large_batch_over_many_experts():
    T, E, k, H = 5000, 256, 8, 96
    logits, b = make(T, E, bias=True)
    x = torch.randn(T, H).bfloat16().to(DEV)
    kw = dict(scoring="sigmoid", n_group=8, topk_group=4, scaling=2.5)
    r = gfr.moe_route(logits, k, x=x, bias=b, **kw)
    torch.cuda.synchronize()
    ids, _ = check_choice(r, logits, k, b, **kw)
    check_rows(r, x, ids, E, torch.float8_e4m3fn)


def test_one_expert_takes_all():
    T = 700
    logits = torch.zeros(T, 4, device=DEV)
    logits[:, 2] = 5
    x = torch.randn(T, 64).bfloat16().to(DEV)
    r = gfr.moe_route(logits, 1, x=x)
    torch.cuda.synchronize()
    assert r.group_list.tolist() == [0, 0, T, 0]
    check_rows(r, x, np.full((T, 1), 2, np.int32), 4, torch.float8_e4m3fn)


def test_no_tokens():
    r = gfr.moe_route(torch.empty(0, 8, device=DEV), 2,
                      x=torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    assert r.topk_ids.shape == (0, 2) and r.xin.shape == (0, 64)
    assert r.group_list.tolist() == [0] * 8
