"""What the exactly summed inputs of exact_inputs notice, on the CPU: mistakes
planted in their float64 result."""
import numpy as np
import pytest
import torch

from oracle import layer

from . import exact_inputs


def bf16(v):
    return torch.from_numpy(v).float().bfloat16().double().numpy()


def two_terms(h):
    return bf16(h) + bf16(h - bf16(h))


DECODE = [(1, 2, 4, 128, 512, 512, 1), (5, 2, 3, 4160, 448, 1344, 1), (40, 2, 3, 128, 128, 64, 2)]


@pytest.mark.parametrize("T, k, E, H, I, N, spread", DECODE)
def test_decode_notices_silu_times_up_in_fewer_bits(T, k, E, H, I, N, spread):
    _, want, p = exact_inputs.decode_case(T, k, E, H, I, N, spread=spread)
    for h_of in (bf16, two_terms):
        got, _, _ = exact_inputs.decode_expected(p["x"], p["w13"], p["w2"], p["ids"],
                                                 p["weights"], h_of)
        assert (got != want).mean() > 0.25
    h = np.abs(p["h"][p["h"] != 0])
    assert np.log2(h).max() >= 17


@pytest.mark.parametrize("T, k, E, H, I, N, spread", DECODE + [(16, 8, 64, 768, 512, 64, 8)])
def test_decode_notices_a_lost_step(T, k, E, H, I, N, spread):
    """64 rows of H lost change nearly every result; 64 rows of I those of the columns
    that have one of these rows in any of the token's experts."""
    _, want, p = exact_inputs.decode_case(T, k, E, H, I, N, spread=spread)
    for first in (0, (H // 64 // 2) * 64, H - 64):
        x = p["x"].copy()
        lost = np.zeros_like(x)
        big = int(np.flatnonzero((x == 64).all(0))[0])
        lost[:, first:first + 64] = x[:, first:first + 64]
        lost[:, big] = 0                              # (the gate's base stays)
        got, _, _ = exact_inputs.decode_expected(x - lost, p["w13"], p["w2"], p["ids"],
                                                 p["weights"])
        assert (got != want).mean() > 0.9
    for first in (0, (I // 64 // 2) * 64, I - 64):
        w2 = p["w2"].copy()
        w2[:, first:first + 64] = 0
        hit = np.stack([(w2[e] != p["w2"][e]).any(0) for e in p["ids"].reshape(-1)])
        hit = hit.reshape(T, k, N).any(1)
        got, _, _ = exact_inputs.decode_expected(p["x"], p["w13"], w2, p["ids"], p["weights"])
        assert hit.any() and (got != want)[hit].mean() > 0.9


@pytest.mark.parametrize("act", ["none", "relu", "swiglu"])
@pytest.mark.parametrize("M, N, K", [(4, 64, 28672), (100, 64, 28680), (65, 75, 4107),
                                     (130, 40, 520), (5, 33, 131)])
def test_linear_notices_a_lost_step_or_tail(M, N, K, act):
    _, want, p = exact_inputs.linear_case(M, N, K, act, bias=torch.float32, residual=True)
    p = dict(p)
    x, tail = p.pop("x"), K % 64 or 64
    keep = (x == 64).all(0) if act == "swiglu" else np.zeros(K, bool)
    for first, n in ((0, 64), (K // 128 * 64, 64), (K - tail, tail)):
        lost = x.copy()
        lost[:, first:first + n] = 0
        lost[:, keep] = x[:, keep]
        got = exact_inputs.linear_expected(lost, **p)
        live = want != p["r"] if act == "relu" else np.ones_like(want, bool)
        assert (got != want)[live].mean() > 0.8


@pytest.mark.parametrize("M, N, K", [(4, 64, 28672), (100, 64, 28680), (65, 75, 4107)])
def test_linear_notices_sums_in_16_bits(M, N, K):
    _, want, p = exact_inputs.linear_case(M, N, K)
    half = K // 128 * 64
    a, b = (bf16(p["x"][:, s] @ p["w"][:, s].T) for s in (slice(0, half), slice(half, K)))
    assert (a + b != want).mean() > 0.25


def test_decode_bound_covers_a_sum_per_64_rows():
    """The bound of joining covers as many pieces as a product may come in: here each
    of 64 rows of I, added in FP32 one after the other, the largest sums first."""
    rng = np.random.default_rng(5)
    k, I, N = 8, 4096, 16
    x = np.full((1, 64), 1.0)
    w13 = np.zeros((1, 64, 2 * I))
    w13[:, 0, :I] = 64.0                              # silu(64) = 64 to 1e-26
    w13[:, 0, I:] = 1.0
    w2 = rng.standard_normal((1, I, N))
    ids, weights = np.zeros((1, k), np.int64), np.ones((1, k))
    want, bound = layer.moe_decode(x, w13, w2, ids, weights)
    pieces = np.float32((64.0 * w2[0]).reshape(-1, 64, N).sum(1))
    total = np.zeros(N, np.float32)
    for piece in sorted(np.repeat(pieces, k, 0), key=lambda v: -np.abs(v).max()):
        total = total + piece
    assert (np.abs(total - want[0]) <= bound[0]).all()
    # what is charged beyond the products' own sums is at least a rounding per piece
    mag = k * 64.0 * np.abs(w2[0]).sum(0)
    assert (bound[0] >= (3 * I + k * I // 64) * layer.ULP * mag).all()
