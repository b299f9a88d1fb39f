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
        got, _, _ = exact_inputs.expected(p["x"], p["w13"], p["w2"], p["ids"], p["weights"], h_of)
        assert (got != want).mean() > 0.25
    h = np.abs(p["h"][p["h"] != 0])
    assert np.log2(h).max() >= 17


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
