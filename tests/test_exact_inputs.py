"""What the exactly summed inputs of exact_inputs notice, on the CPU: mistakes
planted in their float64 result."""
import numpy as np
import pytest
import torch

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
