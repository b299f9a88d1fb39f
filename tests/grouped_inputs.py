"""Groups and inputs of the 16-bit grouped products, and their definitions in 64 bits.

Integer inputs: every product and every sum of magnitudes stays below 2^24, so that
FP32 holds any order of summation exactly and results are equal, or, in 16 bits, the
exact value rounded once.
"""
import torch

LIMIT = 2 ** 24


def ranges(group_list, group_list_type, M):
    """[(first, end)] of each expert as the library reads a list (bad ones clamped)."""
    out, run, last = [], 0, 0
    for g in group_list:
        count = g if group_list_type == 1 else g - last
        last = g
        count = min(max(count, 0), M)
        out.append((min(run, M), min(run + count, M)))
        run += count
    return out


def as_list(counts, group_list_type):
    if group_list_type == 1:
        return list(counts)
    out, run = [], 0
    for c in counts:
        run += c
        out.append(run)
    return out


def integers(counts, M, K, N, dtype, transpose=False, seed=0):
    """x [M, K], w, dy [M, N] on the CPU."""
    g = torch.Generator().manual_seed(seed + 7919 * M + 31 * N + K)
    draw = lambda high, *s: torch.randint(-high, high + 1, s, generator=g, dtype=torch.int8)
    small = 8 if max(K, N, M) <= 512 else 4
    E = len(counts)
    x, dy = draw(small, M, K), draw(small, M, N)
    w = draw(4, E, *((N, K) if transpose else (K, N)))
    assert small * small * max(K, N, M) < LIMIT
    return x.to(dtype), w.to(dtype), dy.to(dtype)


def forward(x, w, rng, transpose, rest=0.0):
    """float64 [M, N]; rows of no expert hold ``rest``."""
    x, w = x.double(), w.double()
    out = torch.full((x.shape[0], w.shape[1 if transpose else 2]), rest, dtype=torch.float64)
    for e, (a, b) in enumerate(rng):
        out[a:b] = x[a:b] @ (w[e].T if transpose else w[e])
    return out


def wgrad(x, dy, rng, transpose):
    x, dy = x.double(), dy.double()
    g = torch.stack([x[a:b].T @ dy[a:b] for a, b in rng])
    return g.transpose(1, 2).contiguous() if transpose else g
