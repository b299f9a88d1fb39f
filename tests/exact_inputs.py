"""Inputs of the dense product and of the experts for a few tokens whose results
FP32 holds exactly, in any order of summation: small integers with every sum of
magnitudes below 2^24.  A lost K step or tail, a partial sum or a factor held in
fewer bits then changes the result, where a bound of what rounding may do over K
additions would let it pass.
"""
import numpy as np
import torch

LIMIT = 2 ** 24
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def decode_case(T, k, E, H, I, N, fp8="e4m3", t13=False, t2=False, per_expert=False, spread=1,
                seed=0):
    """Arguments of moe_decode (CPU tensors) and the exact result, float64 [T, N].

    gate = 1024 or more plus a sum of small integers: exp(-gate) is nothing beside 1
    in FP32, silu(gate) = gate.  up: a sum of small integers.  gate * up takes 18 to
    23 bits.  Each column of w2 has `spread` rows of an expert, 1 or -1, all rows
    taken in turn; weights of pairs are 1, -1 and 2.  Scales are powers of two whose
    products with the codes are these integers.
    """
    rng = np.random.default_rng(seed + 1000 * T + 10 * E + H + I + N)
    # up's magnitude stays near 2^9 as H grows
    small = 4 if H <= 512 else 2 if H <= 2048 else 1
    x = rng.integers(-small, small + 1, (T, H)).astype(np.float64)
    x[:, rng.integers(H)] = 64
    big = int(np.argmax(x[0] == 64))
    w13 = rng.integers(-4, 5, (E, H, 2 * I)).astype(np.float64)
    w13[:, :, :I] = np.sign(w13[:, :, :I])
    w13[:, big, :I] = 64
    w13[:, big, I:] = 0
    w2 = np.zeros((E, I, N))
    for e in range(E):
        rows = np.concatenate([rng.permutation(I) for _ in range(-(-spread * N // I))])
        cols = np.repeat(np.arange(N), spread)
        w2[e, rows[:spread * N], cols] = rng.choice([-1.0, 1.0], spread * N)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    weights = rng.choice([1.0, -1.0, 2.0], (T, k))
    out, mag, h_all = expected(x, w13, w2, ids, weights)
    assert mag.max() < LIMIT, mag.max()

    dt = FP8[fp8]

    def parts(w, transpose):
        """codes, scales: value = code * 2^(scale - 127), the factor differing by block."""
        kk, n = w.shape[1:]
        s = rng.integers(-2, 1, ((E,) if per_expert else (1,)) + (kk // 32, n))
        codes = w * 2.0 ** -np.repeat(s, 32, axis=1)
        s = (s + 127).reshape(s.shape[0], kk // 64, 2, n)
        s = s.transpose(0, 3, 1, 2) if transpose else s.transpose(0, 1, 3, 2)
        codes = codes.transpose(0, 2, 1) if transpose else codes
        c = torch.from_numpy(np.ascontiguousarray(codes)).to(dt)
        assert np.array_equal(c.double().numpy(), codes)
        s = torch.from_numpy(np.ascontiguousarray(s).astype(np.uint8))
        return c, s if per_expert else s[0].contiguous()

    w13_c, s13 = parts(w13, t13)
    w2_c, s2 = parts(w2, t2)
    args = dict(x=torch.from_numpy(x).bfloat16(), w13=w13_c, scale13=s13, w2=w2_c, scale2=s2,
                topk_ids=torch.from_numpy(ids), topk_weights=torch.from_numpy(weights).float(),
                transpose_w13=t13, transpose_w2=t2)
    assert np.array_equal(args["x"].double().numpy(), x)
    plain = dict(x=x, w13=w13, w2=w2, ids=ids, weights=weights, h=h_all)
    return args, out, plain


def expected(x, w13, w2, ids, weights, h_of=lambda h: h):
    """(out, sum of magnitudes, every pair's silu(gate) * up).  h_of: what becomes of
    silu(gate) * up on its way."""
    T, k = ids.shape
    I, N = w2.shape[1:]
    out, mag, h_all = np.zeros((T, N)), np.zeros((T, N)), np.zeros((T, k, I))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            gu = x[t] @ w13[e]
            assert np.abs(x[t]) @ np.abs(w13[e]).max(1) < LIMIT and gu[:I].min() >= 32
            h = h_all[t, j] = h_of(gu[:I] * gu[I:])
            assert np.abs(h).max() < LIMIT
            out[t] += weights[t, j] * (h @ w2[e])
            mag[t] += abs(weights[t, j]) * (np.abs(h) @ np.abs(w2[e]))
    return out, mag, h_all
