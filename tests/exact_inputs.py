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


def _ints(rng, low, high, shape):
    return rng.integers(low, high + 1, shape, dtype=np.int8)


def linear_case(M, N, K, act="none", dtype=torch.bfloat16, bias=None, residual=False, seed=0):
    """Arguments of linear (CPU tensors) and the exact result, float64 [M, N].

    Small integers; with "swiglu" every gate is 32 or more (as decode_case's).
    """
    rng = np.random.default_rng(seed + 7919 * M + 31 * N + K)
    # sums stay below 2^11 or so as K grows, but above the 2^8 that bf16 holds
    small = 8 if K <= 256 else 4 if K <= 4500 and act != "swiglu" else 2
    x = _ints(rng, -small, small, (M, K)).astype(np.float64)
    rows = 2 * N if act == "swiglu" else N
    w = _ints(rng, -4, 4, (rows, K)).astype(np.float64)
    if act == "swiglu":
        big = int(rng.integers(K))
        x[:, big] = 64
        w[:N] = np.sign(w[:N])
        w[:N, big], w[N:, big] = 32, 0
    b = _ints(rng, -100, 100, rows).astype(np.float64) if bias is not None else None
    r = _ints(rng, -100, 100, (M, N)).astype(np.float64) if residual else None
    assert np.abs(x).max(0) @ np.abs(w).max(0) < LIMIT
    out = linear_expected(x, w, act, b, r)
    assert np.abs(out).max() < LIMIT
    t = lambda v, d: None if v is None else torch.from_numpy(v).to(d)
    args = dict(x=t(x, dtype), w=t(w, dtype), bias=t(b, bias), residual=t(r, dtype),
                activation=act)
    return args, out, dict(x=x, w=w, act=act, b=b, r=r)


def linear_expected(x, w, act, b, r):
    y = x @ w.T + (0.0 if b is None else b)
    if act == "swiglu":
        n = w.shape[0] // 2
        assert y[:, :n].min() >= 32
        y = y[:, :n] * y[:, n:]
        assert np.abs(y).max() < LIMIT
    elif act == "relu":
        y = np.maximum(y, 0.0)
    else:
        assert act == "none"
    return y if r is None else y + r


def decode_case(T, k, E, H, I, N, fp8="e4m3", t13=False, t2=False, per_expert=False, spread=1,
                seed=0):
    """Arguments of moe_decode (CPU tensors) and the exact result, float64 [T, N].

    gate = 512 or more plus a sum of small integers: exp(-gate) is nothing beside 1
    in FP32, silu(gate) = gate.  up: a sum of small integers.  gate * up takes up to
    23 bits.  Each column of w2 has `spread` rows of an expert, 1 or -1, all rows
    taken in turn; weights of pairs are 1, -1 and 2.  Scales are powers of two whose
    products with the codes are these integers.
    """
    rng = np.random.default_rng(seed + 1000 * T + 10 * E + H + I + N)
    # up's magnitude stays near 2^9 as H grows; many pairs' sums below 2^24
    small = 4 if H <= 512 and k < 8 else 2 if H <= 2048 and k < 16 else 1
    x = _ints(rng, -small, small, (T, H)).astype(np.float64)
    big = int(rng.integers(H))
    x[:, big] = 64
    w13 = _ints(rng, -4, 4, (E, H, 2 * I))
    np.sign(w13[:, :, :I], out=w13[:, :, :I])
    w13[:, big, :I] = 64 if k < 4 else 16 if k < 16 else 8
    w13[:, big, I:] = 0
    w2 = np.zeros((E, I, N), np.int8)
    cols = np.repeat(np.arange(N), spread)
    for e in range(E):
        rows = np.concatenate([rng.permutation(I) for _ in range(-(-spread * N // I))])
        w2[e, rows[:spread * N], cols] = rng.choice(np.array([-1, 1], np.int8), spread * N)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    weights = rng.choice([1.0, -1.0, 2.0], (T, k))
    out, mag, h = decode_expected(x, w13, w2, ids, weights)
    assert mag.max() < LIMIT, mag.max()

    def parts(w, transpose):
        """codes, scales: value = code * 2^(scale - 127), the factor differing by block."""
        kk, n = w.shape[1:]
        s = _ints(rng, -2, 0, ((E,) if per_expert else (1,)) + (kk // 32, n))
        codes = torch.empty((E, n, kk) if transpose else (E, kk, n), dtype=FP8[fp8])
        for e in range(E):
            f = np.repeat(np.float32(2.0) ** -s[e if per_expert else 0], 32, axis=0)
            v = torch.from_numpy(w[e] * f)
            v = v.t() if transpose else v
            codes[e] = v.to(FP8[fp8])
            assert torch.equal(codes[e].float(), v)
        s = (s.astype(np.int16) + 127).astype(np.uint8).reshape(s.shape[0], kk // 64, 2, n)
        s = s.transpose(0, 3, 1, 2) if transpose else s.transpose(0, 1, 3, 2)
        s = torch.from_numpy(np.ascontiguousarray(s))
        return codes, s if per_expert else s[0].contiguous()

    w13_c, s13 = parts(w13, t13)
    w2_c, s2 = parts(w2, t2)
    args = dict(x=torch.from_numpy(x).bfloat16(), w13=w13_c, scale13=s13, w2=w2_c, scale2=s2,
                topk_ids=torch.from_numpy(ids), topk_weights=torch.from_numpy(weights).float(),
                transpose_w13=t13, transpose_w2=t2)
    return args, out, dict(x=x, w13=w13, w2=w2, ids=ids, weights=weights, h=h)


def decode_expected(x, w13, w2, ids, weights, h_of=lambda h: h):
    """(out, sum of magnitudes, every pair's silu(gate) * up).  h_of: what becomes of
    silu(gate) * up on its way."""
    T, k = ids.shape
    I, N = w2.shape[1:]
    out, mag, h_all = np.zeros((T, N)), np.zeros((T, N)), np.zeros((T, k, I))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        w = w13[e].astype(np.float64)
        gu = x[t] @ w
        assert (np.abs(x[t]) @ np.abs(w)).max() < LIMIT and gu[:, :I].min() >= 32
        h = h_all[t, j] = h_of(gu[:, :I] * gu[:, I:])
        assert np.abs(h).max() < LIMIT
        w, wt = w2[e].astype(np.float64), weights[t, j][:, None]
        np.add.at(out, t, wt * (h @ w))
        np.add.at(mag, t, np.abs(wt) * (np.abs(h) @ np.abs(w)))
    return out, mag, h_all
