"""GPU parity of gfr.moe_decode against the float64 oracle
(oracle.layer.moe_decode).

Tolerance: the oracle's bound (FP32 sums of H and I products, silu's slope,
silu(gate) * up kept to 2^-16, one rounding per added pair) plus half a step of
out's type.
"""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_group_amd as gfr
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
FP8 = {"e4m3": (torch.float8_e4m3fn, 0), "e5m2": (torch.float8_e5m2, 1)}
FORMATS = {torch.bfloat16: (7, -126), torch.float32: (23, -126)}


def make(T, k, E, H, I, N, fp8="e4m3", t13=False, t2=False, per_expert=False, shared=False,
         seed=0):
    dt, kind = FP8[fp8]
    g = torch.Generator().manual_seed(seed + 101 * T + 7 * E + H + I + N)
    rng = np.random.default_rng(seed + T)
    code = lambda *s: torch.randn(*s, generator=g).to(dt)
    lead = (E,) if per_expert else ()
    scale = lambda *s: torch.from_numpy(rng.integers(119, 125, lead + s, dtype=np.uint8))
    a = dict(
        x=torch.randn(T, H, generator=g).bfloat16(),
        w13=code(E, 2 * I, H) if t13 else code(E, H, 2 * I),
        scale13=scale(2 * I, H // 64, 2) if t13 else scale(H // 64, 2 * I, 2),
        w2=code(E, N, I) if t2 else code(E, I, N),
        scale2=scale(N, I // 64, 2) if t2 else scale(I // 64, N, 2),
        topk_ids=torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int(),
        topk_weights=torch.rand(T, k, generator=g) + 0.1,
        shared_input=torch.randn(T, N, generator=g).bfloat16() if shared else None)
    a = {n: None if v is None else v.to(DEV) for n, v in a.items()}
    a.update(transpose_w13=t13, transpose_w2=t2, shared_input_weight=0.75, kind=kind)
    return a


def call(a, **kw):
    return gfr.moe_decode(a["x"], a["w13"], a["scale13"], a["w2"], a["scale2"], a["topk_ids"],
                          a["topk_weights"], transpose_w13=a["transpose_w13"],
                          transpose_w2=a["transpose_w2"], shared_input=a["shared_input"],
                          shared_input_weight=a["shared_input_weight"], **kw)


def oracle(a):
    u8 = lambda t: t.contiguous().view(torch.uint8).cpu().numpy()
    w13 = layer.mx_weights(u8(a["w13"]), u8(a["scale13"]), a["transpose_w13"], a["kind"])
    w2 = layer.mx_weights(u8(a["w2"]), u8(a["scale2"]), a["transpose_w2"], a["kind"])
    sh = a["shared_input"]
    return layer.moe_decode(a["x"].double().cpu().numpy(), w13, w2, a["topk_ids"].cpu().numpy(),
                            a["topk_weights"].double().cpu().numpy(),
                            None if sh is None else sh.double().cpu().numpy(),
                            a["shared_input_weight"])


def check(a, out, what):
    want, bound = oracle(a)
    tol = bound + layer.half_step(np.abs(want) + bound, *FORMATS[out.dtype])
    err = np.abs(out.double().cpu().numpy() - want)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, worst "
                           f"{np.nanmax(err / tol):.3g} of the tolerance at "
                           f"{np.argwhere(bad)[:3].tolist()}")


@pytest.mark.parametrize("t13, t2", [(False, False), (True, True), (True, False), (False, True)])
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("T, k, E, H, I, N", [
    (1, 1, 1, 64, 64, 64), (1, 4, 8, 256, 128, 192), (3, 2, 4, 192, 320, 128),
    (16, 2, 4, 128, 64, 320), (17, 3, 5, 320, 192, 64), (33, 4, 4, 128, 192, 256),
    (64, 2, 2, 64, 128, 128), (64, 6, 64, 128, 64, 64)])
def test_sizes(T, k, E, H, I, N, t13, t2, fp8):
    what = f"T {T} k {k} E {E} H {H} I {I} N {N} {fp8} {t13} {t2}"
    print(what, flush=True)
    a = make(T, k, E, H, I, N, fp8, t13, t2, per_expert=T % 2 == 1, shared=T > 2)
    out = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    check(a, out, what)


@pytest.mark.parametrize("t", [False, True])
def test_bf16_out_and_wide_layers(t):
    a = make(5, 2, 6, 1024, 768, 512, "e4m3", t, t, per_expert=True, shared=True)
    out = call(a)
    torch.cuda.synchronize()
    assert out.dtype == torch.bfloat16
    check(a, out, "wide")


# many blocks of many rows: blocks of eight waves and runs of several tiles, of
# the gate/up product (wide I) and the down product (wide N)
@pytest.mark.parametrize("T, k, E, H, I, N, t", [
    (60, 6, 64, 128, 3200, 64, False), (60, 6, 64, 64, 128, 6400, False),
    (60, 6, 64, 128, 3200, 64, True), (60, 6, 64, 64, 128, 3328, True),
    (64, 10, 64, 64, 3648, 64, False), (64, 10, 64, 64, 128, 3648, False),
    (64, 10, 64, 128, 1600, 64, True), (64, 10, 64, 64, 192, 1856, True),
    (64, 10, 64, 64, 192, 3264, True)])
def test_many_blocks(T, k, E, H, I, N, t):
    what = f"T {T} k {k} E {E} H {H} I {I} N {N} {t}"
    print(what, flush=True)
    a = make(T, k, E, H, I, N, "e4m3", t, t, shared=True)
    a["topk_ids"][3] = -1
    out = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    check(a, out, what)


# few blocks: the waves of a block share a column tile, with steps left over
@pytest.mark.parametrize("T, k, E, H, I, N", [(1, 2, 8, 1088, 704, 192), (2, 3, 5, 4160, 448, 1344),
                                              (16, 1, 2, 576, 832, 320)])
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
def test_few_blocks(T, k, E, H, I, N, fp8):
    print(f"T {T} k {k} E {E} H {H} I {I} N {N} {fp8}", flush=True)
    a = make(T, k, E, H, I, N, fp8, per_expert=True, shared=True)
    out = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    check(a, out, "few blocks")


def test_most_experts_and_pairs():
    a = make(64, 16, 1024, 64, 64, 64, "e5m2")
    out = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    check(a, out, "1024 experts, 1024 pairs")
    a = make(32, 32, 32, 64, 64, 128, "e4m3", True, True)
    out = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    check(a, out, "32 of 32 experts")


@pytest.mark.parametrize("t", [False, True])
def test_padded_rows_and_no_expert_at_all(t):
    a = make(9, 3, 4, 128, 64, 192, "e4m3", t, t, shared=True)
    a["topk_ids"][6:] = -1
    a["topk_ids"][1, 2] = -1
    a["topk_weights"][6:] = float("nan")        # weights of no expert are not read
    out = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    b = dict(a, topk_weights=torch.nan_to_num(a["topk_weights"]))
    check(b, out, "padded")
    assert torch.equal(out[6:], 0.75 * a["shared_input"][6:].float())
    a["topk_ids"].fill_(-1)
    out = call(a, out_dtype=torch.float32)
    assert torch.equal(out, 0.75 * a["shared_input"].float())
    a["shared_input"] = None
    out = call(a, out=torch.full((9, 192), 7.0, dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    assert (out == 0).all()


def test_an_expert_named_twice_and_one_expert_for_all():
    a = make(40, 2, 3, 128, 128, 64)
    a["topk_ids"].fill_(1)                      # 80 pairs of one expert: several groups
    out = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    check(a, out, "one expert")


def test_bad_ids_are_skipped_and_flagged():
    a = make(7, 2, 4, 64, 64, 64)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    a["topk_ids"][3, 1] = -1
    call(a, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    a["topk_ids"][0, 0], a["topk_ids"][5, 1] = 4, -2
    out = call(a, out_dtype=torch.float32, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == gfr.DEV_BAD_EXPERT
    check(a, out, "bad ids")


def test_extreme_scales_and_nan_stay_in_their_column():
    a = make(2, 1, 2, 64, 64, 64, "e4m3")
    a["topk_ids"].zero_()
    want = call(a, out_dtype=torch.float32)
    a["scale2"][0, 5, 1] = 255                  # E8M0's NaN: column 5
    got = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.isnan(got[:, 5]).all()
    keep = [n for n in range(64) if n != 5]
    assert torch.equal(got[:, keep], want[:, keep])
    a["scale2"][0, 5, 1] = 254                  # 2^127: infinite or NaN sums, this column's
    got = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(got[:, keep], want[:, keep])
    a["scale2"][0, 5, :] = 0                    # 2^-127
    got = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert (got[:, 5].abs() < 1e-30).all() and torch.equal(got[:, keep], want[:, keep])


def test_nan_token_reaches_no_other_token():
    a = make(20, 2, 3, 128, 64, 128)
    want = call(a, out_dtype=torch.float32)
    a["x"][4, 100] = float("nan")
    a["x"][11, 0] = float("inf")
    got = call(a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    rest = [t for t in range(20) if t not in (4, 11)]
    assert torch.equal(got[rest], want[rest]) and torch.isnan(got[4]).all()


@pytest.mark.parametrize("t", [False, True])
def test_same_bits_twice_and_used_workspace(t):
    a = make(12, 4, 8, 256, 512, 256, "e5m2", t, t, shared=True)
    need = gfr.moe_decode_workspace_size(12, 4, 8, 256, 512, 256, t, t)
    ws = torch.randint(0, 256, (need + 256,), dtype=torch.uint8, device=DEV)
    one = call(a, workspace=ws[:need])
    guard = ws[need:].clone()
    two = call(a, workspace=ws[:need])
    three = call(a)
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(one, three)
    assert torch.equal(ws[need:], guard)
    with pytest.raises(gfr.GfrError):
        call(a, workspace=ws[:need - 1])
