"""The GPU tests' sizes still take the kernels they are there for, and between them
take every kernel: on the CPU, from the library's own choice."""
import pytest

from . import dispatch
from . import test_linear_exact_gpu as linear_cases
from . import test_moe_decode_exact_gpu as decode_cases


@pytest.mark.parametrize("M, N, K, act, kernel, split", linear_cases.CASES)
def test_linear_case_takes_its_kernel(M, N, K, act, kernel, split):
    got, pieces = dispatch.linear(M, N, K, act == "swiglu")
    assert (got, pieces > 1) == (kernel, split)


def test_linear_cases_take_every_kernel():
    """Rows by their fragments, tiles by their split, each with K aligned and not, with
    gate * up and without; rows of out whole 16 bytes and not.  (Tiles of 256 rows
    take aligned K alone and do not split.)"""
    def variant(M, K, act, kernel, split):
        rows = 0 if kernel != "rows" else 1 if M <= 16 else 2 if M <= 32 else 4
        return kernel, rows, split, K % 8 == 0, act == "swiglu"
    got = {variant(M, K, act, kernel, split)
           for M, N, K, act, kernel, split in linear_cases.CASES}
    want = {("rows", r, False, a, s) for r in (1, 2, 4) for a in (False, True)
            for s in (False, True)}
    want |= {(t, 0, p, a, s) for t in ("64x64", "128x128") for p in (False, True)
             for a in (False, True) for s in (False, True)}
    want |= {(t, 0, False, True, s) for t in ("256x128", "256x256") for s in (False, True)}
    assert got == want
    wide = {(kernel, split, act == "swiglu", N % 8 == 0)
            for M, N, K, act, kernel, split in linear_cases.CASES}
    for kernel in dispatch.KERNELS:
        for split in ((False, True) if kernel in ("64x64", "128x128") else (False,)):
            for s in (False, True):
                for w in (False, True):
                    assert (kernel, split, s, w) in wide, (kernel, split, s, w)


def shape(part):
    return part.waves, part.shared, int(part.run > 1)


@pytest.mark.parametrize("t, case", [(t, c) for t, cases in ((False, decode_cases.KN),
                                                             (True, decode_cases.NK))
                                     for c in cases])
def test_decode_case_takes_its_variant(t, case):
    *sizes, gate_up, down = case
    d = dispatch.decode(*sizes, t, t)
    assert (shape(d.gate_up), shape(d.down)) == (gate_up, down)


def test_decode_cases_take_every_variant():
    """Each product with one and two fragments of pairs, four and eight waves, a wave
    with one tile and with several, and (for [K, N] and one fragment) shared tiles;
    h formed ahead of the down product and by its blocks."""
    for t, cases in ((False, decode_cases.KN), (True, decode_cases.NK)):
        got, ahead = set(), set()
        for *sizes, gate_up, down in cases:
            d = dispatch.decode(*sizes, t, t)
            got |= {("gate_up", d.row_fragments) + gate_up, ("down", d.row_fragments) + down}
            ahead.add(d.activate)
        want = {(p, r, w, 0) for p in ("gate_up", "down") for r in (1, 2) for w in (4, 8)}
        want |= set() if t else {(p, 1, 4, 1) for p in ("gate_up", "down")}
        assert {g[:4] for g in got} == want
        assert {p for p, *_, runs in got if runs} == {"gate_up", "down"}
        assert ahead == {0, 1}
