"""Which kernel a size takes: the library's own host-side choice (csrc/gfr_layer.h:
linear_choice, decode_layout), called by its C++ symbols.  Tests of a variant assert
by it that their sizes still reach that variant."""
import ctypes

import mxfp8_grouped_gemm_group_amd as gfr

KERNELS = ("rows", "256x256", "256x128", "128x128", "64x64")
SWIGLU = 5


class _Choice(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("split", ctypes.c_int32)]


class _Part(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("chunks", "run", "waves", "shared")]


class _Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("gu", "y", "h", "total")] + [
        ("activate", ctypes.c_int32), ("row_fragments", ctypes.c_int32),
        ("gate_up", _Part), ("down", _Part)]


def linear(M, N, K, swiglu=False):
    """(kernel, K split)."""
    f = gfr.load_library()._ZN3gfr13linear_choiceEllli
    f.restype, f.argtypes = _Choice, [ctypes.c_int64] * 3 + [ctypes.c_int]
    c = f(M, N, K, SWIGLU if swiglu else 0)
    return KERNELS[c.kernel], c.split


def decode(T, k, E, H, I, N, t13=False, t2=False):
    """The layout: activate, row_fragments, and chunks, run, waves and shared of the
    gate_up and down products."""
    f = gfr.load_library()._ZN3gfr13decode_layoutEllllllii
    f.restype, f.argtypes = _Layout, [ctypes.c_int64] * 6 + [ctypes.c_int] * 2
    return f(T, k, E, H, I, N, int(t13), int(t2))
