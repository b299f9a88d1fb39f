"""Which kernels a size of the products chosen by the row takes: the library's own
host-side choice (csrc/gfr_layer.h: grouped_kernel, lora_layout), called by its C++
symbols."""
import ctypes

import mxfp8_grouped_gemm_group_amd as gfr


class _Choice(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("split", ctypes.c_int32)]


class _Lora(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("codes", "dense", "total")] + [
        ("tiles", ctypes.c_int32), ("choice", _Choice)]


def lora(M, N, K, r):
    """Whether lora_linear takes whole tiles."""
    f = gfr.load_library()._ZN3gfr11lora_layoutEllll
    f.restype, f.argtypes = _Lora, [ctypes.c_int64] * 4
    return bool(f(M, N, K, r).tiles)


def grouped(M, E, K, N, wgrad=False, transpose=False, long=False):
    """"direct", "128" or "64" (`long`: "64 long" for its form of four groups of waves)."""
    f = gfr.load_library()._ZN3gfr14grouped_kernelEiillll
    f.restype, f.argtypes = ctypes.c_int32, [ctypes.c_int] * 2 + [ctypes.c_int64] * 4
    return ("direct", "128", "64", "64 long" if long else "64")[f(int(wgrad), int(transpose), M, E, K, N)]
