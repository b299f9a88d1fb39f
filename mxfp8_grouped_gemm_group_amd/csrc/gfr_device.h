// Device helpers of the dense product, the few-token experts and the router.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gfr {
namespace {

typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

// Raw buffer over [base, base + bytes): the base and the step's offset live in
// scalar registers, a lane keeps one 32-bit offset.  Reads past the end give 0;
// the end is that of the last aligned word that holds a valid byte, so that a
// 16-bit element alone in it can be read as a word.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t buffer(const void *base, int64_t bytes) {
    const int n = bytes > 0x7ffffffc ? 0x7ffffffc : static_cast<int>((bytes + 3) & ~int64_t{3});
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, n, 0x00020000);
}
constexpr int kNt = 2;   // non-temporal: read-once data leaves the caches alone
template <int AUX>
__device__ __forceinline__ u4_t load16(rsrc_t r, int lane_off, int off) {
    return __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(r, lane_off, off, AUX));
}
template <int AUX>
__device__ __forceinline__ u2_t load8(rsrc_t r, int lane_off, int off) {
    return __builtin_bit_cast(u2_t, __builtin_amdgcn_raw_buffer_load_b64(r, lane_off, off, AUX));
}
__device__ __forceinline__ uint32_t load2(rsrc_t r, int lane_off, int off) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, lane_off, off, 0);
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <class T>
__device__ __forceinline__ T load(const void *p) {
    return *static_cast<const T *>(p);
}

__device__ __forceinline__ float bf16_f32(uint32_t bits) {
    return __uint_as_float(bits << 16);
}
// Two floats rounded to bf16 (to nearest, ties to even), first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf2_t v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const h2_t v = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

template <int CTRL, int ROWS, int BANKS, bool BOUND>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        static_cast<int>(old), static_cast<int>(x), CTRL, ROWS, BANKS, BOUND));
}

// a of lanes l % 16 >= 8 and b of the others trade places, across eight lanes: of
// 16 rows' 128-byte lines, loaded as a = rows 0-7 (lane (c, g): row c % 8, 16-byte
// piece g + 4 (c / 8)) and b = rows 8-15 likewise, lane (c, g) then holds pieces g
// (a) and 4 + g (b) of row c, the operands of two 16-row MFMAs.  Loading those as
// such would touch 16 half lines at a time.
__device__ __forceinline__ void swap_halves(u4_t &a, u4_t &b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t x = a[j], y = b[j];
        a[j] = dpp<0x128, 0xf, 0xc, false>(x, y);
        b[j] = dpp<0x128, 0xf, 0x3, false>(y, x);
    }
}

// Inclusive prefix sum over the 64 lanes: DPP row shifts, then the row totals
// broadcast into the rows behind them.
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
    uint32_t x = v + dpp<0x111, 0xf, 0xf, true>(0, v);
    x += dpp<0x112, 0xf, 0xf, true>(0, v);
    x += dpp<0x113, 0xf, 0xf, true>(0, v);
    x += dpp<0x114, 0xf, 0xe, false>(0, x);
    x += dpp<0x118, 0xf, 0xc, false>(0, x);
    x += dpp<0x142, 0xa, 0xf, false>(0, x);
    x += dpp<0x143, 0xc, 0xf, false>(0, x);
    return x;
}

// exp(v) to about two units in the last place: v_exp_f32 (2^t) of the rounded
// product t = v log2(e), times 1 + what the rounding left over.  Overflows to
// infinity and underflows to 0 as exp does; NaN stays NaN.
__device__ __forceinline__ float exp_f32(float v) {
    constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-8f;
    const float b = __builtin_amdgcn_fmed3f(v, -200.0f, 200.0f);   // finite, for the remainder
    const float r = fmaf(b, kLo, fmaf(b, kHi, -(b * kHi)));
    return __builtin_amdgcn_exp2f(v * kHi) * fmaf(r, 0.693147182464599609375f, 1.0f);
}
// v / (1 + exp(-v))
__device__ __forceinline__ float silu(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + exp_f32(-v));
}

// Lets kernel K have up to 146 KB of dynamic LDS; the runtime is asked once per
// device.
template <auto K>
hipError_t allow_lds(int bytes) {
    if (bytes <= (32 << 10)) return hipSuccess;
    static std::atomic<bool> done[64];
    int dev = 0;
    if (hipError_t e = hipGetDevice(&dev); e != hipSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed)) return hipSuccess;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(K),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, 146 << 10);
    if (e == hipSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

}  // namespace
}  // namespace gfr
