// Tiles of 16-bit operands in LDS and their MFMA fragments, shared by the products
// whose weight is chosen by the row (gfr_grouped.hip, gfr_lora.hip).
//
// An operand of a product is a set of lines (rows of x, columns of w) along a
// summed index k; a step takes 64 of k.  Two layouts, by which of the two is
// contiguous in memory:
//
//   k-major     a line's 64 k are eight 16-byte pieces, piece j of line r at
//               j ^ (r / 2 & 7): sixteen lanes that read one piece of sixteen lines
//               reach all 64 banks.  (j ^ (r & 7) reaches half of them: 137 of 280
//               thousand LDS clocks of 16384 x 4096 x 4096 were conflicts.)
//   line-major  of each k, BX lines in BX / 8 pieces, piece j at j ^ 4 (k & 3) (of 64
//               lines at j ^ 4 (k & 1)).  Fragments come through the transposing LDS read, which gives a
//               lane four k of one line; the 16 lanes that share it read 32 bytes
//               of four k, and two such groups reach all banks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gfr_device.h"

namespace gfr {
namespace {

typedef float f16_t __attribute__((ext_vector_type(16)));
typedef short s4_t __attribute__((ext_vector_type(4)));
typedef unsigned int v4i_t __attribute__((ext_vector_type(4)));

template <bool F16>
__device__ __forceinline__ f16_t mfma32(u4_t a, u4_t b, f16_t c) {
    if (F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8_t, a),
                                                      __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8_t, a),
                                                   __builtin_bit_cast(bf8_t, b), c, 0, 0, 0);
}

// Where piece j of line r (k-major) or of k (line-major, BX lines) lies, in pieces.
__device__ __forceinline__ int piece_k(int r, int j) { return r * 8 + (j ^ (r >> 1 & 7)); }
template <int BX>
__device__ __forceinline__ int piece_line(int k, int j) {
    return k * (BX / 8) + (j ^ (4 * (k & 3) & (BX / 8 - 1)));
}

// The fragment of lines [line, line + 32), k in [16 part, 16 part + 16): lane l
// gets line l % 32, k 8 (l / 32) .. + 7 of them.
template <bool LINE, int BX>
__device__ __forceinline__ u4_t fragment(const u4_t *tile, int line, int part, int lane) {
    if (!LINE) return tile[piece_k(line + (lane & 31), 2 * part + (lane >> 5))];
    typedef __attribute__((address_space(3))) s4_t *lds_t;
    const int q = lane >> 4, i = lane & 15;
    const int k = 16 * part + 8 * (q >> 1) + (i >> 2);
    const int col = line + 16 * (q & 1) + 4 * (i & 3);
    const char *at = reinterpret_cast<const char *>(tile) +
                     16 * piece_line<BX>(k, col >> 3) + 2 * (col & 7);
    const auto p = (lds_t)(const __attribute__((address_space(3))) char *)(at);
    const s4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
    const s4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + 4 * (BX / 4));
    const u2_t l2 = __builtin_bit_cast(u2_t, lo), h2 = __builtin_bit_cast(u2_t, hi);
    return u4_t{l2[0], l2[1], h2[0], h2[1]};
}

// Lane offset past every buffer's end: loads there give zeros, stores do nothing.
constexpr int kPast = 0x7f000000;

__device__ __forceinline__ void store16(rsrc_t r, u4_t v, int off) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i_t, v), r, off, 0, 0);
}
// A buffer that the compiler sees to be the same in all lanes.
__device__ __forceinline__ rsrc_t uniform_buffer(const char *base, int64_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    const uint32_t lo = uniform(static_cast<int>(at)), hi = uniform(static_cast<int>(at >> 32));
    const int n = bytes > 0x7ffffffc ? 0x7ffffffc : static_cast<int>(bytes);
    return __builtin_amdgcn_make_buffer_rsrc(
        reinterpret_cast<void *>(static_cast<uint64_t>(hi) << 32 | lo), 0, uniform(n), 0x00020000);
}

// Eight elements from byte `off` (even) on, of a buffer whose base is a whole
// word's address: 16 bytes at once where `whole` says that all pieces begin at
// multiples of 16, else the words that hold them, shifted into place.
__device__ __forceinline__ u4_t eight_of(rsrc_t r, int off, bool whole) {
    if (whole) return load16<0>(r, off, 0);
    const int at = off & ~3;
    const bool odd = off & 2;
    const u4_t q = load16<0>(r, at, 0);
    const uint32_t last = __builtin_amdgcn_raw_buffer_load_b32(r, at + (odd ? 16 : 12), 0, 0);
    u4_t s;
    s[0] = __builtin_amdgcn_alignbyte(q[1], q[0], 2);
    s[1] = __builtin_amdgcn_alignbyte(q[2], q[1], 2);
    s[2] = __builtin_amdgcn_alignbyte(q[3], q[2], 2);
    s[3] = __builtin_amdgcn_alignbyte(last, q[3], 2);
    return odd ? s : q;
}

// The same with only the first `valid` (< 8) elements, and zeros behind them.
__device__ __forceinline__ u4_t eight_first(rsrc_t r, int off, int valid) {
    u4_t s = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < valid)
            s[i >> 1] |= load2(r, off + 2 * i, 0) << (16 * (i & 1));
    return s;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return F16 ? pack_f16(a, b) : pack_bf16(a, b);
}
template <bool F16>
__device__ __forceinline__ float unpack1(uint16_t h) {
    return F16 ? static_cast<float>(__builtin_bit_cast(_Float16, h)) : bf16_f32(h);
}

}  // namespace
}  // namespace gfr
