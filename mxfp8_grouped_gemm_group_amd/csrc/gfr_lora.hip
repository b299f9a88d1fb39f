// A dense product with the low-rank adapter of each row's own request.
// include/gfr.h states the operator.
//
//   shrink   inner[t] = scaling[i] (x[t] A[i]^T), FP32 sums
//   dense    x W^T + bias
//   expand   + inner[t] B[i]^T + residual[t], rounded once
//
// Few rows: shrink, the dense product into FP32 (gfr_linear's kernels), expand.  Many:
// shrink on the matrix cores, and the expansion in the dense tiles' epilogue, where a
// wave's results are still in registers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gfr.h"
#include "gfr_device.h"
#include "gfr_direct.h"
#include "gfr_layer.h"
#include "gfr_tile.h"

namespace gfr {
namespace {

__device__ __forceinline__ float element(const void *p, int64_t i, bool f32, bool f16) {
    if (f32) return static_cast<const float *>(p)[i];
    const uint16_t h = static_cast<const uint16_t *>(p)[i];
    return f16 ? unpack1<true>(h) : unpack1<false>(h);
}

// Row t's adapter, -1 for none (and for ids out of range).
__device__ __forceinline__ int adapter(const LoraParams &p, int t) {
    const int i = p.ids[t];
    return i >= 0 && i < p.L ? i : -1;
}
__device__ __forceinline__ void check_adapter(const LoraParams &p, int t) {
    const int i = p.ids[t];
    if (p.status && (i < -1 || i >= p.L)) atomicOr(p.status, GFR_DEV_BAD_ADAPTER);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------

// R ranks of a row per wave, its lanes along K.
template <bool F16, bool ALIGNED, int R>
__global__ __launch_bounds__(256) void shrink_rows_kernel(LoraParams p, int waves_per_row) {
    const int lane = threadIdx.x & 63;
    const int id = uniform(static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 6));
    const int t = id / waves_per_row, j0 = id % waves_per_row * R;
    if (t >= p.M) return;
    if (j0 == 0 && lane == 0) check_adapter(p, t);
    const int i = adapter(p, t);
    if (i < 0) return;
    const uint16_t *x = p.x + static_cast<int64_t>(t) * p.K;
    const uint16_t *a[R];
#pragma unroll
    for (int q = 0; q < R; ++q)
        a[q] = p.a + (static_cast<int64_t>(i) * p.r + min(j0 + q, p.r - 1)) * p.K;
    float sum[R] = {};
    if (ALIGNED) {
#pragma unroll 4
        for (int k = 8 * lane; k < p.K; k += 512) {
            const u4_t xv = load<u4_t>(x + k);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const u4_t av = load<u4_t>(a[q] + k);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[q] = fmaf(unpack1<F16>(xv[e >> 1] >> (16 * (e & 1))),
                                  unpack1<F16>(av[e >> 1] >> (16 * (e & 1))), sum[q]);
            }
        }
    } else {
#pragma unroll 8
        for (int k = lane; k < p.K; k += 64) {
            const float xv = unpack1<F16>(x[k]);
#pragma unroll
            for (int q = 0; q < R; ++q) sum[q] = fmaf(xv, unpack1<F16>(a[q][k]), sum[q]);
        }
    }
    const float scale = p.scaling ? p.scaling[i] : 1.0f;
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const float v = wave_sum(sum[q]) * scale;
        if (lane == 0 && j0 + q < p.r) p.inner[static_cast<int64_t>(t) * p.r + j0 + q] = v;
    }
}

// A thread per column, a block's rows in turn; B's row of a column stays in registers
// while the adapter does (up to 64 ranks).
template <bool F16, bool ALIGNED>
__global__ __launch_bounds__(256) void expand_rows_kernel(LoraParams p, int rows) {
    const int n = blockIdx.x * 256 + threadIdx.x, at_n = min(n, p.N - 1);
    const int t0 = blockIdx.y * rows, t1 = min(t0 + rows, p.M);
    int kept = -1;
    u4_t b[8];
    for (int t = t0; t < t1; ++t) {
        const int64_t at = static_cast<int64_t>(t) * p.N + at_n;
        const float dense = p.dense[at];
        const uint16_t res = p.residual ? p.residual[at] : 0;
        const int i = uniform(adapter(p, t));
        float sum = 0.0f;
        if (i >= 0) {
            const float *s = p.inner + static_cast<int64_t>(t) * p.r;
            const uint16_t *row = p.b + (static_cast<int64_t>(i) * p.N + at_n) * p.r;
            if (ALIGNED && p.r <= 64) {
                if (i != kept)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (8 * c < p.r) b[c] = load<u4_t>(row + 8 * c);
                kept = i;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (8 * c < p.r)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            sum = fmaf(s[8 * c + e], unpack1<F16>(b[c][e >> 1] >> (16 * (e & 1))),
                                       sum);
            } else if (ALIGNED) {
                for (int j = 0; j < p.r; j += 8) {
                    const u4_t v = load<u4_t>(row + j);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum = fmaf(s[j + e], unpack1<F16>(v[e >> 1] >> (16 * (e & 1))), sum);
                }
            } else {
                for (int j = 0; j < p.r; ++j) sum = fmaf(s[j], unpack1<F16>(row[j]), sum);
            }
        }
        float y = dense + sum;
        if (p.residual) y += unpack1<F16>(res);
        if (n >= p.N) continue;
        if (p.out_f32)
            static_cast<float *>(p.out)[at] = y;
        else
            static_cast<uint16_t *>(p.out)[at] = static_cast<uint16_t>(pack2<F16>(y, 0.0f));
    }
}

// ---------------------------------------------------------------------------
// Many rows
// ---------------------------------------------------------------------------

// 32 rows a block, its eight waves along K, 32 RF ranks at a time; an adapter after the
// other where the rows have several.  inner is kept as two 16-bit terms, the value and
// what its rounding left over: 16 bits of mantissa or more, for the matrix cores.
constexpr int kShrinkWaves = 8;
template <bool F16, int RF>
__global__ __launch_bounds__(kShrinkWaves * 64, 2) void shrink_tile_kernel(LoraParams p) {
    __shared__ float part[kShrinkWaves][32][33];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 31, g = lane >> 5, t0 = blockIdx.x * 32;
    const int rows = min(32, p.M - t0), row_bytes = 2 * p.K;
    const int id = c < rows ? adapter(p, t0 + c) : -1;
    if (wave == 0 && lane < rows) check_adapter(p, t0 + lane);
    const rsrc_t xr = buffer(p.x + static_cast<int64_t>(t0) * p.K,
                             static_cast<int64_t>(rows) * row_bytes);
    const int steps = (p.K + 63) / 64;
    const int s0 = steps * wave / kShrinkWaves, s1 = steps * (wave + 1) / kShrinkWaves;
    uint64_t todo = __builtin_amdgcn_ballot_w64(id >= 0);
    while (todo) {
        const int i = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        todo &= ~__builtin_amdgcn_ballot_w64(id == i);
        const float scale = p.scaling ? p.scaling[i] : 1.0f;
        const rsrc_t ar = buffer(p.a + static_cast<int64_t>(i) * p.r * p.K,
                                 static_cast<int64_t>(p.r) * row_bytes);
        for (int j0 = 0; j0 < p.r; j0 += 32 * RF) {
            f16_t acc[RF] = {};
#pragma unroll 1
            for (int s = s0; s < s1; ++s) {
                u4_t xv[4], av[RF][4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int k = 64 * s + 16 * h + 8 * g;
                    const int off = k < p.K ? c * row_bytes + 2 * k : kPast;
                    xv[h] = load16<0>(xr, off, 0);
#pragma unroll
                    for (int f = 0; f < RF; ++f)
                        av[f][h] = load16<0>(ar, off, (j0 + 32 * f) * row_bytes);
                }
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int f = 0; f < RF; ++f) acc[f] = mfma32<F16>(av[f][h], xv[h], acc[f]);
            }
#pragma unroll
            for (int f = 0; f < RF; ++f) {
                // lane (c, g): row c, ranks 8 q + 4 g .. + 3
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    part[wave][c][8 * (e >> 2) + 4 * g + (e & 3)] = acc[f][e];
                __syncthreads();
                const int row = threadIdx.x >> 4, j = threadIdx.x & 15;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int rank = j0 + 32 * f + j + 16 * h;
                    float v = 0.0f;
#pragma unroll
                    for (int w = 0; w < kShrinkWaves; ++w) v += part[w][row][j + 16 * h];
                    if (row < rows && rank < p.r && adapter(p, t0 + row) == i) {
                        v *= scale;
                        uint16_t *to = p.terms + static_cast<int64_t>(t0 + row) * 2 * p.r + rank;
                        const uint16_t hi = static_cast<uint16_t>(pack2<F16>(v, 0.0f));
                        to[0] = hi;
                        to[p.r] = static_cast<uint16_t>(pack2<F16>(v - unpack1<F16>(hi), 0.0f));
                    }
                }
                __syncthreads();
            }
        }
    }
}

// The dense product's tiles: bands of eight by all columns, an eighth of them per XCD.
struct LoraTiles {
    const LoraParams &p;
    int tiles_m, tiles_n, begin, end, stride;
    Divisor by_band;

    __device__ __forceinline__ explicit LoraTiles(const LoraParams &p_)
        : p(p_), tiles_m((p.M + kTile - 1) / kTile), tiles_n((p.N + kTile - 1) / kTile),
          by_band(8 * tiles_n) {
        const int total = tiles_m * tiles_n, per = (total + 7) / 8, xcd = blockIdx.x & 7;
        stride = gridDim.x >> 3;
        begin = xcd * per + (blockIdx.x >> 3);
        end = min(total, (xcd + 1) * per);
    }
    __device__ __forceinline__ TileAt at(int id) const {
        const int band = by_band.of(id), in_band = id - band * 8 * tiles_n;
        const int depth = min(8, tiles_m - band * 8), column = Divisor(depth).of(in_band);
        TileAt t;
        t.e = 0;
        t.n0 = uniform(column * kTile);
        t.m0 = uniform((band * 8 + in_band - column * depth) * kTile);
        t.rows = uniform(min(kTile, p.M - t.m0));
        t.steps = (p.K + 63) / 64;
        return t;
    }
    template <class A, class B>
    __device__ __forceinline__ void loads(const TileAt &t, A &da, B &db) const {
        const int64_t k = p.K;
        da.tile(p.x + t.m0 * k, 2 * t.rows * k, p.K, t.rows);
        db.tile(p.w + t.n0 * k, 2 * min(kTile, p.N - t.n0) * k, p.K, 0);
    }
};

template <bool F16>
struct LoraFinish {
    const LoraParams &p;

    // The adapters' part of a wave's results.  Rows with one adapter between them take
    // its products straight into their sums; where a fragment's 32 rows have several,
    // each adapter's product is made apart and kept by its own rows alone, so that what
    // another request's adapter holds (NaN too) reaches nobody else.
    template <int FM, int FN>
    __device__ __forceinline__ void expand(const TileAt &t, f16_t (&acc)[FM][FN], int wm, int wn,
                                           int lane) const {
        const int c = lane & 31, g = lane >> 5, row0 = t.m0 + wm, rows = t.rows - wm;
        if (rows <= 0) return;
        int id[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i) id[i] = adapter(p, row0 + min(32 * i + c, rows - 1));
        const int one = uniform(id[0]);
        bool same = true;
#pragma unroll
        for (int i = 0; i < FM; ++i) same &= id[i] == one;
        const int64_t r = p.r;
        const int s_row = 4 * p.r, b_row = 2 * p.r, parts = (p.r + 15) / 16;
        const rsrc_t sr = uniform_buffer(reinterpret_cast<const char *>(p.terms + row0 * 2 * r),
                                         static_cast<int64_t>(rows) * s_row);
        auto b_of = [&](int i) {
            const int64_t n = t.n0 + wn;
            return uniform_buffer(reinterpret_cast<const char *>(p.b + (i * int64_t{p.N} + n) * r),
                                  n < p.N ? (p.N - n) * b_row : 0);
        };
        if (__builtin_amdgcn_ballot_w64(same) == ~uint64_t{0}) {
            if (one < 0) return;
            const rsrc_t br = b_of(one);
#pragma unroll 1
            for (int part = 0; part < parts; ++part) {
                const int k = 16 * part + 8 * g;
                u4_t bv[FN];
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    bv[j] = load16<0>(br, k < p.r ? (32 * j + c) * b_row + 2 * k : kPast, 0);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const int off = k < p.r ? (32 * i + c) * s_row + 2 * k : kPast;
                    const u4_t hi = load16<0>(sr, off, 0), lo = load16<0>(sr, off, b_row);
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        acc[i][j] = mfma32<F16>(bv[j], hi, acc[i][j]);
                        acc[i][j] = mfma32<F16>(bv[j], lo, acc[i][j]);
                    }
                }
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            uint64_t todo = __builtin_amdgcn_ballot_w64(id[i] >= 0 && 32 * i + c < rows);
            while (todo) {
                const int a = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(todo));
                const bool mine = id[i] == a;
                todo &= ~__builtin_amdgcn_ballot_w64(mine);
                const rsrc_t br = b_of(a);
                f16_t own[FN] = {};
#pragma unroll 1
                for (int part = 0; part < parts; ++part) {
                    const int k = 16 * part + 8 * g;
                    const int off = k < p.r ? (32 * i + c) * s_row + 2 * k : kPast;
                    const u4_t hi = load16<0>(sr, off, 0), lo = load16<0>(sr, off, b_row);
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const u4_t bv =
                            load16<0>(br, k < p.r ? (32 * j + c) * b_row + 2 * k : kPast, 0);
                        own[j] = mfma32<F16>(bv, hi, own[j]);
                        own[j] = mfma32<F16>(bv, lo, own[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] += mine ? own[j][e] : 0.0f;
            }
        }
    }

    template <int FM, int FN>
    __device__ __forceinline__ int tile(const TileAt &t, f16_t (&acc)[FM][FN], int wm, int wn,
                                        int lane) const {
        expand(t, acc, wm, wn, lane);
        __builtin_amdgcn_sched_barrier(0);
        // A lane has four columns of row lane % 32 at a time; it trades halves with its
        // row's other lane for eight, and 16-bit results once more, for runs of 64 bytes.
        const int c = lane & 31, g = lane >> 5, es = p.out_f32 ? 4 : 2;
        const int bias_es = p.bias_f32 ? 4 : 2;
        const rsrc_t bias = uniform_buffer(static_cast<const char *>(p.bias),
                                           p.bias ? static_cast<int64_t>(p.N) * bias_es : 0);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int64_t row = t.m0 + wm + 32 * i;
            const int rows = max(0, min(32, t.rows - wm - 32 * i));
            const rsrc_t to =
                uniform_buffer(static_cast<char *>(p.out) + row * p.N * es,
                               static_cast<int64_t>(rows) * p.N * es);
            const rsrc_t from = uniform_buffer(
                reinterpret_cast<const char *>(p.residual + (p.residual ? row * p.N : 0)),
                p.residual ? static_cast<int64_t>(rows) * p.N * 2 : 0);
            u4_t res[FN][2];
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int n = t.n0 + wn + 32 * j + 16 * q + 8 * g;
                    res[j][q] = load16<0>(from, n < p.N ? 2 * (c * p.N + n) : kPast, 0);
                }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                u4_t h[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int n = t.n0 + wn + 32 * j + 16 * q + 8 * g;
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const auto w = __builtin_amdgcn_permlane32_swap(
                            __float_as_uint(acc[i][j][8 * q + e]),
                            __float_as_uint(acc[i][j][8 * q + 4 + e]), false, false);
                        y[e] = __uint_as_float(w[0]);
                        y[4 + e] = __uint_as_float(w[1]);
                    }
                    if (p.bias_f32) {
                        const f4_t b0 = __builtin_bit_cast(f4_t, load16<0>(bias, 4 * n, 0));
                        const f4_t b1 = __builtin_bit_cast(f4_t, load16<0>(bias, 4 * n, 16));
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] += b0[e], y[4 + e] += b1[e];
                    } else if (p.bias) {
                        const u4_t b = load16<0>(bias, 2 * n, 0);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            y[e] += unpack1<F16>(b[e >> 1] >> (16 * (e & 1)));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] += unpack1<F16>(res[j][q][e >> 1] >> (16 * (e & 1)));
                    if (p.out_f32) {
                        const int off = n < p.N ? 4 * (c * p.N + n) : kPast;
                        store16(to, __builtin_bit_cast(u4_t, f4_t{y[0], y[1], y[2], y[3]}), off);
                        store16(to, __builtin_bit_cast(u4_t, f4_t{y[4], y[5], y[6], y[7]}),
                                off + 16);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[q][e] = pack2<F16>(y[2 * e], y[2 * e + 1]);
                }
                if (!p.out_f32) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const auto w =
                            __builtin_amdgcn_permlane16_swap(h[0][e], h[1][e], false, false);
                        h[0][e] = w[0];
                        h[1][e] = w[1];
                    }
                    const int n = t.n0 + wn + 32 * j + 16 * (lane >> 4 & 1) + 8 * g;
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        store16(to, h[q],
                                n < p.N ? 2 * (((lane & 15) + 16 * q) * p.N + n) : kPast);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        return FM * FN * 2;
    }
    __device__ __forceinline__ void clear(const TileAt &) const {}
};

template <bool F16>
__global__ __launch_bounds__(kWaves * 64, 1) void lora_tile_kernel(LoraParams p) {
    extern __shared__ u4_t lds[];     // [2][x's 256 rows, w's][8]
    const LoraTiles tiles(p);
    const LoraFinish<F16> finish{p};
    run_tiles<F16, false, false>(lds, tiles, finish, p.K, p.K);
}

template <bool F16, bool ALIGNED, int R>
hipError_t launch_shrink_rows(const LoraParams &p, hipStream_t stream) {
    const int per = (p.r + R - 1) / R;
    const int64_t blocks = (static_cast<int64_t>(p.M) * per + 3) / 4;
    hipLaunchKernelGGL((shrink_rows_kernel<F16, ALIGNED, R>), dim3(static_cast<uint32_t>(blocks)),
                       dim3(256), 0, stream, p, per);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_rows(const LoraParams &p, hipStream_t stream) {
    const bool many = static_cast<int64_t>(p.M) * p.r >= 8192;
    hipError_t e;
    if (p.K % 8 == 0)
        e = many ? launch_shrink_rows<F16, true, 4>(p, stream)
                 : launch_shrink_rows<F16, true, 1>(p, stream);
    else
        e = many ? launch_shrink_rows<F16, false, 4>(p, stream)
                 : launch_shrink_rows<F16, false, 1>(p, stream);
    if (e != hipSuccess) return e;
    LinearParams d{};
    d.x = p.x;
    d.w = p.w;
    d.bias = p.bias;
    d.bias_f32 = p.bias_f32;
    d.out = p.dense;
    d.out_f32 = 1;
    d.f16 = p.f16;
    d.act = GFR_ACT_NONE;
    d.wide = p.N % 8 == 0;
    d.M = p.M;
    d.N = p.N;
    d.K = p.K;
    d.kernel = p.choice.kernel;
    d.split = p.choice.split;
    d.partial = p.partial;
    if (e = launch_linear(d, stream); e != hipSuccess) return e;
    // about 2048 blocks, of one row or more
    const int columns = (p.N + 255) / 256;
    int64_t rows = (static_cast<int64_t>(p.M) * columns + 2047) / 2048;
    if (const int64_t least = (p.M + 65534) / 65535; rows < least) rows = least;
    const dim3 grid(columns, static_cast<uint32_t>((p.M + rows - 1) / rows));
    if (p.r % 8 == 0)
        hipLaunchKernelGGL((expand_rows_kernel<F16, true>), grid, dim3(256), 0, stream, p,
                           static_cast<int>(rows));
    else
        hipLaunchKernelGGL((expand_rows_kernel<F16, false>), grid, dim3(256), 0, stream, p,
                           static_cast<int>(rows));
    return hipGetLastError();
}

template <bool F16, int RF>
hipError_t launch_shrink_tiles(const LoraParams &p, hipStream_t stream) {
    hipLaunchKernelGGL((shrink_tile_kernel<F16, RF>), dim3((p.M + 31) / 32),
                       dim3(kShrinkWaves * 64), 0, stream, p);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_tiles(const LoraParams &p, hipStream_t stream) {
    const hipError_t e = p.r <= 32   ? launch_shrink_tiles<F16, 1>(p, stream)
                         : p.r <= 64 ? launch_shrink_tiles<F16, 2>(p, stream)
                                     : launch_shrink_tiles<F16, 4>(p, stream);
    if (e != hipSuccess) return e;
    constexpr int lds = 2 * kStage * 16;
    constexpr auto kernel = &lora_tile_kernel<F16>;
    if (const hipError_t a = allow_lds<kernel>(lds); a != hipSuccess) return a;
    hipLaunchKernelGGL(kernel, dim3(256), dim3(kWaves * 64), lds, stream, p);
    return hipGetLastError();
}

}  // namespace

LoraLayout lora_layout(int64_t M, int64_t N, int64_t K, int64_t r) {
    const auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    LoraLayout l{};
    // Whole tiles where they fill half of the CUs.
    l.tiles = K % 8 == 0 && N % 8 == 0 && r % 8 == 0 &&
              ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile) >= 128;
    if (l.tiles) {
        l.total = up(2 * sizeof(uint16_t) * M * r);
        return l;
    }
    l.choice = linear_choice(M, N, K, GFR_ACT_NONE);
    l.dense = up(sizeof(float) * M * r);
    l.partial = l.dense + up(sizeof(float) * M * N);
    l.total = l.partial;
    if (l.choice.split > 1)
        l.total += up(sizeof(float) * l.choice.split * M * ((N + 7) / 8 * 8));
    return l;
}

hipError_t launch_lora(const LoraParams &p, hipStream_t stream) {
    if (p.tiles)
        return p.f16 ? launch_tiles<true>(p, stream) : launch_tiles<false>(p, stream);
    return p.f16 ? launch_rows<true>(p, stream) : launch_rows<false>(p, stream);
}

}  // namespace gfr
