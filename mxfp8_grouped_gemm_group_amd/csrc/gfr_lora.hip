// A dense product with the low-rank adapter of each row's own request.
// include/gfr.h states the operator.
//
//   shrink   inner[t] = scaling[i] (x[t] A[i]^T), FP32 sums
//   dense    x W^T + bias
//   expand   + inner[t] B[i]^T + residual[t], rounded once
//
// Few rows: shrink, the dense product into FP32 (gfr_linear's kernels), expand.  Many:
// shrink on the matrix cores; the dense tiles, of which 32 rows with one adapter between
// them take its expansion as a few steps more of their sum (bf16: inner as three terms); and
// for the 32 rows that have several, whose sums were kept in FP32, a launch that goes on with
// each row's own, so that what another request's adapter holds (NaN too) reaches nobody else.
// With F16 that launch expands all rows, on the FP32 matrix instructions: F16 terms do not
// have inner's range (4096 rows of 4096 x 7168 by rank 64: tiles 237 us and it 78, in bf16
// 239 and 16; whole calls by rank 16 254 and 228).
#include <hip/hip_runtime.h>
#include <math.h>
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

// inner as three bf16 terms whose sum it is: of 16 ranks (or the last 8) the smallest terms,
// then the middle ones, then the largest, which so join in FP32 without loss.  All have its
// sign, and none is zero unless it is: their products with an infinity of B, and those of an
// infinite inner, are what the one product would be.  (A bf16 value goes as its half and two
// quarters.)
__device__ __forceinline__ void put_terms(const LoraParams &p, int64_t t, int rank, float v) {
    const auto cut = [](float f) { return __uint_as_float(__float_as_uint(f) & 0xffff0000u); };
    float first = cut(v);
    const float rest = v - first;                        // up to 16 bits
    float second = cut(rest), third = rest - second;     // up to 8
    if (rest == 0.0f) first = 0.5f * v, second = third = 0.25f * v;
    else if (third == 0.0f) second = third = 0.5f * rest;
    // (a NaN may have all its payload below)
    if (!(fabsf(v) < INFINITY)) first = second = third = v != v ? NAN : v;
    const int group = rank & ~15, width = group + 16 <= p.r ? 16 : 8;
    uint16_t *to = p.terms + t * 3 * p.r + 3 * group + (rank - group);
    to[0] = static_cast<uint16_t>(__float_as_uint(third) >> 16);
    to[width] = static_cast<uint16_t>(__float_as_uint(second) >> 16);
    to[2 * width] = static_cast<uint16_t>(__float_as_uint(first) >> 16);
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
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + uniform(threadIdx.x >> 6);
    const int t = static_cast<int>(id / waves_per_row);
    const int j0 = static_cast<int>(id % waves_per_row) * R;
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

// A result of the dense product: its K splits' sums, in order, and the bias.
template <bool F16>
__device__ __forceinline__ float dense_sum(const LoraParams &p, int t, int n, float bias) {
    const int64_t pitch = p.choice.split > 1 ? (p.N + 7) / 8 * 8 : p.N;
    const float *at = p.dense + t * pitch + n;
    float v = 0.0f;
    for (int s = 0; s < p.choice.split; ++s) v += at[s * p.M * pitch];
    return v + bias;
}

// A thread per column, a block's rows in turn; B's row of a column stays in registers
// while the adapter does (up to 64 ranks; V of them come at a time).  inner, in FP32, is the
// same in all lanes and comes through scalar loads.
template <bool F16, int V>
__global__ __launch_bounds__(256) void expand_rows_kernel(LoraParams p, int rows) {
    typedef const __attribute__((address_space(4))) float *scalar_t;
    const int n = blockIdx.x * 256 + threadIdx.x, at_n = min(n, p.N - 1);
    const int t0 = blockIdx.y * rows, t1 = min(t0 + rows, p.M);
    const float bias = p.bias ? element(p.bias, at_n, p.bias_f32, F16) : 0.0f;
    int kept = -1;
    uint32_t b[32];                   // two ranks each
    for (int t = t0; t < t1; ++t) {
        const int64_t at = static_cast<int64_t>(t) * p.N + at_n;
        const int i = uniform(adapter(p, t));
        const uint16_t *row = p.b + (static_cast<int64_t>(max(i, 0)) * p.N + at_n) * p.r;
        const uint16_t res = p.residual ? p.residual[at] : 0;
        float y = dense_sum<F16>(p, t, at_n, bias);
        const scalar_t s = (scalar_t)(p.inner + static_cast<int64_t>(t) * p.r);
        float sum = 0.0f;
        if (i >= 0 && V > 1) {
            for (int k0 = 0; k0 < p.r; k0 += 64) {
                const int ranks = min(64, p.r - k0);
                if (i != kept || p.r > 64)
#pragma unroll
                    for (int j = 0; j < 64; j += V)
                        if (j < ranks) {
                            if (V == 8) {
                                const u4_t v = load<u4_t>(row + k0 + j);
#pragma unroll
                                for (int e = 0; e < 4; ++e) b[j / 2 + e] = v[e];
                            } else {
                                const u2_t v = load<u2_t>(row + k0 + j);
                                b[j / 2] = v[0];
                                b[j / 2 + 1] = v[1];
                            }
                        }
#pragma unroll
                for (int j = 0; j < 64; j += V)
                    if (j < ranks)
#pragma unroll
                        for (int e = j; e < j + V; ++e)
                            sum = fmaf(s[k0 + e], unpack1<F16>(b[e / 2] >> (16 * (e & 1))), sum);
            }
            kept = i;
            y += sum;
        } else if (i >= 0) {
#pragma unroll 8
            for (int j = 0; j < p.r; ++j) sum = fmaf(s[j], unpack1<F16>(row[j]), sum);
            y += sum;
        }
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

// 32 rows by 32 ranks a block, its eight waves along K; an adapter after the other where
// the rows have several.  A wave's two stages of 64 K are filled straight from memory, in
// whole lines (fragments loaded from memory took 32 half lines a load: 4096 rows of 4096
// by rank 64 51 us, so 18).
//
// codes[row / 32]: the adapter of 32 rows, -1 for none, kApart where the dense tiles leave
// the expansion to a launch of its own: of several adapters, and with F16 of any.
constexpr int kApart = -2;
constexpr int kShrinkWaves = 8;
constexpr int kShrinkLds = kShrinkWaves * 2 * 64 * 8 * 16;
template <bool F16>
__global__ __launch_bounds__(kShrinkWaves * 64, 2) void shrink_tile_kernel(LoraParams p) {
    extern __shared__ u4_t lds[];           // [wave][2][x's 32 lines, A's][8]; then the sums
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 31, g = lane >> 5, t0 = blockIdx.x * 32, j0 = blockIdx.y * 32;
    const int rows = min(32, p.M - t0), row_bytes = 2 * p.K;
    const int id = c < rows ? adapter(p, t0 + c) : -1;
    if (blockIdx.y == 0 && wave == 0 && lane < rows) check_adapter(p, t0 + lane);
    const rsrc_t xr = uniform_buffer(
        reinterpret_cast<const char *>(p.x + static_cast<int64_t>(t0) * p.K),
        static_cast<int64_t>(rows) * row_bytes);
    const int steps = (p.K + 63) / 64;
    const int s0 = steps * wave / kShrinkWaves, s1 = steps * (wave + 1) / kShrinkWaves;
    // a load takes eight lines; the lane's piece of even and odd ones
    const int line = lane >> 3;
    int piece[2], off[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        piece[h] = (lane & 7) ^ ((line >> 1) + 4 * h);
        off[h] = line * row_bytes + 16 * piece[h];
    }
    u4_t *const mine = lds + wave * 2 * 64 * 8;
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) void *)lds)) + wave * 2 * 64 * 128;
    const int first_id = uniform(id);
    if (blockIdx.y == 0 && wave == 0) {
        const bool same = __builtin_amdgcn_ballot_w64(c < rows && id != first_id) == 0;
        if (lane == 0) p.codes[blockIdx.x] = same && (!F16 || id < 0) ? id : kApart;
    }
    uint64_t todo = __builtin_amdgcn_ballot_w64(id >= 0);
    while (todo) {
        const int i = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        todo &= ~__builtin_amdgcn_ballot_w64(id == i);
        const float scale = p.scaling ? p.scaling[i] : 1.0f;
        const int64_t rank0 = static_cast<int64_t>(i) * p.r + j0;
        const rsrc_t ar = uniform_buffer(reinterpret_cast<const char *>(p.a + rank0 * p.K),
                                         static_cast<int64_t>(min(32, p.r - j0)) * row_bytes);
        f16_t acc = {};
        // (behind the wave's last step: zeros)
        auto fetch = [&](int s) GFR_INLINE {
            const uint32_t to = lds0 + (s - s0 & 1) * 64 * 128;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int o = s < s1 && 64 * s + 8 * piece[h & 1] < p.K ? off[h & 1] : kPast;
                load_lds(xr, o, 8 * h * row_bytes + 128 * s, to + h * 1024);
                load_lds(ar, o, 8 * h * row_bytes + 128 * s, to + (4 + h) * 1024);
            }
        };
        fetch(s0);
        for (int s = s0; s < s1; ++s) {
            fetch(s + 1);
            asm volatile("s_waitcnt vmcnt(8)" ::: "memory");       // this step's eight landed
            const u4_t *stage = mine + (s - s0 & 1) * 64 * 8;
            u4_t xv[4], av[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                xv[h] = fragment<false, 32>(stage, 0, h, lane);
                av[h] = fragment<false, 32>(stage + 32 * 8, 0, h, lane);
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) acc = mfma32<F16>(av[h], xv[h], acc);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // read, before it is filled
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();                                           // the sums go over the stages
        float(*part)[32][33] = reinterpret_cast<float(*)[32][33]>(lds);
        // lane (c, g): row c, ranks 8 q + 4 g .. + 3
#pragma unroll
        for (int e = 0; e < 16; ++e) part[wave][c][8 * (e >> 2) + 4 * g + (e & 3)] = acc[e];
        __syncthreads();
        const int row = threadIdx.x >> 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = (threadIdx.x & 15) + 16 * h;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kShrinkWaves; ++w) v += part[w][row][j];
            if (row < rows && j0 + j < p.r && adapter(p, t0 + row) == i) {
                if (!F16 && p.tiles) put_terms(p, t0 + row, j0 + j, v * scale);
                else p.inner[static_cast<int64_t>(t0 + row) * p.r + j0 + j] = v * scale;
            }
        }
        __syncthreads();
    }
}

// The dense product's tiles: bands of eight by all columns, an eighth of them per XCD.  A
// tile of bf16 ends with the expansions of its fragments' adapters, each one run of steps
// over inner's terms, B's ranks three times.
template <bool F16>
struct LoraTiles {
    static constexpr bool kExtra = !F16;
    int tiles_m, tiles_n, begin, end, stride;
    Divisor by_band;

    __device__ __forceinline__ explicit LoraTiles(const LoraParams &p)
        : tiles_m((p.M + kTile - 1) / kTile), tiles_n((p.N + kTile - 1) / kTile),
          by_band(8 * tiles_n) {
        const int total = tiles_m * tiles_n, per = (total + 7) / 8, xcd = blockIdx.x & 7;
        stride = gridDim.x >> 3;
        begin = xcd * per + (blockIdx.x >> 3);
        end = min(total, (xcd + 1) * per);
    }
    __device__ __forceinline__ TileAt at(int id) const {
        const int lane = threadIdx.x & 63;
        const int band = by_band.of(id), in_band = id - band * 8 * tiles_n;
        const int depth = min(8, tiles_m - band * 8), column = Divisor(depth).of(in_band);
        const LoraParams p = fresh<LoraParams>();
        TileAt t;
        t.e = 0;
        t.n0 = uniform(column * kTile);
        t.m0 = uniform((band * 8 + in_band - column * depth) * kTile);
        t.rows = uniform(min(kTile, p.M - t.m0));
        t.extra = 0;
        t.masks = 0;
        t.steps = (p.K + 63) / 64;
        if (F16) return t;
        const int fragments = (t.rows + 31) / 32;
        const int code = p.codes[t.m0 / 32 + min(lane, fragments - 1)];
        uint64_t todo = __builtin_amdgcn_ballot_w64((lane < fragments) & (code >= 0));
        t.extra_run = (3 * p.r + 63) / 64;
        while (todo) {
            const int a = __builtin_amdgcn_readlane(code, __builtin_ctzll(todo));
            const uint64_t mine = todo & __builtin_amdgcn_ballot_w64(code == a);
            todo &= ~mine;
            t.masks |= mine << (8 * (t.extra / t.extra_run));
            t.extra += t.extra_run;
        }
        t.extra = uniform(t.extra);
        t.steps += t.extra;
        return t;
    }
    // The loads' tile and the adapters left in it (masks).
    struct Cursor {
        int id;
        TileAt t;
        __device__ __forceinline__ explicit Cursor(int first) : id(first) { t.masks = 0; }
    };
    template <class A, class B>
    __device__ __forceinline__ int next(Cursor &c, A &da, B &db, int wave, int lane) const {
        const LoraParams p = fresh<LoraParams>();
        if (!F16 && c.t.masks != 0) {
            const int64_t r = p.r, columns = min(kTile, p.N - c.t.n0);
            const int a = uniform(p.codes[c.t.m0 / 32 + __builtin_ctzll(c.t.masks & 0xff)]);
            da.init(3 * r, wave, lane);
            db.init(r, wave, lane);
            da.tile(p.terms + c.t.m0 * 3 * r, 2 * c.t.rows * 3 * r, 3 * p.r, c.t.rows);
            db.tile(p.b + (a * int64_t{p.N} + c.t.n0) * r, 2 * columns * r, 3 * p.r, 0, 0, p.r / 8);
            c.t.masks >>= 8;
            return c.t.extra_run;
        }
        c.id = uniform(c.id + stride);
        if (c.id >= uniform(end)) return 0;
        c.t = at(c.id);
        const int64_t k = p.K, columns = min(kTile, p.N - c.t.n0);
        da.init(k, wave, lane);
        db.init(k, wave, lane);
        da.tile(p.x + c.t.m0 * k, 2 * c.t.rows * k, p.K, c.t.rows);
        db.tile(p.w + c.t.n0 * k, 2 * columns * k, p.K, 0);
        return (p.K + 63) / 64;
    }
};

// The 32 x 32 sums of which FP32 memory holds a copy, in the order that lanes have them: at
// fragment (row / 32, column / 32), four sums of all lanes after another.
__device__ __forceinline__ rsrc_t apart(const LoraParams &p, int row, int n) {
    const int64_t fragment = row / 32 * static_cast<int64_t>((p.N + 31) / 32) + n / 32;
    return uniform_buffer(reinterpret_cast<char *>(p.dense + 1024 * fragment), 4096);
}

// A lane's places in 32 rows of 32 columns from n0 on: lane (c, g) has columns n0 + 16 q +
// 8 g .. + 7 of row c once it has traded halves with its row's other lane.
struct Columns {
    int n0, g;
    __device__ __forceinline__ int of(int q) const { return n0 + 16 * q + 8 * g; }
};

__device__ __forceinline__ rsrc_t residual_rows(const LoraParams &p, int64_t row, int rows) {
    return uniform_buffer(reinterpret_cast<const char *>(p.residual + (p.residual ? row * p.N : 0)),
                          p.residual ? static_cast<int64_t>(rows) * p.N * 2 : 0);
}
__device__ __forceinline__ rsrc_t bias_row(const LoraParams &p) {
    return uniform_buffer(static_cast<const char *>(p.bias),
                          p.bias ? static_cast<int64_t>(p.N) * (p.bias_f32 ? 4 : 2) : 0);
}

// 32 x 32 sums with their bias (16-bit: `bias`) and residual (`res`), rounded and written to
// `rows` rows from `row` on: a lane trades halves for eight columns, and 16-bit results once
// more, for runs of 64 bytes.  Two stores or more.
template <bool F16>
__device__ __forceinline__ void put_sums(const LoraParams &p, const f16_t &acc, int64_t row,
                                         int rows, Columns at, rsrc_t from_bias,
                                         const u4_t (&bias)[2], const u4_t (&res)[2], int lane) {
    const int c = lane & 31, es = p.out_f32 ? 4 : 2;
    const rsrc_t to = uniform_buffer(static_cast<char *>(p.out) + row * p.N * es,
                                     static_cast<int64_t>(rows) * p.N * es);
    u4_t h[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int n = at.of(q);
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[8 * q + e]),
                                                            __float_as_uint(acc[8 * q + 4 + e]),
                                                            false, false);
            y[e] = __uint_as_float(w[0]);
            y[4 + e] = __uint_as_float(w[1]);
        }
        if (p.bias_f32) {
            const f4_t b0 = __builtin_bit_cast(f4_t, load16<0>(from_bias, 4 * n, 0));
            const f4_t b1 = __builtin_bit_cast(f4_t, load16<0>(from_bias, 4 * n, 16));
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] += b0[e], y[4 + e] += b1[e];
        } else if (p.bias) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += unpack1<F16>(bias[q][e >> 1] >> (16 * (e & 1)));
        }
        if (p.residual)
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += unpack1<F16>(res[q][e >> 1] >> (16 * (e & 1)));
        if (p.out_f32) {
            const int off = n < p.N ? 4 * (c * p.N + n) : kPast;
            store16(to, __builtin_bit_cast(u4_t, f4_t{y[0], y[1], y[2], y[3]}), off);
            store16(to, __builtin_bit_cast(u4_t, f4_t{y[4], y[5], y[6], y[7]}), off + 16);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) h[q][e] = pack2<F16>(y[2 * e], y[2 * e + 1]);
    }
    if (p.out_f32) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const auto w = __builtin_amdgcn_permlane16_swap(h[0][e], h[1][e], false, false);
        h[0][e] = w[0];
        h[1][e] = w[1];
    }
    const int n = at.n0 + 16 * (lane >> 4 & 1) + 8 * at.g;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        store16(to, h[q], n < p.N ? 2 * (((lane & 15) + 16 * q) * p.N + n) : kPast);
}

template <bool F16>
struct LoraFinish {
    static constexpr bool kLong = true;
    template <int FM, int FN>
    __device__ __forceinline__ int tile(const TileAt &t, f16_t (&acc)[FM][FN], int wm, int wn,
                                        int lane) const {
        if (t.rows <= wm) return 0;
        const LoraParams p = fresh<LoraParams>();
        const int c = lane & 31, g = lane >> 5;
        const rsrc_t from_bias = bias_row(p);
        auto columns = [&](int j) { return Columns{t.n0 + wn + 32 * j, g}; };
        u4_t bias[FN][2], res[2][FN][2];
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                bias[j][q] = load16<0>(from_bias, p.bias_f32 ? kPast : 2 * columns(j).of(q), 0);
        // (a block of 32 rows ahead of its use)
        auto fetch = [&](int i) GFR_INLINE {
            const rsrc_t from = residual_rows(p, t.m0 + wm + 32 * i,
                                              max(0, min(32, t.rows - wm - 32 * i)));
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int n = columns(j).of(q);
                    res[i & 1][j][q] = load16<0>(from, n < p.N ? 2 * (c * p.N + n) : kPast, 0);
                }
        };
        fetch(0);
        // (lane f: fragment f's code)
        const int codes = p.codes[(t.m0 + wm) / 32 + min(lane, (t.rows - wm - 1) / 32)];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int row = t.m0 + wm + 32 * i, rows = max(0, min(32, t.rows - wm - 32 * i));
            if (i + 1 < FM) fetch(i + 1);
            __builtin_amdgcn_sched_barrier(0);
            const bool later = __builtin_amdgcn_readlane(codes, i) == kApart;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int n0 = columns(j).n0;
                if (later) {
                    const rsrc_t to = apart(p, row, n0);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f4_t y = {acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                        acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                        store16(to, __builtin_bit_cast(u4_t, y),
                                rows > 0 && n0 < p.N ? 1024 * q + 16 * lane : kPast);
                    }
                } else {
                    put_sums<F16>(p, acc[i][j], row, rows, columns(j), from_bias, bias[j],
                                  res[i & 1][j], lane);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        return FM * FN * 2;
    }
    __device__ __forceinline__ void clear(const TileAt &) const {}
};

// The 32 rows left to it, 32 W columns a wave: each adapter's product goes on from all rows'
// dense sums and is kept by its own, the ranks in the dense tiles' order, so that a row gets
// the same bits there and here.  With F16 the products are in FP32.
//
// Bound by its loads, 32 lines each.  bf16 takes two fragments of columns from 24 ranks on,
// which read inner once for both (2048 rows in random order over 64 adapters of 4096 columns,
// us: rank 64 384 and 267, 32 110 and 85, 16 46 and 57); F16, with more rows, one, 32 ranks
// at a time, for more waves (4096 rows of 7168 columns, rank 64: 61, with two 73, with 64
// ranks at a time 65).
template <bool F16, int W>
__global__ __launch_bounds__(256) void expand_tile_kernel(LoraParams p) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 31, g = lane >> 5, t0 = blockIdx.y * 32;
    const int n0 = (blockIdx.x * 4 + wave) * 32 * W;
    const int rows = min(32, p.M - t0), b_row = 2 * p.r, s_row = F16 ? 4 * p.r : 6 * p.r;
    const int id = c < rows ? adapter(p, t0 + c) : -1;
    if (p.codes[blockIdx.y] != kApart || n0 >= p.N) return;
    const rsrc_t from_bias = bias_row(p), from_res = residual_rows(p, t0, rows);
    f16_t sum[W];
    u4_t bias[W][2], res[W][2];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const rsrc_t from = apart(p, t0, n0 + 32 * w);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int off = n0 + 32 * w < p.N ? 1024 * q + 16 * lane : kPast;
            const f4_t v = __builtin_bit_cast(f4_t, load16<0>(from, off, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[w][4 * q + e] = v[e];
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int n = Columns{n0 + 32 * w, g}.of(q);
            bias[w][q] = load16<0>(from_bias, p.bias_f32 ? kPast : 2 * n, 0);
            res[w][q] = load16<0>(from_res, n < p.N ? 2 * (c * p.N + n) : kPast, 0);
        }
    }
    const rsrc_t sr = uniform_buffer((F16 ? reinterpret_cast<const char *>(p.inner)
                                          : reinterpret_cast<const char *>(p.terms)) +
                                         static_cast<int64_t>(t0) * s_row,
                                     static_cast<int64_t>(rows) * s_row);
    // Ranks [16 Q i, 16 Q (i + 1)) in groups of 16: lane (c, g) has ranks 8 g .. + 7 of each,
    // of B's columns c and of inner's row c (bf16: of its three terms; of the last 8 ranks
    // alone the terms are side by side).
    constexpr int Q = F16 ? 2 : 4;
    struct Ranks {
        u4_t b[Q][W], s[Q][F16 ? 2 : 3];
    };
    const auto fetch = [&](rsrc_t br, int i, Ranks &v) GFR_INLINE {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k0 = 16 * (Q * i + q);
            if (k0 >= p.r) break;
            const int width = k0 + 16 <= p.r ? 16 : 8, k = k0 + (8 * g & width - 1);
            const bool live = !F16 || 8 * g < width;
#pragma unroll
            for (int w = 0; w < W; ++w)
                v.b[q][w] = load16<0>(br, live ? (c + 32 * w) * b_row + 2 * k : kPast, 0);
#pragma unroll
            for (int j = 0; j < (F16 ? 2 : 3); ++j) {
                const int at = F16 ? 4 * (k + 4 * j) : 2 * (3 * k0 + 16 * j + 8 * g);
                v.s[q][j] = load16<0>(
                    sr, F16 ? (live ? c * s_row + at : kPast)
                            : (16 * j + 8 * g < 3 * width ? c * s_row + at : kPast), 0);
            }
        }
    };
    uint64_t todo = __builtin_amdgcn_ballot_w64(id >= 0);
    while (todo) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        const bool mine = id == a;
        todo &= ~__builtin_amdgcn_ballot_w64(mine);
        const rsrc_t br = uniform_buffer(
            reinterpret_cast<const char *>(p.b + (a * int64_t{p.N} + n0) * p.r),
            static_cast<int64_t>(p.N - n0) * b_row);
        f16_t own[W];
#pragma unroll
        for (int w = 0; w < W; ++w) own[w] = sum[w];
        for (int i = 0; 16 * Q * i < p.r; ++i) {
            Ranks v;
            fetch(br, i, v);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int k0 = 16 * (Q * i + q);
                if (k0 >= p.r) break;
#pragma unroll
                for (int w = 0; w < W; ++w)
                    if (F16)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            own[w] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                                unpack1<F16>(v.b[q][w][e >> 1] >> (16 * (e & 1))),
                                __uint_as_float(v.s[q][e >> 2][e & 3]), own[w], 0, 0, 0);
                    else
#pragma unroll
                        for (int j = 0; j < 3; ++j) {
                            // (8 ranks alone: 16 terms, then 8)
                            const bool alone = k0 + 16 > p.r;
                            if (alone && j == 2) break;
                            const u4_t b =
                                alone && j == 1 && g == 1 ? u4_t{0, 0, 0, 0} : v.b[q][w];
                            own[w] = mfma32<F16>(b, v.s[q][j], own[w]);
                        }
            }
        }
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[w][e] = mine ? own[w][e] : sum[w][e];
    }
#pragma unroll
    for (int w = 0; w < W; ++w)
        put_sums<F16>(p, sum[w], t0, rows, Columns{n0 + 32 * w, g}, from_bias, bias[w], res[w],
                      lane);
}

template <bool F16>
__global__ __launch_bounds__(kWaves * 64, 1) void lora_tile_kernel(LoraParams p) {
    extern __shared__ u4_t lds[];     // [2][x's 256 rows, w's][8]
    const LoraTiles<F16> tiles(p);
    const LoraFinish<F16> finish{};
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

// The shrink by rows reads an adapter's A for each of them; from 200 MB of that, some 20
// us, on the tiles are faster (4465 rows of 2048 by rank 128 150 us).
bool shrinks_tiles(const LoraParams &p) {
    return p.K % 8 == 0 && p.r % 4 == 0 && p.M <= 32 * 65535 &&
           2.0 * p.M * p.r * p.K > 2e8;
}

template <bool F16>
hipError_t launch_shrink_tiles(const LoraParams &p, hipStream_t stream) {
    constexpr auto shrink = &shrink_tile_kernel<F16>;
    if (const hipError_t e = allow_lds<shrink, kMaxLds>(kShrinkLds); e != hipSuccess) return e;
    hipLaunchKernelGGL(shrink, dim3((p.M + 31) / 32, (p.r + 31) / 32), dim3(kShrinkWaves * 64),
                       kShrinkLds, stream, p);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_rows(const LoraParams &p, hipStream_t stream) {
    const bool many = static_cast<int64_t>(p.M) * p.r >= 8192;
    hipError_t e;
    if (shrinks_tiles(p))
        e = launch_shrink_tiles<F16>(p, stream);
    else if (p.K % 8 == 0)
        e = many ? launch_shrink_rows<F16, true, 4>(p, stream)
                 : launch_shrink_rows<F16, true, 1>(p, stream);
    else
        e = many ? launch_shrink_rows<F16, false, 4>(p, stream)
                 : launch_shrink_rows<F16, false, 1>(p, stream);
    if (e != hipSuccess) return e;
    LinearParams d{};
    d.x = p.x;
    d.w = p.w;
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
    d.partial = p.dense;
    d.keep_partial = 1;
    if (e = launch_linear(d, stream); e != hipSuccess) return e;
    // a row a block, up to about 16384 blocks
    const int columns = (p.N + 255) / 256;
    int64_t rows = (static_cast<int64_t>(p.M) * columns + 16383) / 16384;
    if (const int64_t least = (p.M + 65534) / 65535; rows < least) rows = least;
    const dim3 grid(columns, static_cast<uint32_t>((p.M + rows - 1) / rows));
    const auto kernel = p.r % 8 == 0   ? &expand_rows_kernel<F16, 8>
                        : p.r % 4 == 0 ? &expand_rows_kernel<F16, 4>
                                       : &expand_rows_kernel<F16, 1>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, p, static_cast<int>(rows));
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_tiles(const LoraParams &p, hipStream_t stream) {
    if (const hipError_t e = launch_shrink_tiles<F16>(p, stream); e != hipSuccess) return e;
    constexpr int lds = 2 * kStage * 16;
    constexpr auto kernel = &lora_tile_kernel<F16>;
    if (const hipError_t a = allow_lds<kernel, kMaxLds>(lds); a != hipSuccess) return a;
    hipLaunchKernelGGL(kernel, dim3(256), dim3(kWaves * 64), lds, stream, p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const auto expand = [&](auto kernel, int columns) {
        hipLaunchKernelGGL(kernel, dim3((p.N + columns - 1) / columns, (p.M + 31) / 32), dim3(256),
                           0, stream, p);
    };
    if (!F16 && p.r > 16) expand(&expand_tile_kernel<F16, F16 ? 1 : 2>, 256);
    else expand(&expand_tile_kernel<F16, 1>, 128);
    return hipGetLastError();
}

}  // namespace

LoraLayout lora_layout(int64_t M, int64_t N, int64_t K, int64_t r) {
    const auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    LoraLayout l{};
    // Whole tiles where they fill half of the CUs.
    l.tiles = K % 8 == 0 && N % 8 == 0 && r % 8 == 0 && M <= 32 * 65535 && N <= 1 << 21 &&
              ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile) >= 128;
    if (l.tiles) {
        l.codes = up(3 * sizeof(uint16_t) * M * r);       // (or M r floats)
        l.dense = l.codes + up(sizeof(int32_t) * ((M + 31) / 32));
        l.total = l.dense + up(sizeof(float) * 1024 * ((M + 31) / 32) * ((N + 31) / 32));
        return l;
    }
    l.choice = linear_choice(M, N, K, GFR_ACT_NONE);
    l.codes = up(sizeof(float) * M * r);
    l.dense = l.codes + up(sizeof(int32_t) * ((M + 31) / 32));
    l.total = l.dense + up(sizeof(float) * l.choice.split * M *
                           (l.choice.split > 1 ? (N + 7) / 8 * 8 : N));
    return l;
}

hipError_t launch_lora(const LoraParams &p, hipStream_t stream) {
    if (p.tiles)
        return p.f16 ? launch_tiles<true>(p, stream) : launch_tiles<false>(p, stream);
    return p.f16 ? launch_rows<true>(p, stream) : launch_rows<false>(p, stream);
}

}  // namespace gfr
