// Dense product with bias, activation and residual in its epilogue.
// include/gfr.h states the operator.
//
// Both kernels multiply bf16 or f16 on the matrix cores with FP32 sums and apply
// the epilogue to the sums in LDS, so nothing but the result goes to memory.
//
//   row kernel   up to 64 rows of a short K, v_mfma_f32_16x16x32.  The weights' bytes bound
//                it: a block takes 16 columns (for swiglu their gate and up
//                rows), its waves split K, and the sums meet in LDS; a lane
//                reads 16 bytes along K, straight into MFMA operands.  (Gate/up
//                of 4096 x 6144 with 5 rows, 101 MB: 22.1 us, 4.6 TB/s.)
//   tile kernel  more rows, v_mfma_f32_32x32x16: BM x BN tiles, 64-K steps
//                through LDS in two stages (the next step's loads are in flight
//                in registers while the present one is multiplied).  What a CU
//                takes in from L2 and LDS bounds it, so tiles are as large as
//                the size fills 256 CUs with.  (4096 x 7168 x 4096 with
//                residual: 237 us, 1.01 PFLOP/s.)  Few tiles split K; a second
//                launch then adds the partial sums and finishes.  (128 x 4096 x
//                4096: 64 x 64 tiles split two ways, 17.7 us.)  K not a multiple
//                of 8 is loaded in words and shifted: 1.6 to 2.8 times as long
//                (24 x 4096 x 4099 30 us, x 4096 18).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "gfr.h"
#include "gfr_device.h"
#include "gfr_layer.h"

namespace gfr {
namespace {

template <bool F16>
__device__ __forceinline__ f4_t mfma(u4_t a, u4_t b, f4_t c) {
    if (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, a),
                                                      __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, a),
                                                   __builtin_bit_cast(bf8_t, b), c, 0, 0, 0);
}

// Eight elements at lane_off + off bytes.  With K a multiple of 8 they are 16
// aligned bytes; otherwise rows begin at any even byte, and the four or five
// aligned words that hold them are shifted into place (no word is read that
// holds none of them).
template <bool ALIGNED, int AUX>
__device__ __forceinline__ u4_t eight(rsrc_t r, int lane_off, int off) {
    if (ALIGNED) return load16<AUX>(r, lane_off, off);
    const int at = lane_off & ~3;
    const bool odd = lane_off & 2;
    const u4_t q = load16<AUX>(r, at, off);
    const uint32_t last = __builtin_amdgcn_raw_buffer_load_b32(r, at + (odd ? 16 : 12), off, AUX);
    u4_t s;
    s[0] = __builtin_amdgcn_alignbyte(q[1], q[0], 2);
    s[1] = __builtin_amdgcn_alignbyte(q[2], q[1], 2);
    s[2] = __builtin_amdgcn_alignbyte(q[3], q[2], 2);
    s[3] = __builtin_amdgcn_alignbyte(last, q[3], 2);
    return odd ? s : q;
}

// The same with only the first `valid` elements, and zeros behind them.
template <bool ALIGNED>
__device__ __forceinline__ u4_t eight_tail(rsrc_t r, int lane_off, int off, int valid) {
    u4_t s = {0, 0, 0, 0};
    if (ALIGNED) {
        if (valid > 0) s = load16<0>(r, lane_off, off);
        return s;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < valid)
            s[i >> 1] |= static_cast<uint32_t>(
                             __builtin_amdgcn_raw_buffer_load_b16(r, lane_off + 2 * i, off, 0))
                         << (16 * (i & 1));
    return s;
}

// Lane offset past every buffer's end (K <= 2^21): loads there give zeros.
constexpr int kNowhere = 0x7f000000;

// Buffer over weight rows [first, first + rows).  Its base has to be a whole
// word's address, which the first row's is not where first and K are odd:
// returns the bytes from the base to the row.
template <bool ALIGNED>
__device__ __forceinline__ int weight_rows(const LinearParams &p, int64_t first, int64_t rows,
                                           rsrc_t &r) {
    const int skew = ALIGNED ? 0 : static_cast<int>(first * p.K & 1);
    r = buffer(p.w + (first * p.K - skew), rows * p.K * 2 + 2 * skew);
    return 2 * skew;
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
    case GFR_ACT_RELU: return v < 0.0f ? 0.0f : v;
    case GFR_ACT_SILU: return silu(v);
    case GFR_ACT_GELU:
        // (1 + erf x) / 2 = erfc(-x) / 2: no cancellation for negative v
        return 0.5f * v * erfcf(v * -0.70710678118654752f);
    case GFR_ACT_GELU_TANH: {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2u)): no cancellation for negative u
        const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);
        return v * __builtin_amdgcn_rcpf(1.0f + exp_f32(-2.0f * u));
    }
    default: return v;
    }
}

__device__ __forceinline__ void activate8(float (&y)[8], int act) {
    if (act == GFR_ACT_NONE) return;
#define GFR_ALL8(A)                                           \
    case A:                                                   \
        _Pragma("unroll") for (int j = 0; j < 8; ++j) y[j] = activate(y[j], A); \
        return;
    switch (act) {
        GFR_ALL8(GFR_ACT_RELU)
        GFR_ALL8(GFR_ACT_SILU)
        GFR_ALL8(GFR_ACT_GELU)
        GFR_ALL8(GFR_ACT_GELU_TANH)
    }
#undef GFR_ALL8
}

__device__ __forceinline__ float element(const void *p, int64_t i, bool f32, bool f16) {
    if (f32) return static_cast<const float *>(p)[i];
    const uint16_t h = static_cast<const uint16_t *>(p)[i];
    return f16 ? static_cast<float>(__builtin_bit_cast(_Float16, h)) : bf16_f32(h);
}

// y = act(v + bias) (swiglu: silu(gate + its bias) * (v + bias)) of column n.
template <bool SWIGLU, bool F16>
__device__ __forceinline__ float finish1(const LinearParams &p, int n, float v, float gate) {
    if (p.bias) {
        v += element(p.bias, n + (SWIGLU ? p.N : 0), p.bias_f32, F16);
        if (SWIGLU) gate += element(p.bias, n, p.bias_f32, F16);
    }
    return SWIGLU ? silu(gate) * v : activate(v, p.act);
}

template <bool F16>
__device__ __forceinline__ void store1(const LinearParams &p, int64_t at, float y) {
    if (p.out_f32)
        static_cast<float *>(p.out)[at] = y;
    else
        static_cast<uint16_t *>(p.out)[at] = static_cast<uint16_t>(
            F16 ? pack_f16(y, 0.0f) : pack_bf16(y, 0.0f));
}

// Eight finished columns (16-byte aligned rows: p.wide).
template <bool F16>
__device__ __forceinline__ void store8(const LinearParams &p, int64_t at, const float (&y)[8]) {
    if (p.out_f32) {
        float *out = static_cast<float *>(p.out) + at;
        *reinterpret_cast<f4_t *>(out) = f4_t{y[0], y[1], y[2], y[3]};
        *reinterpret_cast<f4_t *>(out + 4) = f4_t{y[4], y[5], y[6], y[7]};
    } else {
        u4_t h;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = F16 ? pack_f16(y[2 * j], y[2 * j + 1]) : pack_bf16(y[2 * j], y[2 * j + 1]);
        *reinterpret_cast<u4_t *>(static_cast<uint16_t *>(p.out) + at) = h;
    }
}

template <bool F16>
__device__ __forceinline__ void add8(float (&y)[8], u4_t h) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint16_t b = h[j >> 1] >> (16 * (j & 1));
        y[j] += F16 ? static_cast<float>(__builtin_bit_cast(_Float16, b)) : bf16_f32(b);
    }
}

// Columns n .. n + 7 of row m (p.wide): the whole epilogue.
template <bool SWIGLU, bool F16>
__device__ __forceinline__ void finish8(const LinearParams &p, int m, int n, const float (&v)[8],
                                        const float (&gate)[8]) {
    const int64_t at = static_cast<int64_t>(m) * p.N + n;
    u4_t h = {0, 0, 0, 0};
    if (p.residual) h = load<u4_t>(p.residual + at);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = finish1<SWIGLU, F16>(p, n + j, v[j], gate[j]);
    if (p.residual) add8<F16>(y, h);
    store8<F16>(p, at, y);
}

// ---------------------------------------------------------------------------
// Row kernel
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 512;
constexpr int kRowWaves = kRowThreads / 64;

// RG fragments of 16 rows, NF of 16 weight rows (1, or 2 for swiglu: gate and up).
// Weight lines come whole and are swapped into operands: half lines took 25.3 us
// where whole ones take 22.1 (gate/up of 4096 x 6144, 5 rows).
template <bool F16, bool ALIGNED, bool SWIGLU, int RG, int NF>
__global__ __launch_bounds__(kRowThreads) void row_kernel(LinearParams p) {
    static_assert(NF == (SWIGLU ? 2 : 1), "16 columns a block");
    constexpr int kTile = 16 * NF, kDepth = RG == 1 ? 4 : RG == 2 ? 3 : 2;
    __shared__ float tiles[kRowWaves][16 * RG][kTile];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int64_t bytes = 2 * static_cast<int64_t>(p.K);   // of a row
    rsrc_t wr[NF];
    int w_off[NF][2], x_off[RG];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        // (columns past the end read the last one's row)
        const int last = p.N - 1 - n0;
        const int skew = weight_rows<ALIGNED>(p, f ? int64_t{n0} + p.N : n0, last + 1, wr[f]);
        // whole lines, swapped into operands (swap_halves), or each lane's own piece
        for (int b = 0; b < 2; ++b)
            w_off[f][b] = ALIGNED ? min((c & 7) + 8 * b, last) * static_cast<int>(bytes) +
                                        16 * (g + 4 * (c >> 3))
                                  : min(c, last) * static_cast<int>(bytes) + 16 * g +
                                        64 * b + skew;
    }
    const rsrc_t xr = buffer(p.x, p.M * bytes);
#pragma unroll
    for (int q = 0; q < RG; ++q)
        x_off[q] = min(16 * q + c, p.M - 1) * static_cast<int>(bytes) + 16 * g;

    struct Stage {
        u4_t w[NF][2], x[RG][2];
    } st[kDepth];
    f4_t acc[RG][NF] = {};
    const int steps = p.K / 64;
    const int s0 = steps * wave / kRowWaves, s1 = steps * (wave + 1) / kRowWaves;
    auto fetch = [&](Stage &s, int step) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int f = 0; f < NF; ++f)
                s.w[f][h] = eight<ALIGNED, kNt>(wr[f], w_off[f][h], step * 128);
#pragma unroll
            for (int q = 0; q < RG; ++q)
                s.x[q][h] = eight<ALIGNED, 0>(xr, x_off[q], step * 128 + 64 * h);
        }
    };
    auto use = [&](Stage &s, bool swapped) {
        if (ALIGNED && swapped)
#pragma unroll
            for (int f = 0; f < NF; ++f) swap_halves(s.w[f][0], s.w[f][1]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int q = 0; q < RG; ++q)
                    acc[q][f] = mfma<F16>(s.x[q][h], s.w[f][h], acc[q][f]);
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if (s0 + d < s1) fetch(st[d], s0 + d);
    for (int s = s0; s < s1; s += kDepth)
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            if (s + d < s1) {
                use(st[d], true);
                if (s + d + kDepth < s1) fetch(st[d], s + d + kDepth);
            }
    if (wave == kRowWaves - 1 && p.K % 64 != 0) {
        const int own_off = min(c, p.N - 1 - n0) * static_cast<int>(bytes) + 16 * g;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int valid = p.K - (64 * steps + 32 * h + 8 * g);
#pragma unroll
            for (int f = 0; f < NF; ++f)
                st[0].w[f][h] = eight_tail<ALIGNED>(
                    wr[f], ALIGNED ? own_off : w_off[f][0], steps * 128 + 64 * h, valid);
#pragma unroll
            for (int q = 0; q < RG; ++q)
                st[0].x[q][h] = eight_tail<ALIGNED>(xr, x_off[q], steps * 128 + 64 * h, valid);
        }
        use(st[0], false);
    }
#pragma unroll
    for (int q = 0; q < RG; ++q)
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                tiles[wave][16 * q + 4 * g + i][16 * f + c] = acc[q][f][i];
    __syncthreads();
    const int rows = min(p.M, 16 * RG);
    for (int i = threadIdx.x; i < rows * 16; i += kRowThreads) {
        const int m = i / 16, col = i % 16, n = n0 + col;
        if (n >= p.N) continue;
        const int64_t at = static_cast<int64_t>(m) * p.N + n;
        const float r = p.residual ? element(p.residual, at, false, F16) : 0.0f;
        float v = 0.0f, gate = 0.0f;
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) {
            v += tiles[w][m][SWIGLU ? 16 + col : col];
            if (SWIGLU) gate += tiles[w][m][col];
        }
        float y = finish1<SWIGLU, F16>(p, n, v, gate);
        if (p.residual) y += r;
        store1<F16>(p, at, y);
    }
}

// ---------------------------------------------------------------------------
// Tile kernel
// ---------------------------------------------------------------------------
typedef float f16_t __attribute__((ext_vector_type(16)));

template <bool F16>
__device__ __forceinline__ f16_t mfma32(u4_t a, u4_t b, f16_t c) {
    if (F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8_t, a),
                                                      __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8_t, a),
                                                   __builtin_bit_cast(bf8_t, b), c, 0, 0, 0);
}

// LDS bytes of a tile: two stages, or the waves' rows of the epilogue.
constexpr int tile_lds(int bm, int bn, int wm, int wn, bool swiglu) {
    const int stages = 2 * (bm + bn) * 8 * 16;
    const int rows = bm / wm * (bn / wn) * (32 * (wn + 4) + 16 * (swiglu ? wn / 2 : wn)) * 4;
    return stages > rows ? stages : rows;
}

// Every LDS access of this wave has finished, then the other waves' too.  (As
// __syncthreads, but the loads from memory in flight stay in flight.)
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Spreads a part's LDS reads, LDS writes and memory loads over its MFMAs (as the
// compiler would leave them, they come in runs that the MFMAs wait for).
template <int MFMAS, int READS, int WRITES, int LOADS>
__device__ __forceinline__ void spread() {
    constexpr int kTurns = MFMAS > 1 ? MFMAS / 2 : 1;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        // reads in the first half: their latency runs under the second
        constexpr int kR = (READS * 2 + kTurns - 1) / kTurns;
        constexpr int kW = (WRITES + kTurns - 1) / kTurns, kL = (LOADS + kTurns - 1) / kTurns;
        if (READS && i * kR < READS) __builtin_amdgcn_sched_group_barrier(0x100, kR, 0);
        if (WRITES && i * kW < WRITES) __builtin_amdgcn_sched_group_barrier(0x200, kW, 0);
        if (LOADS && i * kL < LOADS) __builtin_amdgcn_sched_group_barrier(0x20, kL, 0);
        __builtin_amdgcn_sched_group_barrier(0x8, MFMAS / kTurns, 0);
    }
}

// BM rows of x by BN weight rows (swiglu: BN / 2 output columns, their gate and
// up rows in turn by fragments of 32), four waves of WM x WN.  In LDS a row of 64
// elements is eight 16-byte pieces, piece j of row r at j ^ (r & 7), so that
// eight lanes that read one piece of eight rows reach all banks.
//
// A step is four 16-K parts.  While one part's MFMAs run, the next part's
// fragments come from LDS.  The next step's tile, loaded to registers three parts
// (with two steps on their way: seven) earlier, is written to the other stage
// during parts 1 (x) and 2 (w), and each half's loads of a later step follow at
// once.  The one barrier stands before part 3, whose fragments are in registers
// by then: behind it the other stage is complete, and nobody reads this one any
// more.
template <bool F16, bool ALIGNED, bool SWIGLU, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, BM == 256 ? BM / WM * (BN / WN) / 4 : 2)
void tile_kernel(LinearParams p, int tiles_m, int tiles_n) {
    constexpr int kWaves = (BM / WM) * (BN / WN), kThreads = kWaves * 64, kRowsPer = kThreads / 8;
    constexpr int kNX = BM * 8 / kThreads, kNW = BN * 8 / kThreads;   // pieces per thread
    constexpr int FM = WM / 32, FN = WN / 32;
    extern __shared__ u4_t lds[];                  // [2][BM + BN][8]
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 31, g = lane >> 5;
    // Blocks go round the eight XCDs; each XCD takes a run of tiles, eight
    // tile rows deep, so that its L2 serves their shared operands.
    const int total = tiles_m * tiles_n, per = (total + 7) / 8;
    const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= per || id >= total) return;
    const int band = id / (8 * tiles_n), in_band = id - band * 8 * tiles_n;
    const int depth = min(8, tiles_m - band * 8);
    const int m0 = (band * 8 + in_band % depth) * BM;
    const int n0 = in_band / depth * (SWIGLU ? BN / 2 : BN);

    const int64_t bytes = 2 * static_cast<int64_t>(p.K);
    const rsrc_t xr = buffer(p.x + m0 * static_cast<int64_t>(p.K), min(BM, p.M - m0) * bytes);
    rsrc_t wr, ur;
    const int rows = min(SWIGLU ? BN / 2 : BN, p.N - n0);
    weight_rows<ALIGNED>(p, n0, rows, wr);          // n0 is even: no skew
    const int skew = weight_rows<ALIGNED>(p, SWIGLU ? int64_t{n0} + p.N : n0, rows, ur);
    int x_off[kNX], w_off[kNW];
    const int piece = threadIdx.x & 7, row0 = threadIdx.x >> 3;
#pragma unroll
    for (int i = 0; i < kNX; ++i)
        x_off[i] = min(row0 + kRowsPer * i, p.M - 1 - m0) * static_cast<int>(bytes) + 16 * piece;
    // (a wave holds eight rows of a pass: all gate or all up rows)
    auto is_up = [&](int i) { return SWIGLU && (uniform(row0) + kRowsPer * i & 32); };
#pragma unroll
    for (int i = 0; i < kNW; ++i) {
        const int r = row0 + kRowsPer * i, row = SWIGLU ? (r >> 6) * 32 + (r & 31) : r;
        w_off[i] = min(row, p.N - 1 - n0) * static_cast<int>(bytes) + 16 * piece +
                   (is_up(i) ? skew : 0);
    }
    // rows a multiple of 8 apart share their swizzle
    u4_t *const put_at = lds + row0 * 8 + (piece ^ (row0 & 7));
    // Steps' tiles on their way: two where the registers leave room (a step of
    // the smaller tiles is shorter than a load takes: 256 x 4096 x 4096 30 us
    // with one, 20 with two).
    constexpr int D = BM * BN < 256 * 256 ? 2 : 1;
    u4_t xs[D][kNX], ws[D][kNW];
    // this block's steps: all, or a K split's
    const int all = (p.K + 63) / 64, sp = blockIdx.y;
    const int s0 = all * sp / p.split, steps = all * (sp + 1) / p.split - s0;
    // x's or w's pieces of a step (behind the last step: zeros)
    auto fetch = [&](auto &to, const auto &offs, auto which, int step) {
        constexpr int n = sizeof(to) / sizeof(to[0]);
        step += s0;
        const int off = step * 128, valid = p.K - step * 64 - 8 * piece;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const rsrc_t r = which(i);
            if (ALIGNED)
                // pieces behind K: zeros, from behind the buffer's end
                to[i] = load16<0>(r, valid > 0 ? offs[i] : kNowhere, off);
            else
                to[i] = step * 64 + 64 <= p.K ? eight<false, 0>(r, offs[i], off)
                                              : eight_tail<false>(r, offs[i], off, valid);
        }
    };
    auto fetch_x = [&](auto set, int step) {
        fetch(xs[set], x_off, [&](int) { return xr; }, step);
    };
    auto fetch_w = [&](auto set, int step) {
        fetch(ws[set], w_off, [&](int i) { return is_up(i) ? ur : wr; }, step);
    };
    const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;
    const u4_t *const x_at = lds + (wm + c) * 8, *const w_at = lds + (BM + wn + c) * 8;
    constexpr int kStage = (BM + BN) * 8;
    u4_t a[2][FM], b[2][FN];
    auto get = [&](int to, int stage, int part) {
        const int at = stage * kStage + ((2 * part + g) ^ (c & 7));
#pragma unroll
        for (int i = 0; i < FM; ++i) a[to][i] = x_at[at + 32 * 8 * i];
#pragma unroll
        for (int j = 0; j < FN; ++j) b[to][j] = w_at[at + 32 * 8 * j];
    };
    f16_t acc[FM][FN] = {};
    auto multiply = [&](int from) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = mfma32<F16>(b[from][j], a[from][i], acc[i][j]);
    };
    auto put_x = [&](auto set, int stage) {
#pragma unroll
        for (int i = 0; i < kNX; ++i) put_at[stage * kStage + kRowsPer * 8 * i] = xs[set][i];
    };
    auto put_w = [&](auto set, int stage) {
#pragma unroll
        for (int i = 0; i < kNW; ++i) put_at[stage * kStage + (BM + kRowsPer * i) * 8] = ws[set][i];
    };
    const std::integral_constant<int, 0> s0_{};
    const std::integral_constant<int, D - 1> s1_{};
    fetch_x(s0_, 0);
    fetch_w(s0_, 0);
    if (D == 2) fetch_x(s1_, 1), fetch_w(s1_, 1);
    put_x(s0_, 0);
    put_w(s0_, 0);
    fetch_x(s0_, D);
    fetch_w(s0_, D);
    lds_barrier();
    get(0, 0, 0);
    // One step; the next one's tile is in set `next`, which then takes the one D
    // steps behind that.
    auto run_step = [&](int step, auto next) {
        const int cur = step & 1;
        get(1, cur, 1);
        multiply(0);
        spread<FM * FN, FM + FN, 0, 0>();
        get(0, cur, 2);
        put_x(next, cur ^ 1);
        multiply(1);
        spread<FM * FN, FM + FN, kNX, 0>();
        get(1, cur, 3);
        fetch_x(next, step + 1 + D);
        put_w(next, cur ^ 1);
        multiply(0);
        spread<FM * FN, FM + FN, kNW, kNX>();
        lds_barrier();
        get(0, cur ^ 1, 0);
        fetch_w(next, step + 1 + D);
        multiply(1);
        spread<FM * FN, FM + FN, 0, kNW>();
    };
    if (D == 1) {
        for (int step = 0; step + 1 < steps; ++step) run_step(step, s0_);
    } else {
        int step = 0;
        for (; step + 2 < steps; step += 2) {
            run_step(step, s1_);
            run_step(step + 1, s0_);
        }
        if (step + 1 < steps) run_step(step, s1_);
    }
    const int cur = (steps - 1) & 1;
    get(1, cur, 1);
    multiply(0);
    get(0, cur, 2);
    multiply(1);
    get(1, cur, 3);
    multiply(0);
    multiply(1);
    // Lane (c, g) holds row 32 i + c, columns 32 j + 8 r + 4 g .. + 3, r < 4.  32 rows
    // at a time go through LDS (the wave's own part of the stages), so that the
    // epilogue reads and writes whole runs of columns.
    constexpr int kPitch = WN + 4;     // spreads the rows over the banks
    constexpr int kCols = SWIGLU ? WN / 2 : WN;
    constexpr int kSlab = 32 * kPitch + 16 * kCols;    // floats: sums, then residual rows
    static_assert(kWaves * kSlab * 4 <= tile_lds(BM, BN, WM, WN, SWIGLU), "the waves' rows fit");
    float *slab = reinterpret_cast<float *>(lds) + wave * kSlab;
    u4_t *res_at = reinterpret_cast<u4_t *>(slab + 32 * kPitch);
    const int col0 = n0 + (SWIGLU ? wn / 2 : wn);
    auto put_sums = [&](int i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<f4_t *>(&slab[c * kPitch + 32 * j + 8 * r + 4 * g]) =
                    f4_t{acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2],
                         acc[i][j][4 * r + 3]};
    };
    auto wave_sync = [] {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    lds_barrier();
    if (p.split > 1) {
        // partial sums [split][M][gate,] up, eight-column rows
        const int pitch = (p.N + 7) / 8 * 8, width = SWIGLU ? 2 * pitch : pitch;
        constexpr int kLanes = kCols / 8, kRows = 64 / kLanes;
        const int er = lane / kLanes, col = lane % kLanes * 8, n = col0 + col;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int first = m0 + wm + 32 * i;
            if (first >= p.M) break;
            put_sums(i);
            wave_sync();
#pragma unroll 2
            for (int r = er; r < 32; r += kRows) {
                if (first + r >= p.M || n >= p.N) continue;
                float *to = p.partial + (static_cast<int64_t>(sp) * p.M + first + r) * width + n;
                const float *at = slab + r * kPitch + (SWIGLU ? (col >> 5) * 64 + (col & 31) : col);
#pragma unroll
                for (int h = 0; h < (SWIGLU ? 2 : 1); ++h)
#pragma unroll
                    for (int j = 0; j < 8; j += 4)
                        *reinterpret_cast<f4_t *>(to + h * pitch + j) = load<f4_t>(at + 32 * h + j);
            }
            wave_sync();
        }
        return;
    }
    if (p.wide) {
        // Eight columns per lane, the same ones in every row it takes: their
        // bias is loaded once, and the next 32 rows' residual while these are
        // finished.  (With both loaded where they are used a 4096 x 7168 x 4096
        // product took 130 us longer: one wave per SIMD hides no latency.)
        constexpr int kLanes = kCols / 8, kRows = 64 / kLanes, kTurns = 32 / kRows;
        const int er = lane / kLanes, n = col0 + lane % kLanes * 8;
        const bool in = n < p.N;
        float bias[8] = {}, gate_bias[8] = {};
        if (p.bias && in)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                bias[j] = element(p.bias, n + j + (SWIGLU ? p.N : 0), p.bias_f32, F16);
                if (SWIGLU) gate_bias[j] = element(p.bias, n + j, p.bias_f32, F16);
            }
        u4_t res[kTurns];
        auto fetch_res = [&](int i) {
            const int first = m0 + wm + 32 * i + er;
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                const int64_t m = min(first + k * kRows, p.M - 1);
                if (in) res[k] = load<u4_t>(p.residual + m * p.N + n);
            }
        };
        if (p.residual) fetch_res(0);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int first = m0 + wm + 32 * i;
            if (first >= p.M) break;
            put_sums(i);
            if (p.residual) {
#pragma unroll
                for (int k = 0; k < kTurns; ++k) res_at[k * 64 + lane] = res[k];
                if (i + 1 < FM) fetch_res(i + 1);
            }
            wave_sync();
#pragma unroll 2
            for (int k = 0; k < kTurns; ++k) {
                const int r = k * kRows + er, m = first + r;
                if (m >= p.M || !in) continue;
                const float *at = slab + r * kPitch;
                const int col = lane % kLanes * 8;
                const float *up = at + (SWIGLU ? (col >> 5) * 64 + 32 + (col & 31) : col);
                const float *gate = at + (col >> 5) * 64 + (col & 31);
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const f4_t v = load<f4_t>(up + j);
                    if (SWIGLU) {
                        const f4_t gt = load<f4_t>(gate + j);
#pragma unroll
                        for (int l = 0; l < 4; ++l)
                            y[j + l] = silu(gt[l] + gate_bias[j + l]) * (v[l] + bias[j + l]);
                    } else {
#pragma unroll
                        for (int l = 0; l < 4; ++l) y[j + l] = v[l] + bias[j + l];
                    }
                }
                if (!SWIGLU) activate8(y, p.act);
                if (p.residual) add8<F16>(y, res_at[k * 64 + lane]);
                store8<F16>(p, static_cast<int64_t>(m) * p.N + n, y);
            }
            wave_sync();
        }
        return;
    }
    // Rows that begin anywhere: a column per lane, eight rows' residual ahead.
    static_assert(kCols <= 64, "a lane keeps its column");
    constexpr int kRows = 64 / kCols, kTurns = 32 / kRows;
    const int er = lane / kCols, col = lane % kCols, n = col0 + col;
    const bool in = n < p.N;
    const float bias = p.bias && in ? element(p.bias, n + (SWIGLU ? p.N : 0), p.bias_f32, F16) : 0;
    const float gate_bias = SWIGLU && p.bias && in ? element(p.bias, n, p.bias_f32, F16) : 0;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int first = m0 + wm + 32 * i;
        if (first >= p.M) break;
        put_sums(i);
        wave_sync();
#pragma unroll 1
        for (int k = 0; k < kTurns; k += 8) {
            float y[8];
            uint16_t res[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t m = min(first + (k + j) * kRows + er, p.M - 1);
                res[j] = 0;
                if (p.residual && in) res[j] = p.residual[m * p.N + n];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float *at = slab + ((k + j) * kRows + er) * kPitch;
                if (SWIGLU) {
                    const int c0 = (col >> 5) * 64 + (col & 31);
                    y[j] = silu(at[c0] + gate_bias) * (at[c0 + 32] + bias);
                } else {
                    y[j] = at[col] + bias;
                }
            }
            if (!SWIGLU) activate8(y, p.act);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int m = first + (k + j) * kRows + er;
                if (m >= p.M || !in) continue;
                if (p.residual)
                    y[j] += F16 ? static_cast<float>(__builtin_bit_cast(_Float16, res[j]))
                                : bf16_f32(res[j]);
                store1<F16>(p, static_cast<int64_t>(m) * p.N + n, y[j]);
            }
        }
        wave_sync();
    }
}

// Adds up a split's partial sums, in order, and finishes eight columns per thread
// (one where rows begin anywhere).
template <bool SWIGLU, bool F16>
__global__ __launch_bounds__(256) void join_kernel(LinearParams p) {
    const int pitch = (p.N + 7) / 8 * 8, width = SWIGLU ? 2 * pitch : pitch;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (!p.wide) {
        if (i >= static_cast<int64_t>(p.M) * p.N) return;
        const int m = static_cast<int>(i / p.N), n = static_cast<int>(i % p.N);
        const float *at = p.partial + static_cast<int64_t>(m) * width + n;
        const int64_t plane = static_cast<int64_t>(p.M) * width;
        const float r = p.residual ? element(p.residual, i, false, F16) : 0.0f;
        float v = 0.0f, gate = 0.0f;
#pragma unroll 2
        for (int s = 0; s < p.split; ++s, at += plane) {
            v += at[SWIGLU ? pitch : 0];
            if (SWIGLU) gate += at[0];
        }
        float y = finish1<SWIGLU, F16>(p, n, v, gate);
        if (p.residual) y += r;
        store1<F16>(p, i, y);
        return;
    }
    if (i >= static_cast<int64_t>(p.M) * (pitch / 8)) return;
    const int m = static_cast<int>(i / (pitch / 8)), n = static_cast<int>(i % (pitch / 8)) * 8;
    const float *at = p.partial + static_cast<int64_t>(m) * width + n;
    const int64_t plane = static_cast<int64_t>(p.M) * width;
    f4_t v[2] = {}, gate[2] = {};
#pragma unroll 2
    for (int s = 0; s < p.split; ++s, at += plane)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v[h] += load<f4_t>(at + (SWIGLU ? pitch : 0) + 4 * h);
            if (SWIGLU) gate[h] += load<f4_t>(at + 4 * h);
        }
    const float a[8] = {v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
    const float g[8] = {gate[0][0], gate[0][1], gate[0][2], gate[0][3],
                        gate[1][0], gate[1][1], gate[1][2], gate[1][3]};
    finish8<SWIGLU, F16>(p, m, n, a, g);
}

template <bool F16, bool ALIGNED, bool SWIGLU, int RG>
hipError_t launch_rows(const LinearParams &p, hipStream_t stream) {
    hipLaunchKernelGGL((row_kernel<F16, ALIGNED, SWIGLU, RG, SWIGLU ? 2 : 1>),
                       dim3((p.N + 15) / 16), dim3(kRowThreads), 0, stream, p);
    return hipGetLastError();
}

template <bool F16, bool ALIGNED, bool SWIGLU, int BM, int BN, int WM, int WN>
hipError_t launch_tiles(const LinearParams &p, hipStream_t stream) {
    constexpr int lds = tile_lds(BM, BN, WM, WN, SWIGLU);
    constexpr int cols = SWIGLU ? BN / 2 : BN;
    constexpr auto kernel = &tile_kernel<F16, ALIGNED, SWIGLU, BM, BN, WM, WN>;
    if (hipError_t e = allow_lds<kernel>(lds); e != hipSuccess) return e;
    const int tm = (p.M + BM - 1) / BM, tn = (p.N + cols - 1) / cols;
    const int64_t grid = (static_cast<int64_t>(tm) * tn + 7) / 8 * 8;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(grid), p.split),
                       dim3((BM / WM) * (BN / WN) * 64), lds, stream, p, tm, tn);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || p.split == 1 || p.keep_partial)
        return e;
    const int64_t threads = static_cast<int64_t>(p.M) * (p.wide ? (p.N + 7) / 8 : p.N);
    hipLaunchKernelGGL((join_kernel<SWIGLU, F16>),
                       dim3(static_cast<uint32_t>((threads + 255) / 256)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

// The kernel for a size and its K split, by estimated time.  Tiles: rounds of 256
// blocks times a block's time per 64-K step (measured at K = 4096: a larger tile
// feeds more MFMAs per byte brought to the CU), and for a split the partial sums'
// traffic at 4 TB/s and the joining launch.  Rows: a wave's eighth of the steps,
// each about as long as its loads take, times the blocks per CU.  Neither is faster
// than the weights come at 4.5 TB/s.  (Rows against
// tiles, N x K: 1 x 4096 x 4096 9.3 us against 11; 16 x 256 x 7168 15.1 against
// 9.5; 32 x 1024 x 1024 5.3 against 7.0; 64 x 4096 x 4096 21.3 against 13.0.)
constexpr int64_t kMaxBlocks = (int64_t{1} << 23) - 8;    // 2^32 threads, up to 512 a block
LinearChoice choose_kernel(int64_t M, int64_t N, int64_t K, bool swiglu) {
    typedef LinearChoice Choice;
    const int64_t rows = swiglu ? 2 * N : N, steps = (K + 63) / 64;
    const bool aligned = K % 8 == 0;
    struct Tile {
        Choice::Kernel kernel;
        int64_t bm, bn;
        double us;     // per step
    };
    const Tile tiles[] = {{Choice::k256, 256, 256, 1.65},
                          {Choice::k256x128, 256, 128, 0.95},
                          {Choice::k128, 128, 128, 0.62},
                          {Choice::k64, 64, swiglu ? 128 : 64, swiglu ? 0.42 : 0.28}};
    Choice best{Choice::k64, 0};
    double least = 1e30;
    const double memory = 2.0 * static_cast<double>(rows) * static_cast<double>(K) / 4.5e6;
    // (the longer of the two hides most of the other)
    auto both = [](double a, double b) { return a > b ? a + 0.2 * b : b + 0.2 * a; };
    if (const int64_t n = (N + 15) / 16; M <= 64 && n <= kMaxBlocks) {
        const double step = (M <= 16 ? 1.0 : M <= 32 ? 1.5 : 2.3) * (swiglu ? 1.6 : 1.0);
        least = both(2.0 + step * static_cast<double>((steps + 7) / 8) *
                               (n > 256 ? static_cast<double>(n) / 256.0 : 1.0),
                     memory);
        best = {Choice::kRows, 1};
    }
    for (const Tile &t : tiles) {
        if (!aligned && (t.kernel == Choice::k256 || t.kernel == Choice::k256x128)) continue;
        const int64_t n = ((M + t.bm - 1) / t.bm) * ((rows + t.bn - 1) / t.bn);
        if (n > kMaxBlocks) continue;
        for (int split = 1; split <= (t.kernel == Choice::k128 || t.kernel == Choice::k64 ? 8 : 1);
             ++split) {
            if (split > 1 && (steps / split < 6 || n * split > 256)) break;
            const double rounds = static_cast<double>((n * split + 255) / 256);
            double us = rounds * (4.0 + t.us * static_cast<double>((steps + split - 1) / split));
            us = both(us, 2.0 + memory);
            if (split > 1) us += 2.0 + 8.0 * static_cast<double>(M * rows * split) / 4e6;
            if (us < least) least = us, best = {t.kernel, split};
        }
    }
    return best;
}

template <bool F16, bool ALIGNED, bool SWIGLU>
hipError_t launch_linear_t(const LinearParams &p, hipStream_t stream) {
    switch (p.kernel) {
    case LinearChoice::kRows:
        if (p.M <= 16) return launch_rows<F16, ALIGNED, SWIGLU, 1>(p, stream);
        if (p.M <= 32) return launch_rows<F16, ALIGNED, SWIGLU, 2>(p, stream);
        return launch_rows<F16, ALIGNED, SWIGLU, 4>(p, stream);
    case LinearChoice::k256:
        if constexpr (ALIGNED)
            return launch_tiles<F16, ALIGNED, SWIGLU, 256, 256, 128, 64>(p, stream);
        return hipErrorInvalidValue;
    case LinearChoice::k256x128:
        if constexpr (ALIGNED)
            return launch_tiles<F16, ALIGNED, SWIGLU, 256, 128, 64, 64>(p, stream);
        return hipErrorInvalidValue;
    case LinearChoice::k128:
        return launch_tiles<F16, ALIGNED, SWIGLU, 128, 128, 64, 64>(p, stream);
    default:
        return launch_tiles<F16, ALIGNED, SWIGLU, 64, SWIGLU ? 128 : 64, 32, SWIGLU ? 64 : 32>(
            p, stream);
    }
}

template <bool F16, bool ALIGNED>
hipError_t launch_linear_a(const LinearParams &p, hipStream_t stream) {
    return p.act == GFR_ACT_SWIGLU ? launch_linear_t<F16, ALIGNED, true>(p, stream)
                                   : launch_linear_t<F16, ALIGNED, false>(p, stream);
}

}  // namespace

LinearChoice linear_choice(int64_t M, int64_t N, int64_t K, int act) {
    return choose_kernel(M, N, K, act == GFR_ACT_SWIGLU);
}

hipError_t launch_linear(const LinearParams &p, hipStream_t stream) {
    const bool aligned = p.K % 8 == 0;
    if (p.f16)
        return aligned ? launch_linear_a<true, true>(p, stream)
                       : launch_linear_a<true, false>(p, stream);
    return aligned ? launch_linear_a<false, true>(p, stream)
                   : launch_linear_a<false, false>(p, stream);
}

}  // namespace gfr
