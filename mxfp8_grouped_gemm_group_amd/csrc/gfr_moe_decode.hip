// The experts of a MoE block for a few tokens, in two launches.
// include/gfr.h states the operator.
//
// At these token counts the bytes of the chosen experts' weights bound the
// time: each is read once, in FP8, and turned into bf16 MFMA operands in
// registers (v_cvt_scalef32_pk_bf16_*, which multiplies by the block's E8M0
// scale on the way; exact, since bf16 has more mantissa bits than FP8 and E8M0's
// exponent range).  The pairs (token, expert) of one expert are the rows of
// v_mfma_f32_16x16x32_bf16, 16 to a fragment.
//
//   gate_up_kernel  h[pair, :] = silu(x w13_gate) * (x w13_up), stored as the
//                   sum of two bf16 terms (16 mantissa bits), so that feeding
//                   it to the MFMAs does not round it to one;
//   down_kernel     y[pair, n] = weight * h w2, FP32; the last block to finish
//                   a column tile adds each token's pairs in order, and the
//                   shared term, and rounds once.
//
// A unit is (group of up to 16 RG pairs of one expert, column tile, and in the
// down product a K range); blocks of eight waves take units in turn.  The
// waves of a block split the unit's K (gate_up_kernel: four K ranges for the
// gate and four for the up columns) and their sums meet in LDS, so even one
// token's few experts keep all CUs' loads in flight.
//
// Weights [K, N]: a lane reads 8 columns of 8 rows (128-byte row pieces per
// wave) and v_perm pairs the rows, so the K-major operands come together in
// registers, without LDS.  Weights [N, K]: 16 bytes along K per lane.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gfr.h"
#include "gfr_device.h"
#include "gfr_layer.h"

namespace gfr {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxPairs = 1024;

// ---------------------------------------------------------------------------
// Plan: the pairs grouped by expert.  Every block makes its own from the ids
// (a launch to make it once would cost more).  Within a group the order of the
// pairs is left to the atomics: each is a row of its own, so no result depends
// on it.  Which group of an expert a pair falls into must be the same in every
// block, so where an expert has several groups the ranks are counted instead.
// ---------------------------------------------------------------------------
struct Plan {
    int start[GFR_MAX_EXPERTS];        // counts, then first index into pairs
    uint16_t pairs[kMaxPairs];         // grouped by expert
    uint16_t expert[kMaxPairs];        // per group
    uint16_t first[kMaxPairs];         // index into pairs
    uint16_t count[kMaxPairs];
    uint16_t ids[kMaxPairs];           // only if an expert has several groups
    uint32_t totals[kWaves];
    int groups;
    int several;
    int last;                          // down_kernel: this block finished its column tile
};

template <int R>
__device__ __forceinline__ void make_plan(const DecodeParams &p, Plan &s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = p.T * p.k;
    for (int e = tid; e < p.E; e += kThreads) s.start[e] = 0;
    if (tid == 0) s.several = 0;
    __syncthreads();
    int id[kMaxPairs / kThreads], rank[kMaxPairs / kThreads];
#pragma unroll
    for (int i = 0; i < kMaxPairs / kThreads; ++i) {
        const int q = tid + i * kThreads;
        id[i] = q < n ? p.ids[q] : -1;
        if (id[i] >= p.E || id[i] < -1) {
            if (p.status) atomicOr(p.status, GFR_DEV_BAD_EXPERT);
            id[i] = -1;
        }
        rank[i] = id[i] >= 0 ? atomicAdd(&s.start[id[i]], 1) : 0;
    }
    __syncthreads();
    // two experts per thread; pairs and groups scanned together (both <= 1024)
    static_assert(GFR_MAX_EXPERTS <= 2 * kThreads, "two experts per thread");
    const int e0 = 2 * tid, e1 = e0 + 1;
    const uint32_t c0 = e0 < p.E ? s.start[e0] : 0, c1 = e1 < p.E ? s.start[e1] : 0;
    const uint32_t g0 = (c0 + R - 1) / R, g1 = (c1 + R - 1) / R;
    const uint32_t v = (c0 + c1) | (g0 + g1) << 16;
    const uint32_t incl = wave_prefix(v);
    if (lane == 63) s.totals[wave] = incl;
    if (g0 > 1 || g1 > 1) s.several = 1;
    __syncthreads();
    uint32_t at = incl - v, all = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) at += s.totals[w];
        all += s.totals[w];
    }
    if (tid == 0) s.groups = all >> 16;
    uint32_t pair = at & 0xffff, group = at >> 16;
    for (int h = 0; h < 2; ++h) {
        const int e = e0 + h;
        const uint32_t c = h ? c1 : c0;
        if (e < p.E) s.start[e] = pair;
        for (uint32_t r = 0; r < c; r += R, ++group) {
            s.expert[group] = e;
            s.first[group] = pair + r;
            s.count[group] = min(c - r, static_cast<uint32_t>(R));
        }
        pair += c;
    }
    const bool several = s.several;
    if (several)
#pragma unroll
        for (int i = 0; i < kMaxPairs / kThreads; ++i)
            s.ids[tid + i * kThreads] = static_cast<uint16_t>(id[i]);
    __syncthreads();
    if (several)
#pragma unroll
        for (int i = 0; i < kMaxPairs / kThreads; ++i) {
            rank[i] = 0;
            if (id[i] >= 0)
                for (int q = 0; q < tid + i * kThreads; ++q) rank[i] += s.ids[q] == id[i];
        }
#pragma unroll
    for (int i = 0; i < kMaxPairs / kThreads; ++i)
        if (id[i] >= 0) s.pairs[s.start[id[i]] + rank[i]] = tid + i * kThreads;
    __syncthreads();
}

// ---------------------------------------------------------------------------
// One wave's part of a product: rows (16 RG, as bf16 terms) times a column
// tile, over K steps [s0, s1).
// ---------------------------------------------------------------------------

__device__ __forceinline__ float e8m0(uint32_t code) { return __uint_as_float(code << 23); }

// Two FP8 values (the low or high half of w) times scale, in bf16.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t to_bf16(uint32_t w, float scale) {
    if (FMT == 0)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI));
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, HI));
}

__device__ __forceinline__ f4_t mfma(u4_t a, u4_t b, f4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, a),
                                                   __builtin_bit_cast(bf8_t, b), c, 0, 0, 0);
}

// What a wave reads: an expert's weights and scales and the operand rows, each
// through a buffer with one lane offset.  Row r of fragment f is addressed by
// the lanes with lane % 16 = r; a second bf16 term lies `second` bytes behind
// the first.
template <int RG>
struct Source {
    rsrc_t w, sc, x;
    int w_off, sc_off, x_off[RG];
    int ld;              // [K, N]: weight bytes per K row; [N, K]: K
    int second;
    int live;            // fragments with rows
};

// Weights [K, N]: lane (c, g) reads rows 8g .. 8g + 7 of a 32-row step, columns
// 8c .. 8c + 7 of the tile (past the `cols` columns: the last 8); accumulator j
// holds column 8c + j.
template <int FMT, int RG, int TERMS>
struct PartKN {
    static constexpr int kTile = 128, kAcc = 8, kStep = 32, kDepth = RG == 2 ? 3 : 2;
    static constexpr bool kKN = true;
    struct Stage {
        u2_t w[8];
        u4_t s;
        u4_t x[RG][TERMS];
    };
    static __device__ __forceinline__ void place(Source<RG> &a, int col0, int n0, int cols, int c,
                                                 int g) {
        const int col = col0 + min(n0 + 8 * c, cols - 8);
        a.w_off = 8 * g * a.ld + col;
        a.sc_off = 2 * col;
#pragma unroll
        for (int q = 0; q < RG; ++q) a.x_off[q] += 16 * g;
    }
    static __device__ __forceinline__ void fetch(Stage &f, const Source<RG> &a, int step) {
        const int k0 = step * kStep;
#pragma unroll
        for (int i = 0; i < 8; ++i) f.w[i] = load8<kNt>(a.w, a.w_off, (k0 + i) * a.ld);
        f.s = load16<0>(a.sc, a.sc_off, (k0 >> 6) * 2 * a.ld);
#pragma unroll
        for (int q = 0; q < RG; ++q)
            if (q < a.live)
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
                    f.x[q][t] = load16<0>(a.x, a.x_off[q], t * a.second + 2 * k0);
    }
    static __device__ __forceinline__ void use(const Stage &f, const Source<RG> &a, int step,
                                               f4_t (&acc)[RG][kAcc]) {
        const int odd = (step & 1) * 8;
#pragma unroll
        for (int d = 0; d < 2; ++d) {       // four columns each
            u4_t b[4];
            float scale[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                scale[j] = e8m0((f.s[2 * d + (j >> 1)] >> ((j & 1) * 16 + odd)) & 0xff);
#pragma unroll
            for (int q = 0; q < 4; ++q) {   // two K rows each
                const uint32_t lo = f.w[2 * q][d], hi = f.w[2 * q + 1][d];
                const uint32_t u = __builtin_amdgcn_perm(hi, lo, 0x05010400);
                const uint32_t v = __builtin_amdgcn_perm(hi, lo, 0x07030602);
                b[0][q] = to_bf16<FMT, false>(u, scale[0]);
                b[1][q] = to_bf16<FMT, true>(u, scale[1]);
                b[2][q] = to_bf16<FMT, false>(v, scale[2]);
                b[3][q] = to_bf16<FMT, true>(v, scale[3]);
            }
#pragma unroll
            for (int q = 0; q < RG; ++q)
                if (q < a.live)
#pragma unroll
                    for (int t = 0; t < TERMS; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[q][4 * d + j] = mfma(f.x[q][t], b[j], acc[q][4 * d + j]);
        }
    }
    static __device__ __forceinline__ int column(int c, int j) { return 8 * c + j; }
};

// Weights [N, K]: lane (c, g) reads K bytes 16g .. 16g + 15 of a 64-byte step
// of columns 16 f + c, f < NF; accumulator f holds column 16 f + c.  (Columns
// are a multiple of 64 and tiles divide 64: no fragment straddles the end.)
template <int FMT, int RG, int TERMS, int NF>
struct PartNK {
    static constexpr int kTile = 16 * NF, kAcc = NF, kStep = 64,
                         kDepth = TERMS == 2 ? 3 : 4;
    static constexpr bool kKN = false;
    struct Stage {
        u4_t w[NF];
        uint32_t s[NF];
        u4_t x[RG][TERMS][2];
    };
    static __device__ __forceinline__ void place(Source<RG> &a, int col0, int n0, int cols, int c,
                                                 int g) {
        (void)cols;
        const int col = col0 + n0 + c;
        a.w_off = col * a.ld + 16 * g;
        a.sc_off = col * (a.ld >> 5) + (g >> 1);
#pragma unroll
        for (int q = 0; q < RG; ++q) a.x_off[q] += 32 * g;
    }
    static __device__ __forceinline__ void fetch(Stage &f, const Source<RG> &a, int step) {
        const int k0 = step * kStep;
#pragma unroll
        for (int i = 0; i < NF; ++i) f.w[i] = load16<kNt>(a.w, a.w_off, i * 16 * a.ld + k0);
#pragma unroll
        for (int i = 0; i < NF; ++i)
            f.s[i] = load1(a.sc, a.sc_off, i * 16 * (a.ld >> 5) + 2 * step);
#pragma unroll
        for (int q = 0; q < RG; ++q)
            if (q < a.live)
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        f.x[q][t][h] =
                            load16<0>(a.x, a.x_off[q], t * a.second + 2 * k0 + 16 * h);
    }
    static __device__ __forceinline__ void use(const Stage &f, const Source<RG> &a, int step,
                                               f4_t (&acc)[RG][kAcc]) {
        (void)step;
#pragma unroll
        for (int i = 0; i < NF; ++i) {
            const float scale = e8m0(f.s[i]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u4_t b;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    b[2 * q] = to_bf16<FMT, false>(f.w[i][2 * h + q], scale);
                    b[2 * q + 1] = to_bf16<FMT, true>(f.w[i][2 * h + q], scale);
                }
#pragma unroll
                for (int q = 0; q < RG; ++q)
                    if (q < a.live)
#pragma unroll
                        for (int t = 0; t < TERMS; ++t)
                            acc[q][i] = mfma(f.x[q][t][h], b, acc[q][i]);
            }
        }
    }
    static __device__ __forceinline__ int column(int c, int j) { return 16 * j + c; }
};

// Steps [s0, s1) with kDepth steps' loads in flight.
template <class Part, int RG>
__device__ __forceinline__ void run_part(const Source<RG> &a, int s0, int s1,
                                         f4_t (&acc)[RG][Part::kAcc]) {
    constexpr int D = Part::kDepth;
    typename Part::Stage f[D];
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (s0 + d < s1) Part::fetch(f[d], a, s0 + d);
    for (int s = s0; s < s1; s += D)
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (s + d < s1) {
                Part::use(f[d], a, s + d, acc);
                if (s + d + D < s1) Part::fetch(f[d], a, s + d + D);
            }
}

// The accumulators of row fragment q into this wave's LDS tile [16][kTile]
// (rows past `rows` stay unwritten; nothing reads them).
template <class Part, int RG>
__device__ __forceinline__ void put_part(float *tile, const f4_t (&acc)[RG][Part::kAcc], int q,
                                         int rows, int c, int g) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 4 * g + i;
        if (row >= rows) continue;
#pragma unroll
        for (int f = 0; f < RG; ++f)
            if (f == q)
#pragma unroll
                for (int j = 0; j < Part::kAcc; ++j)
                    tile[row * Part::kTile + Part::column(c, j)] = acc[f][j][i];
    }
}

template <class Part, int RG>
__global__ __launch_bounds__(kThreads, RG == 1 ? 4 : 2) void gate_up_kernel(DecodeParams p) {
    extern __shared__ float tiles[];           // [8 waves][16][kTile]
    __shared__ Plan plan;
    constexpr int kTile = Part::kTile, R = 16 * RG;
    // down_kernel's counters
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.N / 16; i += kThreads) p.counter[i] = 0;
    make_plan<R>(p, plan);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int half = wave & 1, part = wave >> 1;
    const int ct = (p.I + kTile - 1) / kTile, units = uniform(plan.groups) * ct;
    const int steps = p.H / Part::kStep;
    const int s0 = steps * part / 4, s1 = steps * (part + 1) / 4;
    const int64_t slice = static_cast<int64_t>(p.H) * 2 * p.I;   // an expert's weights
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int gr = u / ct, n0 = (u - gr * ct) * kTile;
        const int e = uniform(plan.expert[gr]), first = uniform(plan.first[gr]),
                  count = uniform(plan.count[gr]);
        Source<RG> a;
        a.w = buffer(p.w13 + e * slice, slice);
        a.sc = buffer(p.s13 + e * p.s13_e, slice / 32);
        a.x = buffer(p.x, static_cast<int64_t>(p.T) * p.H * 2);
        a.ld = Part::kKN ? 2 * p.I : p.H;
        a.second = 0;
        a.live = (count + 15) >> 4;
#pragma unroll
        for (int q = 0; q < RG; ++q)
            a.x_off[q] = plan.pairs[first + min(q * 16 + c, count - 1)] / p.k * p.H * 2;
        Part::place(a, half * p.I, n0, p.I, c, g);
        f4_t acc[RG][Part::kAcc] = {};
        run_part<Part, RG>(a, s0, s1, acc);
#pragma unroll
        for (int q = 0; q < RG; ++q) {
            if (q >= a.live) break;
            const int rows = min(count - 16 * q, 16);
            put_part<Part, RG>(tiles + wave * 16 * kTile, acc, q, rows, c, g);
            __syncthreads();
            // four columns per thread: sums over the K ranges, SwiGLU, two terms
            for (int i = threadIdx.x; i < rows * (kTile / 4); i += kThreads) {
                const int row = i / (kTile / 4), col = i % (kTile / 4) * 4;
                if (n0 + col >= p.I) continue;
                f4_t gate = {0, 0, 0, 0}, up = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    gate += *reinterpret_cast<f4_t *>(&tiles[((2 * s) * 16 + row) * kTile + col]);
                    up += *reinterpret_cast<f4_t *>(&tiles[((2 * s + 1) * 16 + row) * kTile + col]);
                }
                u2_t hi, lo;
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = silu(gate[j]) * up[j];
                hi[0] = pack_bf16(v[0], v[1]);
                hi[1] = pack_bf16(v[2], v[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // an infinite or NaN first term stands for the whole value
                    const float head = __uint_as_float(
                        j & 1 ? hi[j >> 1] & 0xffff0000u : hi[j >> 1] << 16);
                    v[j] = fabsf(head) < INFINITY ? v[j] - head : 0.0f;
                }
                lo[0] = pack_bf16(v[0], v[1]);
                lo[1] = pack_bf16(v[2], v[3]);
                const int pair = plan.pairs[first + 16 * q + row];
                uint16_t *h = p.h + static_cast<int64_t>(pair) * p.I + n0 + col;
                *reinterpret_cast<u2_t *>(h) = hi;
                *reinterpret_cast<u2_t *>(h + static_cast<int64_t>(p.T) * p.k * p.I) = lo;
            }
            __syncthreads();
        }
    }
}

template <class Part, int RG>
__global__ __launch_bounds__(kThreads, RG == 1 ? 4 : 2) void down_kernel(DecodeParams p) {
    extern __shared__ float tiles[];
    __shared__ Plan plan;
    constexpr int kTile = Part::kTile, R = 16 * RG;
    make_plan<R>(p, plan);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int ct = (p.N + kTile - 1) / kTile, n = p.T * p.k, groups = uniform(plan.groups);
    // without any pair the column tiles still get the shared term or zeros
    const int per_tile = max(groups, 1) * p.split, units = ct * per_tile;
    const int steps = p.I / Part::kStep;
    const int64_t slice = static_cast<int64_t>(p.I) * p.N;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int tile = u / per_tile, n0 = tile * kTile;
        const int gr = (u - tile * per_tile) / p.split, sp = u % p.split;
        if (groups > 0) {
            const int e = uniform(plan.expert[gr]), first = uniform(plan.first[gr]),
                      count = uniform(plan.count[gr]);
            Source<RG> a;
            a.w = buffer(p.w2 + e * slice, slice);
            a.sc = buffer(p.s2 + e * p.s2_e, slice / 32);
            a.x = buffer(p.h, static_cast<int64_t>(n) * p.I * 4);
            a.ld = Part::kKN ? p.N : p.I;
            a.second = n * p.I * 2;
            a.live = (count + 15) >> 4;
#pragma unroll
            for (int q = 0; q < RG; ++q)
                a.x_off[q] = plan.pairs[first + min(q * 16 + c, count - 1)] * p.I * 2;
            Part::place(a, 0, n0, p.N, c, g);
            const int parts = kWaves * p.split, part = sp * kWaves + wave;
            f4_t acc[RG][Part::kAcc] = {};
            run_part<Part, RG>(a, steps * part / parts, steps * (part + 1) / parts, acc);
#pragma unroll
            for (int q = 0; q < RG; ++q) {
                if (q >= a.live) break;
                const int rows = min(count - 16 * q, 16);
                put_part<Part, RG>(tiles + wave * 16 * kTile, acc, q, rows, c, g);
                __syncthreads();
                for (int i = threadIdx.x; i < rows * (kTile / 4); i += kThreads) {
                    const int row = i / (kTile / 4), col = i % (kTile / 4) * 4;
                    if (n0 + col >= p.N) continue;
                    f4_t v = {0, 0, 0, 0};
#pragma unroll
                    for (int s = 0; s < kWaves; ++s)
                        v += *reinterpret_cast<f4_t *>(&tiles[(s * 16 + row) * kTile + col]);
                    const int pair = plan.pairs[first + 16 * q + row];
                    v *= p.weights[pair];
                    *reinterpret_cast<f4_t *>(
                        p.y + (static_cast<int64_t>(sp) * n + pair) * p.N + n0 + col) = v;
                }
                __syncthreads();
            }
        }
        // The block that finishes the column tile last adds up its rows.
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) plan.last = atomicAdd(&p.counter[tile], 1) == per_tile - 1;
        __syncthreads();
        if (plan.last) {
            __threadfence();
            for (int i = threadIdx.x; i < p.T * (kTile / 4); i += kThreads) {
                const int t = i / (kTile / 4), col = n0 + i % (kTile / 4) * 4;
                if (col >= p.N) continue;
                f4_t v = {0, 0, 0, 0};
                for (int j = 0; j < p.k; ++j) {
                    const int q = t * p.k + j, id = p.ids[q];
                    if (id < 0 || id >= p.E) continue;
                    for (int s = 0; s < p.split; ++s)
                        v += load<f4_t>(p.y + (static_cast<int64_t>(s) * n + q) * p.N + col);
                }
                const int64_t at = static_cast<int64_t>(t) * p.N + col;
                if (p.shared) {
                    const u2_t h = load<u2_t>(p.shared + at);
                    v[0] += p.shared_w * __uint_as_float(h[0] << 16);
                    v[1] += p.shared_w * __uint_as_float(h[0] & 0xffff0000u);
                    v[2] += p.shared_w * __uint_as_float(h[1] << 16);
                    v[3] += p.shared_w * __uint_as_float(h[1] & 0xffff0000u);
                }
                if (p.out_f32)
                    *reinterpret_cast<f4_t *>(static_cast<float *>(p.out) + at) = v;
                else
                    *reinterpret_cast<u2_t *>(static_cast<uint16_t *>(p.out) + at) =
                        u2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            }
        }
        __syncthreads();
    }
}

// Blocks per launch: two to a CU (at most; the units are dealt round).
template <class K>
hipError_t launch_units(K kernel, int64_t units, int rg, int tile, const DecodeParams &p,
                        hipStream_t stream) {
    const int64_t room = int64_t{cu_count()} * (rg == 1 ? 2 : 1);
    const int lds = kWaves * 16 * tile * static_cast<int>(sizeof(float));
    if (lds > (32 << 10)) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(units < room ? units : room)),
                       dim3(kThreads), lds, stream, p);
    return hipGetLastError();
}

// Groups of the plan, at most.
int64_t max_groups(int64_t pairs, int64_t E, int rg) {
    const int64_t g = (pairs < E ? pairs : E) + pairs / (16 * rg);
    return g < pairs ? g : pairs;
}

template <class Part, int RG>
hipError_t launch_gate_up(const DecodeParams &p, hipStream_t stream) {
    const int64_t ct = (p.I + Part::kTile - 1) / Part::kTile;
    return launch_units(&gate_up_kernel<Part, RG>, max_groups(p.T * p.k, p.E, RG) * ct, RG,
                        Part::kTile, p, stream);
}
template <class Part, int RG>
hipError_t launch_down(const DecodeParams &p, hipStream_t stream) {
    const int64_t ct = (p.N + Part::kTile - 1) / Part::kTile;
    return launch_units(&down_kernel<Part, RG>, max_groups(p.T * p.k, p.E, RG) * ct * p.split, RG,
                        Part::kTile, p, stream);
}

template <int FMT, int RG>
hipError_t launch_decode_t(const DecodeParams &p, int t13, int t2, hipStream_t stream) {
    constexpr int NF = RG == 1 ? 2 : 4;
    hipError_t e = t13 ? launch_gate_up<PartNK<FMT, RG, 1, NF>, RG>(p, stream)
                       : launch_gate_up<PartKN<FMT, RG, 1>, RG>(p, stream);
    if (e != hipSuccess) return e;
    return t2 ? launch_down<PartNK<FMT, RG, 2, NF>, RG>(p, stream)
              : launch_down<PartKN<FMT, RG, 2>, RG>(p, stream);
}

// Row fragments per group.  Two where an expert has more than 16 pairs often
// enough for the second reading of its weights to matter; one otherwise, which
// leaves registers for twice the waves.
int row_fragments(int64_t T, int64_t k, int64_t E) {
    const int64_t mean = T * k / E;
    return T <= 16 || mean <= 8 ? 1 : 2;
}

}  // namespace

DecodeLayout decode_layout(int64_t T, int64_t k, int64_t E, int64_t I, int64_t N,
                           int transpose_w2) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    DecodeLayout d{};
    const int64_t pairs = T * k;
    // split the down product's K until there are two units per CU, a step per
    // wave left to each
    const int rg = row_fragments(T, k, E);
    const int64_t tile = transpose_w2 ? (rg == 1 ? 32 : 64) : 128;
    const int64_t units = (pairs < E ? pairs : E) * ((N + tile - 1) / tile);
    const int64_t steps = I / (transpose_w2 ? 64 : 32);
    int split = 1;
    while (units * split < 512 && steps / (kWaves * split * 2) >= 1 && split < 8) split *= 2;
    d.split = split;
    d.h = 0;
    d.y = up(sizeof(uint16_t) * 2 * pairs * I);
    d.counter = d.y + up(sizeof(float) * split * pairs * N);
    d.total = d.counter + up(sizeof(int32_t) * (N / 16 + 1));
    return d;
}

hipError_t launch_decode(const DecodeParams &p, int transpose_w13, int transpose_w2, int e5m2,
                         hipStream_t stream) {
    const int rg = row_fragments(p.T, p.k, p.E);
    if (e5m2) {
        if (rg == 1) return launch_decode_t<1, 1>(p, transpose_w13, transpose_w2, stream);
        return launch_decode_t<1, 2>(p, transpose_w13, transpose_w2, stream);
    }
    if (rg == 1) return launch_decode_t<0, 1>(p, transpose_w13, transpose_w2, stream);
    return launch_decode_t<0, 2>(p, transpose_w13, transpose_w2, stream);
}

}  // namespace gfr
