// The experts of a MoE block for a few tokens.  include/gfr.h states the operator.
//
// At these token counts the bytes of the chosen experts' weights bound the
// time: each is read once, in FP8, and turned into bf16 MFMA operands in
// registers (v_cvt_scalef32_pk_bf16_*, which multiplies by the block's E8M0
// scale on the way).  That is exact from 2^-133, bf16's smallest value, to below
// 2^128, where FP32 ends too: bf16 has more mantissa bits than FP8, and any code is a
// multiple of 2^-133 at scales from 2^-124 (E4M3) or 2^-117 (E5M2) on.  The pairs
// (token, expert) of one expert are the columns of
// v_mfma_f32_16x16x32_bf16's second operand, 16 to a fragment.
//
//   product_kernel  (twice)  partial sums of a K chunk: gu = x w13, then
//                   y = h w2 with h = silu(gate) * up, formed from gu's chunks
//                   as the operand is brought to LDS and kept there as the sum
//                   of three bf16 terms, so that feeding it to the MFMAs does
//                   not round it;
//   activate_kernel  (kActivatePairs pairs and more) h once for all of them;
//   combine_kernel  out[t] = sum over t's pairs and y's chunks, in that order,
//                   plus the shared term, rounded once.
//
// A block takes (group of up to 16 RG pairs of one expert, K chunk, run of
// columns): it brings the group's operand rows of the chunk to LDS, and then
// each of its waves streams its own column tiles' weights, with the next steps'
// loads in flight across tile ends and no barrier.  Chunks and runs are chosen
// (part_shape) so that even one token's few experts keep every CU's loads
// in flight, and so that a long batch writes few partial sums.  (64 tokens of 32
// experts of 4096 x 8192, 3.2 GB: 530 us, 6.1 TB/s.  One token, 8 of 256 experts of
// 2048 x 512, 25 MB: 15.8 us, of which the two products' and the sum's latencies
// one after the other are most.)
//
// Weights [K, N]: a lane reads 8 columns of 8 rows (128-byte row pieces per
// wave) and v_perm pairs the rows, so the K-major operands come together in
// registers, without LDS.  Weights [N, K]: 32 bytes along K per lane, whole
// 128-byte lines per column.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gfr.h"
#include "gfr_device.h"
#include "gfr_layer.h"

namespace gfr {
namespace {

constexpr int kMaxWaves = 8;               // of a block of product_kernel
constexpr int kSumThreads = 256;           // of the small kernels
constexpr int kMaxPairs = 1024;
// From this many pairs on h is made once, by a launch of its own, for the down
// product's blocks, which otherwise each form their rows of it: 96 pairs of 8
// experts 145 -> 135 us, 256 pairs 137 -> 113, but 8 pairs 21 -> 23.
constexpr int kActivatePairs = 32;
// LDS per wave for a chunk's operand rows and their padding.  Of three terms as much
// as two blocks of four waves can have beside their plans (8 tokens of 16 experts of
// 4096 x 6144 with 16 KB 169 us, with this 161).
constexpr int operand_bytes(int terms) { return terms == 1 ? 16512 : 18624; }

// ---------------------------------------------------------------------------
// Plan: the pairs grouped by expert.  Every block makes its own from the ids
// (a launch to make it once would cost more).  Within a group the order of the
// pairs is left to the atomics: each is a row of its own, so no result depends
// on it.  Which group of an expert a pair falls into must be the same in every
// block, so where an expert has several groups its pairs are marked in a bit
// mask, and a pair's rank is the count of the marks below its own.
// ---------------------------------------------------------------------------
struct Plan {
    int start[GFR_MAX_EXPERTS];        // counts, then first index into pairs
    uint16_t pairs[kMaxPairs];         // grouped by expert
    uint32_t totals[kMaxWaves];
    int expert, first, count;          // this block's group
};
constexpr int kMaskWords = kMaxPairs / 32;
constexpr int kMaskBytes = kMaxPairs / 16 * kMaskWords * 4;   // experts with over 16 pairs

// The same for at most 64 pairs, one per lane, without a barrier: every wave
// goes through the experts in the order of their first pairs until it reaches
// group `mine`, and all write the same list.  (One token, 8 of 256 experts of 2048
// x 512: 29 -> 22 us for the whole call with this, the weights' loads ahead of the
// operand and a combine_kernel that takes columns in slices.)
template <int R>
__device__ __forceinline__ bool make_small_plan(const DecodeParams &p, Plan &s, int mine, int &e,
                                                int &first, int &count) {
    const int lane = threadIdx.x & 63;
    int id = lane < p.T * p.k ? p.ids[lane] : -1;
    if (id >= p.E || id < -1) {
        if (p.status) atomicOr(p.status, GFR_DEV_BAD_EXPERT);
        id = -1;
    }
    uint64_t left = __ballot(id >= 0);
    while (left) {
        e = __builtin_amdgcn_readlane(id, __ffsll(static_cast<unsigned long long>(left)) - 1);
        const uint64_t same = __ballot(id == e);
        const int pairs = __popcll(same), groups = (pairs + R - 1) / R;
        if (mine < groups) {
            first = mine * R;
            count = min(pairs - first, R);
            if (id == e) s.pairs[__popcll(same & ((uint64_t{1} << lane) - 1))] = lane;
            return true;
        }
        mine -= groups;
        left &= ~same;
    }
    return false;
}

// Fills `s` for group `mine`; false if there are fewer groups.  `mask`: kMaskBytes
// of LDS that nothing else uses meanwhile.
template <int R, int kWaves>
__device__ __forceinline__ bool make_plan(const DecodeParams &p, Plan &s, uint32_t *mask,
                                          int mine) {
    constexpr int kThreads = 64 * kWaves;
    constexpr int kPer = kMaxPairs / kThreads, kExperts = GFR_MAX_EXPERTS / kThreads;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = p.T * p.k;
    int id[kPer], rank[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int q = tid + i * kThreads;
        id[i] = q < n ? p.ids[q] : -1;
    }
    for (int e = tid; e < p.E; e += kThreads) s.start[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (id[i] >= p.E || id[i] < -1) {
            if (p.status) atomicOr(p.status, GFR_DEV_BAD_EXPERT);
            id[i] = -1;
        }
        rank[i] = id[i] >= 0 ? atomicAdd(&s.start[id[i]], 1) : 0;
    }
    __syncthreads();
    // Consecutive experts per thread.  Pairs (at most 1024), groups (1024) and
    // experts of several groups (64) are scanned together: 11, 11 and 7 bits.
    uint32_t c[kExperts], v = 0;
#pragma unroll
    for (int h = 0; h < kExperts; ++h) {
        const int e = kExperts * tid + h;
        c[h] = e < p.E ? s.start[e] : 0;
        v += c[h] | ((c[h] + R - 1) / R) << 11 | (c[h] > R ? 1u << 22 : 0);
    }
    const uint32_t incl = wave_prefix(v);
    if (lane == 63) s.totals[wave] = incl;
    __syncthreads();
    uint32_t at = incl - v, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) at += s.totals[w];
        all += s.totals[w];
    }
    if (mine >= static_cast<int>(all >> 11 & 0x7ff)) return false;
    const int several = all >> 22;
#pragma unroll
    for (int h = 0; h < kExperts; ++h) {
        const int e = kExperts * tid + h;
        const int pair = at & 0x7ff, group = at >> 11 & 0x7ff, groups = (c[h] + R - 1) / R;
        // first index; mask + 1 above it
        if (e < p.E) s.start[e] = pair | (c[h] > R ? (at >> 22) + 1 : 0) << 16;
        if (mine >= group && mine < group + groups) {
            const int r = (mine - group) * R;
            s.expert = e;
            s.first = pair + r;
            s.count = min(static_cast<int>(c[h]) - r, R);
        }
        at += c[h] | groups << 11 | (c[h] > R ? 1u << 22 : 0);
    }
    for (int i = tid; i < several * kMaskWords; i += kThreads) mask[i] = 0;
    __syncthreads();
    if (several) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int q = tid + i * kThreads, m = id[i] >= 0 ? s.start[id[i]] >> 16 : 0;
            if (m) atomicOr(&mask[(m - 1) * kMaskWords + (q >> 5)], 1u << (q & 31));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int q = tid + i * kThreads, m = id[i] >= 0 ? s.start[id[i]] >> 16 : 0;
            if (!m) continue;
            const uint32_t *w = mask + (m - 1) * kMaskWords;
            rank[i] = __popc(w[q >> 5] & ((1u << (q & 31)) - 1));
            for (int j = 0; j < q >> 5; ++j) rank[i] += __popc(w[j]);
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (id[i] >= 0) s.pairs[(s.start[id[i]] & 0xffff) + rank[i]] = tid + i * kThreads;
    __syncthreads();
    return true;
}

// ---------------------------------------------------------------------------
// Weight streams
// ---------------------------------------------------------------------------

// The scale operand of the conversion, which takes the exponent field alone: 2^(code -
// 127) also for code 0, NaN for 255.
__device__ __forceinline__ float e8m0(uint32_t code) { return __uint_as_float(code << 23); }

// Two FP8 values (the low or high half of w) times scale, in bf16.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t to_bf16(uint32_t w, float scale) {
    if (FMT == 0)
        return __builtin_bit_cast(uint32_t,
                                  __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI));
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, HI));
}

__device__ __forceinline__ f4_t mfma(u4_t a, u4_t b, f4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, a),
                                                   __builtin_bit_cast(bf8_t, b), c, 0, 0, 0);
}

// One expert's weights and scales through buffers; ld is the bytes per K row
// ([K, N]) or per column ([N, K]).
struct Weights {
    rsrc_t w, sc;
    int w_off, sc_off, ld;
};

// The operand rows in LDS: row r of term t at base + (t rows + r) pitch bytes;
// this lane's row c and first K element are in `lane`.
struct Operand {
    const uint8_t *lane;
    int pitch, term;      // bytes between fragments' rows (16 rows), and terms
};

// Weights [K, N]: of a 64-row step, lane (c, g) reads rows 32b + 8g .. + 7, b <
// 2, columns 8c .. 8c + 7 of the 128-column tile; accumulator j holds columns
// 8 r + j for fragment rows r.  (In a tile that the columns' end cuts, lanes
// past the end read the next row's bytes, or zeros; nothing keeps them.)
template <int FMT>
struct StreamKN {
    static constexpr bool kKN = true;
    static constexpr int kTile = 128, kAcc = 8, kStep = 64, kDepth = 2;
    struct Stage {
        u2_t w[2][8];
        u4_t s;
    };
    static __device__ __forceinline__ void place(Weights &a, int c, int g) {
        a.w_off = 8 * g * a.ld + 8 * c;
        a.sc_off = 16 * c;
    }
    static __device__ __forceinline__ int lane_k(int g) { return 8 * g; }
    static __device__ __forceinline__ void fetch(Stage &f, const Weights &a, int n0, int k0) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f.w[b][i] = load8<kNt>(a.w, a.w_off, (k0 + 32 * b + i) * a.ld + n0);
        f.s = load16<0>(a.sc, a.sc_off, (k0 >> 6) * 2 * a.ld + 2 * n0);
    }
    template <int RG, int TERMS>
    static __device__ __forceinline__ void use(Stage &f, const Operand &x, int k, int left,
                                               int live, f4_t (&acc)[RG][kAcc]) {
        (void)left;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            u4_t o[RG][TERMS];
#pragma unroll
            for (int q = 0; q < RG; ++q)
                if (q < live)
#pragma unroll
                    for (int t = 0; t < TERMS; ++t)
                        o[q][t] = load<u4_t>(x.lane + q * x.pitch + t * x.term + 2 * (k + 32 * b));
#pragma unroll
            for (int d = 0; d < 2; ++d) {       // four columns each
                u4_t m[4];
                float scale[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    scale[j] = e8m0((f.s[2 * d + (j >> 1)] >> ((j & 1) * 16 + 8 * b)) & 0xff);
#pragma unroll
                for (int q = 0; q < 4; ++q) {   // two K rows each
                    const uint32_t lo = f.w[b][2 * q][d], hi = f.w[b][2 * q + 1][d];
                    const uint32_t u = __builtin_amdgcn_perm(hi, lo, 0x05010400);
                    const uint32_t v = __builtin_amdgcn_perm(hi, lo, 0x07030602);
                    m[0][q] = to_bf16<FMT, false>(u, scale[0]);
                    m[1][q] = to_bf16<FMT, true>(u, scale[1]);
                    m[2][q] = to_bf16<FMT, false>(v, scale[2]);
                    m[3][q] = to_bf16<FMT, true>(v, scale[3]);
                }
#pragma unroll
                for (int q = 0; q < RG; ++q)
                    if (q < live)
#pragma unroll
                        for (int t = 0; t < TERMS; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                acc[q][4 * d + j] = mfma(m[j], o[q][t], acc[q][4 * d + j]);
            }
        }
    }
    // Lane (c, g): row c's columns n0 + 8 (4g + i) + j.
    static __device__ __forceinline__ void store(float *row, int n0, int cols, int g,
                                                 const f4_t (&acc)[kAcc]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 32 * g + 8 * i;
            if (n >= cols) break;
            *reinterpret_cast<f4_t *>(row + n) =
                f4_t{acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
            *reinterpret_cast<f4_t *>(row + n + 4) =
                f4_t{acc[4][i], acc[5][i], acc[6][i], acc[7][i]};
        }
    }
};

// Weights [N, K]: a step is KL 128-byte lines of columns 16 f + r, f < NF = 4 /
// KL, loaded whole and swapped into operands (swap_halves); accumulator f holds
// columns 16 f + r for fragment rows r.  The step's scales of column c, eight
// 16-bit pairs, are read two to a lane and handed round: a load per fragment and
// half would touch as many lines as the weights do.  (16 experts of 4096 x 6144, 8
// tokens: half-line loads and scale loads apart 237 us, scales handed round 175,
// whole lines 157.)  KL = 2 with one row fragment (there: KL = 1 185 us, KL = 4
// 170), 1 with two, whose operand reads a wider tile shares.
template <int FMT, int KL>
struct StreamNK {
    static constexpr bool kKN = false;
    static constexpr int NF = 4 / KL;
    static constexpr int kTile = 16 * NF, kAcc = NF, kStep = 128 * KL, kDepth = 3;
    struct Stage {
        u4_t w[NF][KL][2];
        uint32_t s[2];
    };
    static __device__ __forceinline__ void place(Weights &a, int c, int g) {
        a.w_off = (c & 7) * a.ld + 16 * (g + 4 * (c >> 3));
        // pairs v = 2g, 2g + 1 of column c: fragment v / (2 KL), half v % (2 KL)
        a.sc_off = (16 * (g / KL) + c) * (a.ld >> 5) + 4 * (g % KL);
    }
    static __device__ __forceinline__ int lane_k(int g) { return 16 * g; }
    static __device__ __forceinline__ void fetch(Stage &f, const Weights &a, int n0, int k0) {
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int l = 0; l < KL; ++l)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    f.w[i][l][b] =
                        load16<kNt>(a.w, a.w_off, (n0 + 16 * i + 8 * b) * a.ld + k0 + 128 * l);
#pragma unroll
        for (int v = 0; v < 2; ++v)
            f.s[v] = load2(a.sc, a.sc_off, n0 * (a.ld >> 5) + (k0 >> 5) + 2 * v);
    }
    template <int RG, int TERMS>
    static __device__ __forceinline__ void use(Stage &f, const Operand &x, int k, int left,
                                               int live, f4_t (&acc)[RG][kAcc]) {
        const int shift = threadIdx.x & 32 ? 8 : 0;    // g >= 2: the half's second block
        const uint32_t pair = f.s[0] | f.s[1] << 16;
        uint32_t s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            s[j] = __shfl(pair, (threadIdx.x & 15) + 16 * j) >> shift;
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int l = 0; l < KL; ++l) swap_halves(f.w[i][l][0], f.w[i][l][1]);
        if (left < kStep) {
            // halves behind K's end are zeros (K is a multiple of 64), and their
            // scales, another column's, one
#pragma unroll
            for (int h = 1; h < 2 * KL; ++h)
                if (64 * h >= left)
#pragma unroll
                    for (int i = 0; i < NF; ++i) {
                        f.w[i][h >> 1][h & 1] = u4_t{0, 0, 0, 0};
                        const int v = i * 2 * KL + h;
                        s[v >> 1] = v & 1 ? (s[v >> 1] & 0xffff) | 0x7f0000
                                          : (s[v >> 1] & 0xffff0000u) | 0x7f;
                    }
        }
#pragma unroll
        for (int h = 0; h < 4 * KL; ++h) {             // 64-byte halves' 8-byte halves
            u4_t o[RG][TERMS];
#pragma unroll
            for (int q = 0; q < RG; ++q)
                if (q < live)
#pragma unroll
                    for (int t = 0; t < TERMS; ++t)
                        o[q][t] = load<u4_t>(x.lane + q * x.pitch + t * x.term +
                                             2 * (k + 64 * (h >> 1) + 8 * (h & 1)));
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const int v = i * 2 * KL + (h >> 1);
                const float scale = e8m0(s[v >> 1] >> (16 * (v & 1)) & 0xff);
                u4_t m;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t w = f.w[i][h >> 2][h >> 1 & 1][2 * (h & 1) + q];
                    m[2 * q] = to_bf16<FMT, false>(w, scale);
                    m[2 * q + 1] = to_bf16<FMT, true>(w, scale);
                }
#pragma unroll
                for (int q = 0; q < RG; ++q)
                    if (q < live)
#pragma unroll
                        for (int t = 0; t < TERMS; ++t)
                            acc[q][i] = mfma(m, o[q][t], acc[q][i]);
            }
        }
    }
    static __device__ __forceinline__ void store(float *row, int n0, int cols, int g,
                                                 const f4_t (&acc)[kAcc]) {
        (void)cols;
#pragma unroll
        for (int i = 0; i < NF; ++i) *reinterpret_cast<f4_t *>(row + n0 + 16 * i + 4 * g) = acc[i];
    }
};

// h = silu(gate) * up of four neighbouring columns as three bf16 terms whose sum is
// the FP32 value: 8 mantissa bits each, cut off (what is left is exact), so that the
// matrix unit's FP32 sums see all 24.  (With two terms a bf16 result is off from
// that of an FP32 h in 0.3 % of the elements, an FP32 result by 2.4e-6 instead of
// 3e-7.  Bits below 2^-133, bf16's smallest, are lost.)
__device__ __forceinline__ void three_terms(f4_t gate, f4_t up, u2_t (&term)[3]) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = silu(gate[j]) * up[j];
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        uint32_t bits[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bits[j] = __float_as_uint(v[j]) & 0xffff0000u;
            // an infinite or NaN first term stands for the whole value
            v[j] = fabsf(v[j]) < INFINITY ? v[j] - __uint_as_float(bits[j]) : 0.0f;
        }
        term[t] = u2_t{bits[1] | bits[0] >> 16, bits[3] | bits[2] >> 16};
    }
}

// Partial sums of a K chunk.  TERMS = 1: operand x, out gu [chunks][pairs][2I];
// TERMS = 3: operand h from gu, out y [chunks][pairs][N].  Grid: (column runs,
// chunks, groups).
// SHARED: the block's waves share one column tile, each takes every kWaves-th step,
// and their sums meet in LDS.
template <class Stream, int RG, int TERMS, int kWaves, bool SHARED>
__global__ __launch_bounds__(64 * kWaves, 2) void product_kernel(DecodeParams p) {
    constexpr int kThreads = 64 * kWaves;
    // (aligned: 16-byte accesses to LDS at odd words take about twice as long)
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ __align__(16) Plan plan;
    constexpr int R = 16 * RG, kStep = Stream::kStep, kTile = Stream::kTile;
    int e = 0, first = 0, count = 0;
    if (p.T * p.k <= 64) {
        if (!make_small_plan<R>(p, plan, blockIdx.z, e, first, count)) return;
    } else {
        if (!make_plan<R, kWaves>(p, plan, reinterpret_cast<uint32_t *>(lds), blockIdx.z)) return;
        e = uniform(plan.expert), first = uniform(plan.first), count = uniform(plan.count);
    }
    const DecodePart &d = TERMS == 1 ? p.gate_up : p.down;
    const int K = TERMS == 1 ? p.H : p.I, cols = TERMS == 1 ? 2 * p.I : p.N, n = p.T * p.k;

    const int all = (K + kStep - 1) / kStep, chunk = blockIdx.y;
    const int s0 = all * chunk / d.chunks, steps = all * (chunk + 1) / d.chunks - s0;
    const int k0 = s0 * kStep, width = steps * kStep, real = min(width, K - k0);
    const int pitch = 2 * width + 16;       // spreads the rows over the banks
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int64_t slice = static_cast<int64_t>(K) * cols;
    Weights a;
    a.w = buffer((TERMS == 1 ? p.w13 : p.w2) + e * slice, slice);
    a.sc = buffer(TERMS == 1 ? p.s13 + e * p.s13_e : p.s2 + e * p.s2_e, slice / 32);
    a.ld = Stream::kKN ? cols : K;
    Stream::place(a, c, g);
    Operand x;
    x.lane = lds + c * pitch + 2 * Stream::lane_k(g);
    x.pitch = 16 * pitch;
    x.term = R * pitch;
    const int live = (count + 15) >> 4;

    // This wave's tiles: every kWaves-th of the block's run.
    const int tiles = (cols + kTile - 1) / kTile;
    int tile = SHARED ? blockIdx.x : blockIdx.x * d.run * kWaves + wave;
    const int mine = max(min(d.run, (tiles - tile + kWaves - 1) / kWaves), 0);
    // Blocks side by side begin at different steps and go round: rows and
    // columns a power of two apart share memory channels.  (By the expert and not by
    // the group: where other tokens' groups lie must not change a token's sums.)
    const int turn = SHARED ? wave : (blockIdx.x + e) % steps;
    const int total = SHARED ? max(steps - wave + kWaves - 1, 0) / kWaves : mine * steps;
    int fetch_step = turn, fetch_n0 = tile * kTile, fetched = 0;
    typename Stream::Stage f[Stream::kDepth];
    auto fetch = [&](typename Stream::Stage &s) {
        Stream::fetch(s, a, fetch_n0, k0 + fetch_step * kStep);
        if (SHARED) {
            fetch_step += kWaves;
        } else {
            if (++fetch_step == steps) fetch_step = 0;
            if (fetch_step == turn) fetch_n0 += kWaves * kTile;
        }
        ++fetched;
    };
#pragma unroll
    for (int i = 0; i < Stream::kDepth; ++i)
        if (i < total) fetch(f[i]);
    // The chunk's operand rows.  Rows past the group's are left as they are: a
    // row's sums depend on its own operand alone.
    if (TERMS == 1) {
#pragma unroll 4
        for (int i = threadIdx.x; i < count * (width / 8); i += kThreads) {
            const int r = i / (width / 8), k = i % (width / 8) * 8;
            const int64_t t = plan.pairs[first + r] / p.k;
            *reinterpret_cast<u4_t *>(lds + r * pitch + 2 * k) =
                k < real ? load<u4_t>(p.x + t * p.H + k0 + k) : u4_t{0, 0, 0, 0};
        }
    } else if (p.h) {
        const int64_t plane = static_cast<int64_t>(n) * p.I;
#pragma unroll 4
        for (int i = threadIdx.x; i < count * (width / 8); i += kThreads) {
            const int r = i / (width / 8), k = i % (width / 8) * 8;
            const uint16_t *at = p.h + static_cast<int64_t>(plan.pairs[first + r]) * p.I + k0 + k;
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
                *reinterpret_cast<u4_t *>(lds + (t * R + r) * pitch + 2 * k) =
                    k < real ? load<u4_t>(at + t * plane) : u4_t{0, 0, 0, 0};
        }
    } else {
        const int64_t plane = static_cast<int64_t>(n) * 2 * p.I;
        const int last = p.gate_up.chunks - 1;
#pragma unroll 2
        for (int i = threadIdx.x; i < count * (width / 4); i += kThreads) {
            const int r = i / (width / 4), k = i % (width / 4) * 4;
            u2_t term[3] = {};
            if (k < real) {
                const float *at =
                    p.gu + static_cast<int64_t>(plan.pairs[first + r]) * 2 * p.I + k0 + k;
                f4_t gate = {0, 0, 0, 0}, up = {0, 0, 0, 0};
                // four chunks' loads at a time, past the last one its own again
                for (int s = 0; s <= last; s += 4) {
                    f4_t v[4], u[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[j] = load<f4_t>(at + min(s + j, last) * plane);
                        u[j] = load<f4_t>(at + min(s + j, last) * plane + p.I);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (s + j <= last) gate += v[j], up += u[j];
                }
                three_terms(gate, up, term);
            }
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
                *reinterpret_cast<u2_t *>(lds + (t * R + r) * pitch + 2 * k) = term[t];
        }
    }
    __syncthreads();
    f4_t acc[RG][Stream::kAcc] = {};
    int step = turn;
    float *out = (TERMS == 1 ? p.gu : p.y) + static_cast<int64_t>(chunk) * n * cols;
    for (int i = 0; i < total; i += Stream::kDepth)
#pragma unroll
        for (int j = 0; j < Stream::kDepth; ++j) {
            if (i + j >= total) break;
            Stream::template use<RG, TERMS>(f[j], x, step * kStep, K - k0 - step * kStep, live,
                                            acc);
            if (fetched < total) fetch(f[j]);
            if (SHARED) {
                step += kWaves;
                continue;
            }
            if (++step == steps) step = 0;
            if (step == turn) {
#pragma unroll
                for (int q = 0; q < RG; ++q) {
                    if (16 * q + c < count)
                        Stream::store(out + static_cast<int64_t>(plan.pairs[first + 16 * q + c]) *
                                                cols,
                                      tile * kTile, cols, g, acc[q]);
#pragma unroll
                    for (int m = 0; m < Stream::kAcc; ++m) acc[q][m] = f4_t{0, 0, 0, 0};
                }
                tile += kWaves;
            }
        }
    if constexpr (SHARED) {
        // A lane's 32 sums are four runs of eight columns (Stream::store); wave i adds
        // up and stores run i of all waves, in order.
        static_assert(Stream::kKN && RG == 1 && kWaves == 4, "four runs of eight columns");
        f4_t *const sums = reinterpret_cast<f4_t *>(lds);
        __syncthreads();
        if (c < count)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sums[((i * 2 + h) * kWaves + wave) * 64 + lane] =
                        f4_t{acc[0][4 * h][i], acc[0][4 * h + 1][i], acc[0][4 * h + 2][i],
                             acc[0][4 * h + 3][i]};
        __syncthreads();
        const int col = tile * kTile + 32 * g + 8 * wave;
        if (c >= count || col >= cols) return;
        float *to = out + static_cast<int64_t>(plan.pairs[first + c]) * cols + col;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f4_t *at = sums + (wave * 2 + h) * kWaves * 64 + lane;
            f4_t v = at[0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += at[64 * w];
            *reinterpret_cast<f4_t *>(to + 4 * h) = v;
        }
    }
}

// h = silu(gate) * up as three bf16 terms, once for all blocks of the down product.
__global__ __launch_bounds__(kSumThreads) void activate_kernel(DecodeParams p) {
    const int64_t n = static_cast<int64_t>(p.T) * p.k, fours = p.I / 4;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kSumThreads + threadIdx.x;
    if (i >= n * fours) return;
    const int64_t q = i / fours, k = i % fours * 4;
    const int id = p.ids[q];
    if (id < 0 || id >= p.E) return;             // nothing wrote, or reads, its row
    const float *at = p.gu + q * 2 * p.I + k;
    f4_t gate = {0, 0, 0, 0}, up = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < p.gate_up.chunks; ++s, at += n * 2 * p.I) {
        gate += load<f4_t>(at);
        up += load<f4_t>(at + p.I);
    }
    u2_t term[3];
    three_terms(gate, up, term);
#pragma unroll
    for (int t = 0; t < 3; ++t) *reinterpret_cast<u2_t *>(p.h + (t * n + q) * p.I + k) = term[t];
}

// out[t, n .. n + 3] = sum over t's pairs j and y's chunks s of weight[t, j]
// y[s][t k + j], plus the shared term.  A block takes 128 columns of a token:
// eight slices of the (j, s) terms at a time, so that the loads of one token's
// few columns run side by side; then the slices in order.
constexpr int kSlices = 8, kFours = kSumThreads / kSlices;
__global__ __launch_bounds__(kSumThreads) void combine_kernel(DecodeParams p) {
    __shared__ float weight[GFR_MAX_TOPK];
    __shared__ int live[GFR_MAX_TOPK];
    __shared__ f4_t part[kSlices][kFours];
    const int t = blockIdx.y, slice = threadIdx.x / kFours, four = threadIdx.x % kFours;
    const int col = (blockIdx.x * kFours + four) * 4;
    if (threadIdx.x < p.k) {
        const int id = p.ids[t * p.k + threadIdx.x];
        live[threadIdx.x] = id >= 0 && id < p.E;
        weight[threadIdx.x] = p.weights[t * p.k + threadIdx.x];
    }
    __syncthreads();
    f4_t v = {0, 0, 0, 0};
    if (col < p.N) {
        const int chunks = p.down.chunks, terms = p.k * chunks;
        const float *at = p.y + static_cast<int64_t>(t) * p.k * p.N + col;
        const int64_t plane = static_cast<int64_t>(p.T) * p.k * p.N;
#pragma unroll 4
        for (int i = slice; i < terms; i += kSlices) {
            const int j = i / chunks, s = i - j * chunks;
            const int64_t off = s * plane + static_cast<int64_t>(j) * p.N;
            if (live[j]) v += weight[j] * load<f4_t>(at + off);
        }
    }
    part[slice][four] = v;
    __syncthreads();
    if (slice != 0 || col >= p.N) return;
#pragma unroll
    for (int s = 1; s < kSlices; ++s) v += part[s][four];
    const int64_t at = static_cast<int64_t>(t) * p.N + col;
    if (p.shared) {
        const u2_t h = load<u2_t>(p.shared + at);
        v += p.shared_w * f4_t{__uint_as_float(h[0] << 16), __uint_as_float(h[0] & 0xffff0000u),
                               __uint_as_float(h[1] << 16), __uint_as_float(h[1] & 0xffff0000u)};
    }
    if (p.out_f32)
        *reinterpret_cast<f4_t *>(static_cast<float *>(p.out) + at) = v;
    else
        *reinterpret_cast<u2_t *>(static_cast<uint16_t *>(p.out) + at) =
            u2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Row fragments per group.  Two where an expert has more than 16 pairs often
// enough for the second reading of its weights to matter; one otherwise.
int row_fragments(int64_t T, int64_t k, int64_t E) {
    const int64_t mean = T * k / E;
    return T <= 16 || mean <= 8 ? 1 : 2;
}

// Groups of the plan, at most.
int64_t max_groups(int64_t pairs, int64_t E, int rg) {
    const int64_t g = (pairs < E ? pairs : E) + pairs / (16 * rg);
    return g < pairs ? g : pairs;
}

// Lines of K per [N, K] step (StreamNK's KL).
constexpr int lines(int rg) { return rg == 1 ? 2 : 1; }

// Chunks, runs and waves of one product.  As few chunks as the LDS allows; runs as
// long as leaves enough blocks; if even runs of one tile per wave are fewer, more
// chunks.  Blocks of eight waves, one to a CU, hold chunks twice as wide as two
// of four waves, which halves the partial sums and the operand's reading: worth
// it where a group has rows enough for that to count and blocks are many (64
// tokens of 32 experts, 4096 x 8192: 577 -> 518 us; 8 tokens of 16, 157 -> 172).
// [N, K] with two row fragments, whose tiles are wider, needs nearly two rounds of
// them (64 tokens, 4 of 16 experts of 4096 x 4096, 2.3 rounds: 227 -> 204 us; 4 of 8
// of 4096 x 2048, 1.1 rounds: 113 -> 123).
// Where blocks of a [K, N] tile per wave are fewer than three per CU, a block's
// waves share a tile and split its steps: four times the blocks, and no more
// partial sums (one token, 8 of 256 experts of 2048 x 512: 21.3 -> 15.8 us; 2 of 8
// of 4096 x 7168: 53.7 -> 46.8).  [N, K] tiles are a quarter as wide and fill the CUs
// without.  (These pairs of times were measured with the down product's operand in two
// terms; three cost it up to 8 %.)
DecodePart part_shape(double groups, double rows, int64_t K, int64_t cols, int transpose, int rg,
                      int terms) {
    const int64_t step = transpose ? 128 * lines(rg) : 64;
    const int64_t tile = transpose ? 64 / lines(rg) : 128;
    const int64_t steps = (K + step - 1) / step, tiles = (cols + tile - 1) / tile;
    DecodePart d{};
    for (int waves : {4, 8}) {
        if (waves == 8 && rows < 4.0) break;
        // wanted: 12 waves a CU, or 7 where two row fragments take their registers
        const double blocks = 256.0 * (rg == 1 ? 12 : 7) / waves;
        // steps per chunk, at most
        const int64_t wide =
            (operand_bytes(terms) * waves / (terms * 16 * rg) - 16) / 2 / step;
        int64_t chunks = (steps + wide - 1) / wide;
        const double runs = groups * chunks * tiles / (waves * blocks);
        if (waves == 8 && transpose && rg == 2 && runs < 1.75) break;
        int64_t run = static_cast<int64_t>(runs);
        const bool enough = run >= 1;
        if (!enough) {
            run = 1;
            const double got = groups * ((tiles + waves - 1) / waves);
            while (got * chunks < blocks && steps / (chunks + 1) >= (transpose ? 1 : 2) &&
                   chunks < 8)
                ++chunks;
        }
        const int64_t most = (tiles + waves - 1) / waves;
        d = {static_cast<int32_t>(chunks), static_cast<int32_t>(run < most ? run : most), waves, 0};
        if (!enough) {
            if (waves == 4 && rg == 1 && !transpose &&
                groups * ((tiles + waves - 1) / waves) * chunks < blocks) {
                for (chunks = (steps + wide - 1) / wide;
                     groups * tiles * chunks < blocks && steps / (chunks + 1) >= 4 && chunks < 8;)
                    ++chunks;
                d = {static_cast<int32_t>(chunks), 1, waves, 1};
            }
            break;
        }
    }
    return d;
}

template <class Stream, int RG, int TERMS, int kWaves, bool SHARED = false>
hipError_t launch_product(const DecodeParams &p, hipStream_t stream) {
    const DecodePart &d = TERMS == 1 ? p.gate_up : p.down;
    const int K = TERMS == 1 ? p.H : p.I, cols = TERMS == 1 ? 2 * p.I : p.N;
    const int steps = (K + Stream::kStep - 1) / Stream::kStep;
    const int width = (steps + d.chunks - 1) / d.chunks * Stream::kStep;
    const int operand = TERMS * 16 * RG * (2 * width + 16);
    constexpr int kLeast = SHARED ? 8 * kWaves * 64 * 16 : kMaskBytes;    // SHARED: the sums
    const int lds = operand > kLeast ? operand : kLeast;
    const int tiles = (cols + Stream::kTile - 1) / Stream::kTile;
    const int per_run = SHARED ? 1 : d.run * kWaves, runs = (tiles + per_run - 1) / per_run;
    constexpr auto kernel = &product_kernel<Stream, RG, TERMS, kWaves, SHARED>;
    if (hipError_t e = allow_lds<kernel>(lds); e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel,
                       dim3(runs, d.chunks, static_cast<uint32_t>(max_groups(p.T * p.k, p.E, RG))),
                       dim3(64 * kWaves), lds, stream, p);
    return hipGetLastError();
}

template <int FMT, int RG, int TERMS>
hipError_t launch_product_any(const DecodeParams &p, int transpose, hipStream_t stream) {
    typedef StreamNK<FMT, lines(RG)> NK;
    typedef StreamKN<FMT> KN;
    if constexpr (RG == 1)
        if ((TERMS == 1 ? p.gate_up : p.down).shared)
            return launch_product<KN, RG, TERMS, 4, true>(p, stream);
    if ((TERMS == 1 ? p.gate_up : p.down).waves == 8)
        return transpose ? launch_product<NK, RG, TERMS, 8>(p, stream)
                         : launch_product<KN, RG, TERMS, 8>(p, stream);
    return transpose ? launch_product<NK, RG, TERMS, 4>(p, stream)
                     : launch_product<KN, RG, TERMS, 4>(p, stream);
}

template <int FMT, int RG>
hipError_t launch_decode_t(const DecodeParams &p, int t13, int t2, hipStream_t stream) {
    hipError_t e = launch_product_any<FMT, RG, 1>(p, t13, stream);
    if (e != hipSuccess) return e;
    if (p.h) {
        const int64_t fours = static_cast<int64_t>(p.T) * p.k * (p.I / 4);
        const auto blocks = static_cast<uint32_t>((fours + kSumThreads - 1) / kSumThreads);
        hipLaunchKernelGGL(activate_kernel, dim3(blocks), dim3(kSumThreads), 0, stream, p);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    e = launch_product_any<FMT, RG, 3>(p, t2, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(combine_kernel, dim3((p.N + 4 * kFours - 1) / (4 * kFours), p.T),
                       dim3(kSumThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

DecodeLayout decode_layout(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int64_t N,
                           int transpose_w13, int transpose_w2) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    DecodeLayout d{};
    const int64_t pairs = T * k;
    const int rg = row_fragments(T, k, E);
    // experts that get a pair if the choice is even, each with its rows' groups
    double groups = E * (1.0 - pow(1.0 - 1.0 / E, static_cast<double>(pairs)));
    const double full = pairs / (groups * 16 * rg);
    if (full > 1.0) groups *= full;
    d.gate_up = part_shape(groups, pairs / groups, H, 2 * I, transpose_w13, rg, 1);
    d.down = part_shape(groups, pairs / groups, I, N, transpose_w2, rg, 3);
    d.row_fragments = rg;
    d.gu = 0;
    d.y = up(sizeof(float) * d.gate_up.chunks * pairs * 2 * I);
    d.h = d.y + up(sizeof(float) * d.down.chunks * pairs * N);
    d.activate = pairs >= kActivatePairs;
    d.total = d.h + (d.activate ? up(sizeof(uint16_t) * 3 * pairs * I) : 0);
    return d;
}

hipError_t launch_decode(const DecodeParams &p, int transpose_w13, int transpose_w2, int e5m2,
                         hipStream_t stream) {
    if (e5m2) {
        if (p.row_fragments == 1)
            return launch_decode_t<1, 1>(p, transpose_w13, transpose_w2, stream);
        return launch_decode_t<1, 2>(p, transpose_w13, transpose_w2, stream);
    }
    if (p.row_fragments == 1) return launch_decode_t<0, 1>(p, transpose_w13, transpose_w2, stream);
    return launch_decode_t<0, 2>(p, transpose_w13, transpose_w2, stream);
}

}  // namespace gfr
