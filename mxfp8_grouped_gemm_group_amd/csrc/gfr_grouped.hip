// Products of rows sorted by expert with their expert's weights in 16 bits, and the
// weights' gradients.  include/gfr.h states the operators.
//
//   forward   out[t, n] = sum_k x[t, k] w[e, k, n]: lines are a group's rows, summed
//             over K (also the gradient by x, on the weights' other layout)
//   wgrad     out[e, k, n] = sum_t x[t, k] dy[t, n]: lines are columns of both, summed
//             over a group's rows
//
// Every block makes the groups' row ranges from group_list itself (a scan of at
// most 1024 numbers), so nothing is launched ahead and nothing is read on the host.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gfr.h"
#include "gfr_device.h"
#include "gfr_direct.h"
#include "gfr_layer.h"
#include "gfr_tile.h"

namespace gfr {
namespace {

// The groups: rows [start[e], start[e + 1]) are expert e's, start[E] all of them;
// units[e] counts the row blocks (of a kernel's height) of the experts before e,
// units[E] of all, and units[E + 1] also those of the rows behind the last group;
// cost[e] the time of a column of tiles of the experts before e, in a measure of the
// kernel's.
struct Groups {
    int start[GFR_MAX_EXPERTS + 2];
    int units[GFR_MAX_EXPERTS + 2];
    int cost[GFR_MAX_EXPERTS + 1];
    uint32_t waves[2][16];
};

// Exclusive prefix sum over a block of THREADS threads.
template <int THREADS>
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t *waves, uint32_t &total) {
    const int wave = threadIdx.x >> 6;
    const uint32_t upto = wave_prefix(v);
    if ((threadIdx.x & 63) == 63) waves[wave] = upto;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) before += waves[w];
        total += waves[w];
    }
    __syncthreads();
    return before + upto - v;
}

// Counts below zero or beyond M are clamped into [0, M], and the ranges, one behind
// another, into [0, M); either is a bad list.  256 threads take part; ends with a barrier.
template <int UNIT, int THREADS, class Cost>
__device__ __forceinline__ void find_groups(const GroupedParams &p, Groups &s, Cost cost_of) {
    constexpr int kPer = GFR_MAX_EXPERTS / 256;
    const int e0 = threadIdx.x * kPer;
    int64_t g[kPer + 1];
    g[0] = p.cumsum && e0 > 0 && e0 <= p.E ? p.group_list[e0 - 1] : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) g[i + 1] = e0 + i < p.E ? p.group_list[e0 + i] : 0;
    bool bad = false;
    int64_t count[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        int64_t c = e0 + i < p.E ? (p.cumsum ? g[i + 1] - g[i] : g[i + 1]) : 0;
        bad |= c < 0 || c > p.M;
        c = c < 0 ? 0 : c > p.M ? p.M : c;
        count[i] = c;
        sum += c;
    }
    // (two scans of 16 bits and the rest: 1024 counts of 31 bits do not fit one)
    uint32_t low_total, high_total, total;
    const uint32_t low =
        block_prefix<THREADS>(static_cast<uint32_t>(sum & 0xffff), s.waves[0], low_total);
    const uint32_t high =
        block_prefix<THREADS>(static_cast<uint32_t>(sum >> 16), s.waves[1], high_total);
    int64_t run = static_cast<int64_t>(low) + (static_cast<int64_t>(high) << 16);
    bad |= static_cast<int64_t>(low_total) + (static_cast<int64_t>(high_total) << 16) > p.M;
    uint32_t n = 0, cost = 0, cost_total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t first = run < p.M ? run : p.M;
        run += count[i];
        const int64_t end = run < p.M ? run : p.M;
        count[i] = end - first;
        if (e0 + i < p.E) s.start[e0 + i] = static_cast<int>(first);
        if (e0 + i == p.E - 1) s.start[p.E] = static_cast<int>(end);
        n += static_cast<uint32_t>((count[i] + UNIT - 1) / UNIT);
        if (e0 + i < p.E) cost += cost_of(static_cast<int>(count[i]));
    }
    uint32_t at = block_prefix<THREADS>(n, s.waves[0], total);
    cost = block_prefix<THREADS>(cost, s.waves[1], cost_total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (e0 + i < p.E) {
            s.units[e0 + i] = static_cast<int>(at);
            s.cost[e0 + i] = static_cast<int>(cost);
        }
        at += static_cast<uint32_t>((count[i] + UNIT - 1) / UNIT);
        cost += cost_of(static_cast<int>(count[i]));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        s.start[p.E + 1] = p.M;
        s.units[p.E] = static_cast<int>(total);
        s.cost[p.E] = static_cast<int>(cost_total);
        s.units[p.E + 1] = static_cast<int>(total) + (p.M - s.start[p.E] + UNIT - 1) / UNIT;
    }
    if (bad && p.status && blockIdx.x == 0) atomicOr(p.status, GFR_DEV_BAD_GROUP_LIST);
    __syncthreads();
}

// The expert whose units hold unit u (E: the rows behind the last group).
__device__ __forceinline__ int expert_of(const Groups &s, int E, int u) {
    int lo = 0, hi = E;                  // units[lo] <= u < units[hi + 1]
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (uniform(s.units[mid]) <= u) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ---------------------------------------------------------------------------
// General kernel: any K and N
// ---------------------------------------------------------------------------

// One operand's T lines of a step, T / 32 pieces a thread, through registers.
// k-major: lines are rows of `ld` = K elements, of which the step's 64 may end
// early.  line-major: the step's k are rows of `ld` elements, `k_end` of them.
template <bool LINE, int T, int D>
struct Staged {
    static constexpr int kPieces = T / 32;
    const uint16_t *base;      // k-major: the tile's first line; else its first column at k 0
    int64_t ld, elements;      // of a row; from base to the end of what may be read
    int k_end, lines, tid;     // tid: of the 256 threads that take the tile
    u4_t v[D][kPieces];

    __device__ __forceinline__ void tile(const uint16_t *base_, int64_t ld_, int64_t elements_,
                                         int k_end_, int lines_) {
        base = base_, ld = ld_, elements = elements_, k_end = k_end_, lines = lines_;
        tid = threadIdx.x & 255;
    }
    __device__ __forceinline__ void fetch(u4_t (&to)[kPieces], int step) {
        const bool whole = ld % 8 == 0;
        if (!LINE) {
            const int skew = reinterpret_cast<uintptr_t>(base) & 2;
            const rsrc_t r = buffer(reinterpret_cast<const char *>(base) - skew,
                                    2 * elements + skew);
            const int piece = tid & 7, valid = k_end - 64 * step - 8 * piece;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int line = (tid >> 3) + 32 * i;
                const int off = line * static_cast<int>(2 * ld) + skew + 128 * step + 16 * piece;
                to[i] = u4_t{0, 0, 0, 0};
                if (line < lines && valid > 0)
                    to[i] = valid >= 8 ? eight_of(r, off, whole) : eight_first(r, off, valid);
            }
        } else {
            const uint16_t *at = base + 64 * step * ld;
            const int skew = reinterpret_cast<uintptr_t>(at) & 2;
            const rsrc_t r = buffer(reinterpret_cast<const char *>(at) - skew,
                                    2 * (elements - 64 * step * ld) + skew);
            constexpr int kPer = T / 8;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int k = tid / kPer + 256 / kPer * i;
                const int off =
                    k * static_cast<int>(2 * ld) + skew + 16 * (tid % kPer);
                to[i] = u4_t{0, 0, 0, 0};
                if (64 * step + k < k_end) to[i] = eight_of(r, off, whole);
            }
        }
    }
    __device__ __forceinline__ void put(u4_t *tile, const u4_t (&from)[kPieces]) const {
        constexpr int kPer = T / 8;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            tile[LINE ? piece_line<T>(tid / kPer + 256 / kPer * i, tid % kPer)
                      : piece_k((tid >> 3) + 32 * i, tid & 7)] = from[i];
    }
};

// T x T tiles of G groups of four waves, each with the loads of two of its steps in flight
// in registers.  The groups take steps in turn and add up what they have in LDS: what
// bounds a step of few tiles is its loads' latency, and G groups have G steps on their way
// (512 rows of one expert of 2048 x 1024: 26.0 us with one group, which had four steps in
// flight, 18.8 with two, 17.2 with four; 64 rows over 8 experts of 4096 x 1024 31.6 and 25.6).
template <bool F16, bool WGRAD, bool WLINE, int T, int G>
__global__ __launch_bounds__(G * 256, G == 1 ? 2 : 4) void general_kernel(GroupedParams p) {
    constexpr int D = 2, F = T / 64;
    __shared__ Groups s;
    __shared__ u4_t tile[G][2][2][T * 8];
    find_groups<T, G * 256>(p, s, [](int) { return 0u; });
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6 & 3);
    const int half = G == 1 ? 0 : uniform(threadIdx.x >> 8);
    const int wm = wave / 2 * (T / 2), wn = wave % 2 * (T / 2);
    const int tiles_n = (p.N + T - 1) / T, tiles_k = (p.K + T - 1) / T;
    const int64_t total = WGRAD ? static_cast<int64_t>(p.E) * tiles_k * tiles_n
                                : static_cast<int64_t>(s.units[p.fill ? p.E + 1 : p.E]) * tiles_n;
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        int e, m0, rows, steps;
        const int n0 = static_cast<int>(id % tiles_n) * T;
        Staged<WGRAD, T, D> a;
        Staged<WLINE, T, D> b;
        if (WGRAD) {
            const int64_t rest = id / tiles_n;
            e = static_cast<int>(rest / tiles_k);
            m0 = static_cast<int>(rest % tiles_k) * T;
            rows = min(T, p.K - m0);
            const int first = s.start[e], count = s.start[e + 1] - first;
            steps = (count + 63) / 64;
            if (p.accumulate && count == 0) continue;
            a.tile(p.x + static_cast<int64_t>(first) * p.K + m0, p.K,
                   static_cast<int64_t>(count) * p.K - m0, count, T);
            b.tile(p.w + static_cast<int64_t>(first) * p.N + n0, p.N,
                   static_cast<int64_t>(count) * p.N - n0, count, T);
        } else {
            const int u = uniform(static_cast<int>(id / tiles_n));
            e = expert_of(s, p.E, u);
            m0 = s.start[e] + (u - s.units[e]) * T;
            rows = min(T, s.start[e + 1] - m0);
            steps = e < p.E ? (p.K + 63) / 64 : 0;
            const uint16_t *w = p.w + static_cast<int64_t>(e) * p.K * p.N;
            a.tile(p.x + static_cast<int64_t>(m0) * p.K, p.K, static_cast<int64_t>(rows) * p.K,
                   p.K, rows);
            if (WLINE)
                b.tile(w + n0, p.N, static_cast<int64_t>(p.K) * p.N - n0, p.K, T);
            else
                b.tile(w + static_cast<int64_t>(n0) * p.K, p.K,
                       static_cast<int64_t>(min(T, p.N - n0)) * p.K, p.K, min(T, p.N - n0));
        }
        f16_t acc[F][F] = {};
        // this group's steps: half, half + G, ...
        const int mine = (steps - half + G - 1) / G, rounds = (steps + G - 1) / G;
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (d < mine) a.fetch(a.v[d], half + G * d), b.fetch(b.v[d], half + G * d);
        for (int first = 0; first < rounds; first += D)
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int n = first + d;
                if (n >= rounds) break;
                // (a stage is written again two rounds later: behind the barrier between)
                u4_t(&to)[2][T * 8] = tile[half][d & 1];
                if (n < mine) {
                    a.put(to[0], a.v[d]);
                    b.put(to[1], b.v[d]);
                }
                __syncthreads();
                if (n >= mine) continue;
                if (n + D < mine) {
                    a.fetch(a.v[d], half + G * (n + D));
                    b.fetch(b.v[d], half + G * (n + D));
                }
#pragma unroll
                for (int part = 0; part < 4; ++part) {
                    u4_t fa[F], fb[F];
#pragma unroll
                    for (int i = 0; i < F; ++i) {
                        fa[i] = fragment<WGRAD, T>(to[0], wm + 32 * i, part, lane);
                        fb[i] = fragment<WLINE, T>(to[1], wn + 32 * i, part, lane);
                    }
#pragma unroll
                    for (int i = 0; i < F; ++i)
#pragma unroll
                        for (int j = 0; j < F; ++j)
                            acc[i][j] = mfma32<F16>(fb[j], fa[i], acc[i][j]);
                }
            }
        __syncthreads();
        // Lane l holds line 32 i + l % 32, columns 32 j + 8 r + 4 (l / 32) .. + 3.  A wave's
        // results go through its part of the stages, four columns of row m at piece j ^
        // m, so that rows are written in runs (straight from here a store took 64
        // places: zeros for 105 empty experts of 676 x 3588 0.7 ms).
        constexpr int W = T / 2, kRow = W / 4;          // a wave's rows and columns; pieces
        f4_t *const slab = reinterpret_cast<f4_t *>(tile) + wave * W * kRow;
        constexpr int kGroup = 4 * W * kRow;            // pieces of a group's results
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int m = 32 * i + (lane & 31), piece = 8 * j + 2 * r + (lane >> 5);
                    slab[half * kGroup + m * kRow + (piece ^ (m & (kRow - 1)))] =
                        f4_t{acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2],
                             acc[i][j][4 * r + 3]};
                }
        __syncthreads();
        const int64_t row0 = (WGRAD ? static_cast<int64_t>(e) * p.K : 0) + m0 + wm;
        if (p.N % 4 == 0) {
            // four columns a lane
            for (int k = lane + 64 * half; k < W * kRow; k += 64 * G) {
                const int m = k / kRow, n = n0 + wn + 4 * (k % kRow);
                if (wm + m >= rows || n >= p.N) continue;
                const int64_t at = (row0 + m) * p.N + n;
                const f4_t *from = slab + m * kRow + (k % kRow ^ (m & (kRow - 1)));
                f4_t y = from[0];
#pragma unroll
                for (int g = 1; g < G; ++g) y += from[g * kGroup];
                if (p.out_f32) {
                    f4_t *to = reinterpret_cast<f4_t *>(static_cast<float *>(p.out) + at);
                    if (p.accumulate) y += *to;
                    *to = y;
                } else {
                    u2_t *to = reinterpret_cast<u2_t *>(static_cast<uint16_t *>(p.out) + at);
                    if (p.accumulate) {
                        const u2_t old = *to;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            y[q] += unpack1<F16>(old[q >> 1] >> (16 * (q & 1)));
                    }
                    *to = u2_t{pack2<F16>(y[0], y[1]), pack2<F16>(y[2], y[3])};
                }
            }
        } else {
            // a column a lane
            for (int k = lane + 64 * half; k < W * W; k += 64 * G) {
                const int m = k / W, c = k % W, n = n0 + wn + c;
                if (wm + m >= rows || n >= p.N) continue;
                const int64_t at = (row0 + m) * p.N + n;
                const f4_t *from = slab + m * kRow + (c / 4 ^ (m & (kRow - 1)));
                float y = from[0][c % 4];
#pragma unroll
                for (int g = 1; g < G; ++g) y += from[g * kGroup][c % 4];
                if (p.out_f32) {
                    float *to = static_cast<float *>(p.out) + at;
                    *to = p.accumulate ? *to + y : y;
                } else {
                    uint16_t *to = static_cast<uint16_t *>(p.out) + at;
                    if (p.accumulate) y += unpack1<F16>(*to);
                    *to = static_cast<uint16_t>(pack2<F16>(y, 0.0f));
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Direct kernel: rows of whole pieces
// ---------------------------------------------------------------------------
constexpr int kPitch = 36;      // floats of a row of 32 results in LDS: spreads rows over banks
constexpr int kSlab = 17 * kPitch;
static_assert(kWaves * kSlab % 4 == 0, "the groups begin at a whole piece");
constexpr int kDirectLds = 2 * kStage * 16 + kWaves * kSlab * 4 +
                           static_cast<int>(sizeof(Groups));
static_assert(kDirectLds <= kMaxLds, "as allow_lds allows");

// The last of E + 1 experts whose entry is at most u, found by a wave side by side.
__device__ __forceinline__ int expert_at(const int *from, int E, int u, int lane) {
    int n = 0;
    for (int e = 0; e <= E; e += 64)
        n += __builtin_popcountll(
            __builtin_amdgcn_ballot_w64((e + lane <= E) & (from[min(e + lane, E)] <= u)));
    return uniform(n - 1);
}

// How results are written: FP32 or 16 bits, added to what is there or not; or, for rows
// that begin anywhere, element by element.
enum Store { kF32, kF32Add, k16, k16Add, kElements };

// 32 x 32 results of a wave (lane l: row l % 32, columns 8 r + 4 (l / 32) .. + 3) to
// `rows` rows from `row` on, columns from n0 on.  No branch of a lane's own: the block's
// tiles and loads stay in scalar registers.
template <bool F16, int STORE>
__device__ __forceinline__ void put_block(const GroupedParams &p, float *slab, const f16_t &v,
                                          int64_t row, int rows, int n0, int lane) {
    const int shift = STORE == kF32 || STORE == kF32Add ? 2
                      : STORE == kElements              ? p.out_f32 + 1
                                                        : 1;
    const int row_bytes = p.N << shift, g = lane >> 5;
    char *const out = static_cast<char *>(p.out) + row * row_bytes;
    // (a buffer over the rows: what is behind the last one is not written)
    const int64_t bytes = static_cast<int64_t>(max(0, min(32, rows))) * row_bytes;
    if (STORE == kElements) {
        auto wave_sync = [] {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        // through the wave's own LDS, 16 rows at a time: a column per lane
        const int n = n0 + (lane & 31), skew = reinterpret_cast<uintptr_t>(out) & 2;
        const rsrc_t to = uniform_buffer(out - skew, bytes + skew);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // (the other half's go to a row that nobody reads)
            const int line = (lane >> 4 & 1) == h ? lane & 15 : 16;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<f4_t *>(&slab[line * kPitch + 8 * r + 4 * g]) =
                    f4_t{v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
            wave_sync();
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
                const int m = 2 * q + g;
                const float y = slab[m * kPitch + (lane & 31)];
                const int off =
                    n < p.N ? (16 * h + m) * row_bytes + (n << shift) + skew : kPast;
                if (p.out_f32)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y), to, off, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b16(
                        static_cast<uint16_t>(pack2<F16>(y, 0.0f)), to, off, 0, 0);
            }
            wave_sync();
        }
        return;
    }
    // Lanes trade what they hold (halves of 32, then rows of 16 lanes), until a store's 64
    // lanes have 16 rows of 64 bytes.
    const rsrc_t to = uniform_buffer(out, bytes);
    const int at = (lane & 15) * row_bytes;
    if (STORE == kF32 || STORE == kF32Add) {
        const int col = 8 * (lane >> 4 & 1) + 4 * g;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            u4_t y[2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[8 * q + j]),
                                                                __float_as_uint(v[8 * q + 4 + j]),
                                                                false, false);
                y[0][j] = w[0];
                y[1][j] = w[1];
            }
            const int n = n0 + 16 * q + col;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int off = n < p.N ? at + 16 * h * row_bytes + 4 * n : kPast;
                f4_t sum = __builtin_bit_cast(f4_t, y[h]);
                if (STORE == kF32Add) sum += __builtin_bit_cast(f4_t, load16<0>(to, off, 0));
                store16(to, __builtin_bit_cast(u4_t, sum), off);
            }
        }
        return;
    }
    const int n = n0 + 16 * (lane >> 4 & 1) + 8 * g;
    if (STORE == k16Add) {
        // eight columns a lane in FP32: the lane's row is lane % 32 still
        const int full = (lane & 31) * row_bytes;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int c = n0 + 16 * q + 8 * g, off = c < p.N ? full + 2 * c : kPast;
            float y[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[8 * q + j]),
                                                                __float_as_uint(v[8 * q + 4 + j]),
                                                                false, false);
                y[j] = __uint_as_float(w[0]);
                y[4 + j] = __uint_as_float(w[1]);
            }
            const u4_t old = load16<0>(to, off, 0);
            u4_t h;
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += unpack1<F16>(old[j >> 1] >> (16 * (j & 1)));
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = pack2<F16>(y[2 * j], y[2 * j + 1]);
            store16(to, h, off);
        }
        return;
    }
    u4_t h[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const auto w = __builtin_amdgcn_permlane32_swap(
                pack2<F16>(v[8 * q + 2 * j], v[8 * q + 2 * j + 1]),
                pack2<F16>(v[8 * q + 4 + 2 * j], v[8 * q + 5 + 2 * j]), false, false);
            h[q][j] = w[0];
            h[q][2 + j] = w[1];
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const auto w = __builtin_amdgcn_permlane16_swap(h[0][j], h[1][j], false, false);
        h[0][j] = w[0];
        h[1][j] = w[1];
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
        store16(to, h[q], n < p.N ? at + 16 * q * row_bytes + 2 * n : kPast);
}

// Stores of a wave's 32 x 32 results, at least.
constexpr int block_stores(int store) {
    return store == k16 || store == k16Add ? 2 : 4;
}

// The block's run: Blocks go round the eight XCDs; each XCD takes a run of tiles, an eighth
// of the time.
template <bool WGRAD, bool WLINE>
struct GroupedTiles {
    const GroupedParams &p;
    const Groups &s;
    int lane, tiles_n, tiles_k, total;
    Divisor by_n, by_k, by_band;
    int begin, end, stride;

    __device__ __forceinline__ GroupedTiles(const GroupedParams &p_, const Groups &s_)
        : p(p_), s(s_), lane(threadIdx.x & 63), tiles_n((p.N + kTile - 1) / kTile),
          tiles_k((p.K + kTile - 1) / kTile),
          total(tiles_n * (WGRAD ? p.E * tiles_k : uniform(s.units[p.E]))),
          by_n(tiles_n), by_k(tiles_k), by_band(8 * tiles_n) {
        const int xcd = blockIdx.x & 7;
        stride = gridDim.x >> 3;
        begin = run_begin(xcd) + (blockIdx.x >> 3);
        end = run_begin(xcd + 1);
    }
    __device__ __forceinline__ int run_begin(int x) const {
        if (x == 0) return 0;
        if (x == 8) return total;
        const int64_t place = static_cast<int64_t>(uniform(s.cost[p.E])) * x;   // in eighths
        const int e = expert_at(s.cost, p.E, static_cast<int>(place >> 3), lane);
        if (e >= p.E) return total;
        // (the cost of the experts before e is at most the place, and that of e too is more)
        const int64_t cost = uniform(s.cost[e + 1]) - uniform(s.cost[e]);
        const int first = WGRAD ? e * tiles_k : uniform(s.units[e]);
        const int units = WGRAD ? tiles_k : uniform(s.units[e + 1]) - first;
        const int64_t in = place - 8 * static_cast<int64_t>(uniform(s.cost[e]));
        return uniform(first * tiles_n + static_cast<int>(in * units * tiles_n / (8 * cost)));
    }
    __device__ __forceinline__ TileAt at(int id) const {
        TileAt t;
        if (WGRAD) {
            const int rest = by_n.of(id);
            t.n0 = (id - rest * tiles_n) * kTile;
            t.e = by_k.of(rest);
            t.m0 = (rest - t.e * tiles_k) * kTile;
            t.rows = min(kTile, p.K - t.m0);
            t.steps = uniform((s.start[t.e + 1] - s.start[t.e] + 63) / 64);
        } else {
            t.e = expert_at(s.units, p.E, by_n.of(id), lane);
            // within an expert, bands of eight units by all columns; a column's units begin
            // one further every 32 tiles, or a block would meet the same unit each time,
            // and the last one is cheaper
            const int u0 = uniform(s.units[t.e]), units = uniform(s.units[t.e + 1]) - u0;
            const int at = id - u0 * tiles_n;
            const int band = by_band.of(at), in_band = at - band * 8 * tiles_n;
            const int depth = min(8, units - band * 8), column = Divisor(depth).of(in_band);
            int unit = in_band - column * depth + (column * depth / 32) % depth;
            if (unit >= depth) unit -= depth;
            t.n0 = column * kTile;
            t.m0 = uniform(s.start[t.e]) + (band * 8 + unit) * kTile;
            t.rows = uniform(min(kTile, uniform(s.start[t.e + 1]) - t.m0));
            t.steps = uniform(t.e < p.E ? (p.K + 63) / 64 : 0);
        }
        t.m0 = uniform(t.m0);
        t.n0 = uniform(t.n0);
        return t;
    }
    static constexpr bool kExtra = false;
    struct Cursor {
        int id;
        __device__ __forceinline__ explicit Cursor(int first) : id(first) {}
    };
    template <class A, class B>
    __device__ __forceinline__ int next(Cursor &c, A &da, B &db, int wave, int lane) const {
        TileAt t;
        do {
            c.id = uniform(c.id + stride);
            if (c.id >= uniform(end)) return 0;
            t = at(c.id);
        } while (t.steps == 0);
        const int64_t k = p.K, n = p.N;
        if (WGRAD) {
            const int first = uniform(s.start[t.e]), count = uniform(s.start[t.e + 1]) - first;
            da.tile(p.x + first * k + t.m0, 2 * (count * k - t.m0), count, 0);
            db.tile(p.w + first * n + t.n0, 2 * (count * n - t.n0), count, 0);
        } else {
            const uint16_t *w = p.w + t.e * k * n;
            // Few rows: the weights' bytes bound it, and rows of w that lie a power of two
            // apart meet the same memory channels wherever all tiles are at the same k; so
            // column tiles begin at steps of their own (128 rows over 16 experts of 4096 x
            // 4096 120 -> 95 us).  Many rows share x's steps in L2: 8192 cubed 946 -> 992.
            const int turn = WLINE || !p.turn ? 0 : by_n.of(t.n0 / kTile * t.steps);
            da.tile(p.x + t.m0 * k, 2 * t.rows * k, p.K, t.rows, turn);
            if (WLINE) db.tile(w + t.n0, 2 * (k * n - t.n0), p.K, 0);
            else db.tile(w + t.n0 * k, 2 * min(kTile, p.N - t.n0) * k, p.K, 0, turn);
        }
        return t.steps;
    }
};

template <bool F16, bool WGRAD, bool WLINE>
struct GroupedFinish {
    static constexpr bool kLong = false;
    const GroupedParams &p;
    float *slab;

    __device__ __forceinline__ int64_t row0(const TileAt &t) const {
        return WGRAD ? static_cast<int64_t>(t.e) * p.K + t.m0 : t.m0;
    }
    template <int STORE, int FM, int FN>
    __device__ __forceinline__ int put(const TileAt &t, const f16_t (&acc)[FM][FN], int wm, int wn,
                                       int lane) const {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                put_block<F16, STORE>(p, slab, acc[i][j], row0(t) + wm + 32 * i,
                                      t.rows - wm - 32 * i, t.n0 + wn + 32 * j, lane);
                __builtin_amdgcn_sched_barrier(0);
            }
        return FM * FN * block_stores(STORE);
    }
    template <int FM, int FN>
    __device__ __forceinline__ int tile(const TileAt &t, const f16_t (&acc)[FM][FN], int wm, int wn,
                                        int lane) const {
        if (!WGRAD && !WLINE && !p.wide) return put<kElements>(t, acc, wm, wn, lane);
        if (WGRAD && p.accumulate)
            return p.out_f32 ? put<kF32Add>(t, acc, wm, wn, lane)
                             : put<k16Add>(t, acc, wm, wn, lane);
        return p.out_f32 ? put<kF32>(t, acc, wm, wn, lane) : put<k16>(t, acc, wm, wn, lane);
    }
    // Zeros (in wgrad of an empty group, if they are not added).
    __device__ __forceinline__ void clear(const TileAt &t) const {
        if (WGRAD && p.accumulate) return;
        const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
        const int shift = p.out_f32 ? 2 : 1, row_bytes = p.N << shift;
        const int columns = min(kTile, p.N - t.n0) << shift;
        for (int m = wave; m < t.rows; m += kWaves) {
            char *const to =
                static_cast<char *>(p.out) + (row0(t) + m) * row_bytes + (t.n0 << shift);
            const int skew = reinterpret_cast<uintptr_t>(to) & 2;
            const rsrc_t r = uniform_buffer(to - skew, columns + skew);
            if (p.wide) {
                store16(r, u4_t{0, 0, 0, 0}, 16 * lane);
            } else {
                for (int i = 0; i < columns; i += 128)
                    __builtin_amdgcn_raw_buffer_store_b16(0, r, skew + i + 2 * lane, 0, 0);
            }
        }
    }
};

template <bool F16, bool WGRAD, bool WLINE>
__global__ __launch_bounds__(kWaves * 64, 1) void direct_kernel(GroupedParams p) {
    extern __shared__ u4_t lds[];     // [2][A's 256 lines, B's][8], the waves' results, the groups
    Groups &s = *reinterpret_cast<Groups *>(lds + 2 * kStage + kWaves * kSlab / 4);
    // A tile's time: wgrad, its steps and about two more; forward, its rows by the tile
    // shapes there are.
    find_groups<kTile, kWaves * 64>(p, s, [](int count) -> uint32_t {
        if (WGRAD) return (count + 63) / 64 + 2;
        return 4 * (count / kTile) + (count % kTile + 63) / 64;
    });
    float *const slab =
        reinterpret_cast<float *>(lds + 2 * kStage) + uniform(threadIdx.x >> 6) * kSlab;
    const GroupedTiles<WGRAD, WLINE> tiles(p, s);
    const GroupedFinish<F16, WGRAD, WLINE> finish{p, slab};
    run_tiles<F16, WGRAD, WLINE>(lds, tiles, finish, p.K, WLINE ? p.N : p.K);
    // the rows behind the last group, by all blocks
    if (!WGRAD && p.fill) {
        const int all = tiles.tiles_n * uniform(s.units[p.E + 1]);
        for (int id = tiles.total + blockIdx.x; id < all; id += gridDim.x)
            finish.clear(tiles.at(id));
    }
}

template <bool F16, bool WGRAD, bool WLINE, int T, int G>
hipError_t launch_general_t(const GroupedParams &p, hipStream_t stream) {
    hipLaunchKernelGGL((general_kernel<F16, WGRAD, WLINE, T, G>), dim3(G == 4 ? 256 : 512),
                       dim3(G * 256), 0, stream, p);
    return hipGetLastError();
}

template <bool F16, bool WGRAD, bool WLINE>
hipError_t launch_direct(const GroupedParams &p, hipStream_t stream) {
    constexpr auto kernel = &direct_kernel<F16, WGRAD, WLINE>;
    if (hipError_t e = allow_lds<kernel, kMaxLds>(kDirectLds); e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(256), dim3(kWaves * 64), kDirectLds, stream, p);
    return hipGetLastError();
}

template <bool F16, bool WGRAD, bool WLINE>
hipError_t launch_kernel(const GroupedParams &p, hipStream_t stream) {
    switch (p.kernel) {
    case GroupedKernel::kDirect: return launch_direct<F16, WGRAD, WLINE>(p, stream);
    case GroupedKernel::k128: return launch_general_t<F16, WGRAD, WLINE, 128, 1>(p, stream);
    case GroupedKernel::k64Long: return launch_general_t<F16, WGRAD, WLINE, 64, 4>(p, stream);
    default: return launch_general_t<F16, WGRAD, WLINE, 64, 2>(p, stream);
    }
}

template <bool F16>
hipError_t launch_grouped_t(const GroupedParams &p, hipStream_t stream) {
    if (p.wgrad) return launch_kernel<F16, true, true>(p, stream);
    return p.transpose ? launch_kernel<F16, false, false>(p, stream)
                       : launch_kernel<F16, false, true>(p, stream);
}

}  // namespace

// The kernel for a size, by estimated time; groups are taken as equal, an expert as
// having a row if there is one for it.  A block's time per 64-step of the direct kernel
// by its tile's rows, with the CUs one round after the other; of the general kernel by the
// tiles a CU has.  Four groups of waves begin later than two and end sooner from 20 steps
// on, as long as the tiles fill no more than the CUs (16 steps of 256 tiles 13.1 us and
// 12.5, 32 steps of 512 40.6 and 36.7).  (Direct against general, us: 8 rows over 256
// experts of 2048 x 1024 24 and 17.6; 64 over 64 27 and 45; 64 over 8 of 4096 x 1024 38.5
// and 25.6; 512 of one 46 and 17.2; 2048 of one of 4096 x 2048 85 and 100; wgrad of 1024
// rows of one of 1024 x 1024 29 and 13, of 2048 rows of one of 4096 x 2048 52 and 59.)
GroupedKernel grouped_kernel(int wgrad, int transpose, int64_t M, int64_t E, int64_t K, int64_t N) {
    const auto up = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
    const auto most = [](double a, double b) { return a > b ? a : b; };
    const int64_t experts = E < M ? E : M, rows = experts > 0 ? up(M, experts) : 0;
    const auto tiles = [&](int64_t t) {
        return wgrad ? static_cast<double>(E * up(K, t)) * static_cast<double>(up(N, t))
                     : static_cast<double>(experts * up(rows, t)) * static_cast<double>(up(N, t));
    };
    const double steps = static_cast<double>(up(wgrad ? rows : K, 64));
    const bool by_groups = tiles(64) <= 256.0 && steps >= 20.0;
    const GroupedKernel general = by_groups            ? GroupedKernel::k64Long
                                  : tiles(128) < 512.0 ? GroupedKernel::k64
                                                       : GroupedKernel::k128;
    // rows of whole pieces, of every operand that is loaded
    if (K % 8 != 0 || (N % 8 != 0 && (wgrad || !transpose))) return general;
    const double rounds = static_cast<double>(static_cast<int64_t>(tiles(256) / 256.0 + 0.999));
    const double step = wgrad || rows > 192 ? 1.2
                        : rows > 128        ? 1.0
                        : rows > 64         ? 0.8
                        : rows > 32         ? 0.56
                                            : 0.47;
    const double direct = 8.0 + rounds * (steps * step + (wgrad ? 3.0 : 0.0));
    const double fill = most(1.0, tiles(64) / 256.0);
    const double step64 = general == GroupedKernel::k64 ? 0.46 : 0.375;
    const double other = by_groups ? 8.9 + steps * 0.26
                                   : 5.0 + fill * (steps * step64 + (wgrad ? 0.5 : 0.0));
    return direct <= other ? GroupedKernel::kDirect : general;
}

hipError_t launch_grouped(const GroupedParams &p, hipStream_t stream) {
    return p.f16 ? launch_grouped_t<true>(p, stream) : launch_grouped_t<false>(p, stream);
}

}  // namespace gfr
