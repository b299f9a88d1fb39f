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

#include <type_traits>

#include "gfr.h"
#include "gfr_device.h"
#include "gfr_layer.h"
#include "gfr_tile.h"

namespace gfr {
namespace {

// The groups: rows [start[e], start[e + 1]) are expert e's, start[E] all of them;
// units[e] counts the row blocks (of a kernel's height) of the experts before e,
// units[E] of all, and units[E + 1] also those of the rows behind the last group.
struct Groups {
    int start[GFR_MAX_EXPERTS + 2];
    int units[GFR_MAX_EXPERTS + 2];
    uint32_t waves[2][4];
};

// Exclusive prefix sum over a block of 256 threads.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t *waves, uint32_t &total) {
    const int wave = threadIdx.x >> 6;
    const uint32_t upto = wave_prefix(v);
    if ((threadIdx.x & 63) == 63) waves[wave] = upto;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < wave) before += waves[w];
        total += waves[w];
    }
    __syncthreads();
    return before + upto - v;
}

// Counts below zero or beyond M are clamped into [0, M], and the ranges, one behind
// another, into [0, M); either is a bad list.  256 threads; ends with a barrier.
template <int UNIT>
__device__ __forceinline__ void find_groups(const GroupedParams &p, Groups &s) {
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
    const uint32_t low = block_prefix(static_cast<uint32_t>(sum & 0xffff), s.waves[0], low_total);
    const uint32_t high = block_prefix(static_cast<uint32_t>(sum >> 16), s.waves[1], high_total);
    int64_t run = static_cast<int64_t>(low) + (static_cast<int64_t>(high) << 16);
    bad |= static_cast<int64_t>(low_total) + (static_cast<int64_t>(high_total) << 16) > p.M;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t first = run < p.M ? run : p.M;
        run += count[i];
        const int64_t end = run < p.M ? run : p.M;
        count[i] = end - first;
        if (e0 + i < p.E) s.start[e0 + i] = static_cast<int>(first);
        if (e0 + i == p.E - 1) s.start[p.E] = static_cast<int>(end);
        n += static_cast<uint32_t>((count[i] + UNIT - 1) / UNIT);
    }
    uint32_t at = block_prefix(n, s.waves[0], total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (e0 + i < p.E) s.units[e0 + i] = static_cast<int>(at);
        at += static_cast<uint32_t>((count[i] + UNIT - 1) / UNIT);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        s.start[p.E + 1] = p.M;
        s.units[p.E] = static_cast<int>(total);
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

// Four neighbouring results of a row, columns n .. n + 3 of N.
template <bool F16>
__device__ __forceinline__ void put4(const GroupedParams &p, int64_t row, int n, const float (&v)[4]) {
    const int64_t at = row * p.N + n;
    if (p.wide) {
        if (n >= p.N) return;
        float y[4] = {v[0], v[1], v[2], v[3]};
        if (p.out_f32) {
            f4_t *to = reinterpret_cast<f4_t *>(static_cast<float *>(p.out) + at);
            f4_t o = {y[0], y[1], y[2], y[3]};
            if (p.accumulate) o += *to;
            *to = o;
            return;
        }
        u2_t *to = reinterpret_cast<u2_t *>(static_cast<uint16_t *>(p.out) + at);
        if (p.accumulate) {
            const u2_t old = *to;
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] += unpack1<F16>(old[j >> 1] >> (16 * (j & 1)));
        }
        *to = u2_t{pack2<F16>(y[0], y[1]), pack2<F16>(y[2], y[3])};
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= p.N) return;
        float y = v[j];
        if (p.out_f32) {
            float *to = static_cast<float *>(p.out) + at + j;
            *to = p.accumulate ? *to + y : y;
        } else {
            uint16_t *to = static_cast<uint16_t *>(p.out) + at + j;
            if (p.accumulate) y += unpack1<F16>(*to);
            *to = static_cast<uint16_t>(pack2<F16>(y, 0.0f));
        }
    }
}

// ---------------------------------------------------------------------------
// General kernel: any K and N
// ---------------------------------------------------------------------------

// One operand's 128 lines of a step, four pieces a thread, through registers.
// k-major: lines are rows of `ld` = K elements, of which the step's 64 may end
// early.  line-major: the step's k are rows of `ld` elements, `k_end` of them.
template <bool LINE>
struct Staged {
    const uint16_t *base;      // k-major: the tile's first line; line-major: its first column at k 0
    int64_t ld, elements;      // of a row; from base to the end of what may be read
    int k_end, lines;
    u4_t v[4];

    __device__ __forceinline__ void fetch(int step) {
        const bool whole = ld % 8 == 0;
        if (!LINE) {
            const int skew = reinterpret_cast<uintptr_t>(base) & 2;
            const rsrc_t r = buffer(reinterpret_cast<const char *>(base) - skew,
                                    2 * elements + skew);
            const int piece = threadIdx.x & 7, valid = k_end - 64 * step - 8 * piece;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int line = (threadIdx.x >> 3) + 32 * i;
                const int off = line * static_cast<int>(2 * ld) + skew + 128 * step + 16 * piece;
                v[i] = u4_t{0, 0, 0, 0};
                if (line < lines && valid > 0)
                    v[i] = valid >= 8 ? eight_of(r, off, whole) : eight_first(r, off, valid);
            }
        } else {
            const uint16_t *at = base + 64 * step * ld;
            const int skew = reinterpret_cast<uintptr_t>(at) & 2;
            const rsrc_t r = buffer(reinterpret_cast<const char *>(at) - skew,
                                    2 * (elements - 64 * step * ld) + skew);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = (threadIdx.x >> 4) + 16 * i;
                const int off = k * static_cast<int>(2 * ld) + skew + 16 * (threadIdx.x & 15);
                v[i] = u4_t{0, 0, 0, 0};
                if (64 * step + k < k_end) v[i] = eight_of(r, off, whole);
            }
        }
    }
    __device__ __forceinline__ void put(u4_t *tile) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            tile[LINE ? piece_line<128>((threadIdx.x >> 4) + 16 * i, threadIdx.x & 15)
                      : piece_k((threadIdx.x >> 3) + 32 * i, threadIdx.x & 7)] = v[i];
    }
};

// 128 x 128 tiles of four waves, one step's loads in flight in registers.
template <bool F16, bool WGRAD, bool WLINE>
__global__ __launch_bounds__(256, 2) void general_kernel(GroupedParams p) {
    __shared__ Groups s;
    __shared__ u4_t tile[2][128 * 8];
    find_groups<128>(p, s);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wm = wave / 2 * 64, wn = wave % 2 * 64;
    const int tiles_n = (p.N + 127) / 128, tiles_k = (p.K + 127) / 128;
    const int64_t total = WGRAD ? static_cast<int64_t>(p.E) * tiles_k * tiles_n
                                : static_cast<int64_t>(s.units[p.fill ? p.E + 1 : p.E]) * tiles_n;
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        int e, m0, rows, steps;
        const int n0 = static_cast<int>(id % tiles_n) * 128;
        Staged<WGRAD> a;
        Staged<WLINE> b;
        if (WGRAD) {
            const int64_t rest = id / tiles_n;
            e = static_cast<int>(rest / tiles_k);
            m0 = static_cast<int>(rest % tiles_k) * 128;
            rows = min(128, p.K - m0);
            const int first = s.start[e], count = s.start[e + 1] - first;
            steps = (count + 63) / 64;
            if (p.accumulate && count == 0) continue;
            a = {p.x + static_cast<int64_t>(first) * p.K + m0, p.K,
                 static_cast<int64_t>(count) * p.K - m0, count, 128, {}};
            b = {p.w + static_cast<int64_t>(first) * p.N + n0, p.N,
                 static_cast<int64_t>(count) * p.N - n0, count, 128, {}};
        } else {
            const int u = uniform(static_cast<int>(id / tiles_n));
            e = expert_of(s, p.E, u);
            m0 = s.start[e] + (u - s.units[e]) * 128;
            rows = min(128, s.start[e + 1] - m0);
            steps = e < p.E ? (p.K + 63) / 64 : 0;
            const uint16_t *w = p.w + static_cast<int64_t>(e) * p.K * p.N;
            a = {p.x + static_cast<int64_t>(m0) * p.K, p.K, static_cast<int64_t>(rows) * p.K, p.K,
                 rows, {}};
            if (WLINE)
                b = {w + n0, p.N, static_cast<int64_t>(p.K) * p.N - n0, p.K, 128, {}};
            else
                b = {w + static_cast<int64_t>(n0) * p.K, p.K,
                     static_cast<int64_t>(min(128, p.N - n0)) * p.K, p.K, min(128, p.N - n0), {}};
        }
        f16_t acc[2][2] = {};
        if (steps > 0) a.fetch(0), b.fetch(0);
        for (int step = 0; step < steps; ++step) {
            __syncthreads();
            a.put(tile[0]);
            b.put(tile[1]);
            __syncthreads();
            if (step + 1 < steps) a.fetch(step + 1), b.fetch(step + 1);
#pragma unroll
            for (int part = 0; part < 4; ++part) {
                u4_t fa[2], fb[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    fa[i] = fragment<WGRAD, 128>(tile[0], wm + 32 * i, part, lane);
                    fb[i] = fragment<WLINE, 128>(tile[1], wn + 32 * i, part, lane);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[i][j] = mfma32<F16>(fb[j], fa[i], acc[i][j]);
            }
        }
        // lane l holds line 32 i + l % 32, columns 32 j + 8 r + 4 (l / 32) .. + 3
        const int64_t row0 = WGRAD ? static_cast<int64_t>(e) * p.K + m0 : m0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = wm + 32 * i + (lane & 31);
            if (m >= rows) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float v[4] = {acc[i][j][4 * r], acc[i][j][4 * r + 1],
                                        acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
                    put4<F16>(p, row0 + m, n0 + wn + 32 * j + 8 * r + 4 * (lane >> 5), v);
                }
        }
    }
}

// ---------------------------------------------------------------------------
// Direct kernel: rows of whole pieces
// ---------------------------------------------------------------------------

// BM x BN tiles in waves of WM x WN; a step is 64 of the summed index in two LDS
// stages, filled straight from memory, and four parts of 16.  While one part's MFMAs
// run, the next part's fragments come from LDS.  The one barrier of a step stands
// ahead of part 3, whose fragments are in registers by then: behind it the next
// step's stage is complete, and the loads of the step behind that go to this one.
constexpr int kPitch = 36;       // floats of a row of 32 results in LDS: spreads rows over banks

template <int BM, int BN, int WM, int WN>
constexpr int direct_lds() {
    return 2 * (BM + BN) * 128 + (BM / WM) * (BN / WN) * 32 * kPitch * 4 +
           static_cast<int>(sizeof(Groups));
}

// 32 x 32 results of a wave (lane l: row l % 32, columns 8 r + 4 (l / 32) .. + 3) to
// `rows` rows from `row` on, columns from n0 on.
template <bool F16>
__device__ __forceinline__ void put_block(const GroupedParams &p, float *slab, const f16_t &v,
                                          int64_t row, int rows, int n0, int lane) {
    auto wave_sync = [] {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
#pragma unroll
    for (int r = 0; r < 4; ++r)
        *reinterpret_cast<f4_t *>(&slab[(lane & 31) * kPitch + 8 * r + 4 * (lane >> 5)]) =
            f4_t{v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
    wave_sync();
    if (p.wide) {
        const int n = n0 + 8 * (lane & 3);
#pragma unroll 1
        for (int q = lane >> 2; q < 32; q += 16) {
            if (q >= rows || n >= p.N) break;
            const float *from = &slab[q * kPitch + 8 * (lane & 3)];
            f4_t y[2] = {load<f4_t>(from), load<f4_t>(from + 4)};
            const int64_t at = (row + q) * p.N + n;
            if (p.out_f32) {
                f4_t *to = reinterpret_cast<f4_t *>(static_cast<float *>(p.out) + at);
                if (p.accumulate) y[0] += to[0], y[1] += to[1];
                to[0] = y[0];
                to[1] = y[1];
            } else {
                u4_t *to = reinterpret_cast<u4_t *>(static_cast<uint16_t *>(p.out) + at);
                if (p.accumulate) {
                    const u4_t old = *to;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y[j >> 2][j & 3] += unpack1<F16>(old[j >> 1] >> (16 * (j & 1)));
                }
                u4_t h;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[j] = pack2<F16>(y[j >> 1][2 * (j & 1)], y[j >> 1][2 * (j & 1) + 1]);
                *to = h;
            }
        }
    } else {
        // rows that begin anywhere: a column per lane
        const int n = n0 + (lane & 31);
#pragma unroll 1
        for (int q = lane >> 5; q < 32; q += 2) {
            if (q >= rows || n >= p.N) break;
            float y = slab[q * kPitch + (lane & 31)];
            const int64_t at = (row + q) * p.N + n;
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
    wave_sync();
}

template <bool F16, bool WGRAD, bool WLINE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, (BM / WM) * (BN / WN) / 4)
void direct_kernel(GroupedParams p) {
    constexpr int kWaves = (BM / WM) * (BN / WN);
    constexpr int FM = WM / 32, FN = WN / 32;
    constexpr int kStage = (BM + BN) * 8;                  // pieces
    extern __shared__ u4_t lds[];            // [2][BM + BN][8], the waves' results, the groups
    Groups &s = *reinterpret_cast<Groups *>(lds + 2 * kStage + kWaves * 32 * kPitch / 4);
    find_groups<BM>(p, s);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;
    float *const slab = reinterpret_cast<float *>(lds + 2 * kStage) + wave * 32 * kPitch;
    const int tiles_n = (p.N + BN - 1) / BN, tiles_k = (p.K + BM - 1) / BM;
    const int total = tiles_n * (WGRAD ? p.E * tiles_k : uniform(s.units[p.fill ? p.E + 1 : p.E]));
    // Blocks go round the eight XCDs; each XCD takes a run of tiles.
    const int per = (total + 7) / 8, xcd = blockIdx.x & 7;
    const int end = min(total, (xcd + 1) * per);
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) void *)lds));
    for (int id = xcd * per + (blockIdx.x >> 3); id < end; id += gridDim.x >> 3) {
        int e, m0, n0, rows, steps;
        Direct<WGRAD, BM, kWaves> da;
        Direct<WLINE, BN, kWaves> db;
        if (WGRAD) {
            const int rest = uniform(id / tiles_n);
            n0 = uniform(id % tiles_n) * BN;
            e = uniform(rest / tiles_k);
            m0 = uniform(rest % tiles_k) * BM;
            rows = min(BM, p.K - m0);
            const int first = uniform(s.start[e]), count = uniform(s.start[e + 1]) - first;
            steps = (count + 63) / 64;
            if (p.accumulate && count == 0) continue;
            da.init(p.x + static_cast<int64_t>(first) * p.K + m0, p.K, 0, count, m0, wave, lane);
            db.init(p.w + static_cast<int64_t>(first) * p.N + n0, p.N, 0, count, n0, wave, lane);
        } else {
            e = uniform(expert_of(s, p.E, uniform(id / tiles_n)));
            // within an expert, bands of eight units by all columns
            const int u0 = uniform(s.units[e]), units = uniform(s.units[e + 1]) - u0;
            const int at = id - u0 * tiles_n;
            const int band = at / (8 * tiles_n), in_band = at - band * 8 * tiles_n;
            const int depth = min(8, units - band * 8);
            n0 = uniform(in_band / depth) * BN;
            m0 = uniform(s.start[e]) + uniform(band * 8 + in_band % depth) * BM;
            rows = min(BM, uniform(s.start[e + 1]) - m0);
            steps = e < p.E ? (p.K + 63) / 64 : 0;
            const uint16_t *w = p.w + static_cast<int64_t>(e) * p.K * p.N;
            da.init(p.x + static_cast<int64_t>(m0) * p.K, p.K, rows, p.K, 0, wave, lane);
            if (WLINE)
                db.init(w + n0, p.N, 0, p.K, n0, wave, lane);
            else
                db.init(w + static_cast<int64_t>(n0) * p.K, p.K, min(BN, p.N - n0), p.K, 0, wave,
                        lane);
        }
        f16_t acc[FM][FN] = {};
        u4_t a[2][FM], b[2][FN];
        constexpr int kA = decltype(da)::kLoads, kLoads = kA + decltype(db)::kLoads;
        auto load = [&](int i, int stage) {
            const uint32_t to = lds0 + stage * kStage * 16;
            if (i < kA) da.load(i, to, wave);
            else db.load(i - kA, to + BM * 128, wave);
        };
        auto fetch = [&](int step) {
            da.at(step);
            db.at(step);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load(i, step & 1);
        };
        auto get = [&](int to, int stage, int part, int i) {
            const u4_t *tile = lds + stage * kStage;
            if (i < FM) a[to][i] = fragment<WGRAD, BM>(tile, wm + 32 * i, part, lane);
            else b[to][i - FM] = fragment<WLINE, BN>(tile + BM * 8, wn + 32 * (i - FM), part, lane);
        };
        // One part: its MFMAs, and between them the next part's fragments and loads.
        auto run_part = [&](int from, int stage, int part, auto loads, int to_stage) {
            constexpr int kGets = FM + FN, kMfmas = FM * FN;
            constexpr int kGet = (2 * kGets + kMfmas - 1) / kMfmas;
            constexpr int kLoad = (kLoads + kMfmas - 1) / kMfmas;
#pragma unroll
            for (int m = 0; m < kMfmas; ++m) {
#pragma unroll
                for (int i = m * kGet; i < (m + 1) * kGet && i < kGets; ++i)
                    get(from ^ 1, stage, part, i);
                if (loads)
#pragma unroll
                    for (int i = m * kLoad; i < (m + 1) * kLoad && i < kLoads; ++i)
                        load(i, to_stage);
                acc[m / FN][m % FN] = mfma32<F16>(b[from][m % FN], a[from][m / FN],
                                                  acc[m / FN][m % FN]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        const std::integral_constant<bool, true> yes{};
        const std::integral_constant<bool, false> no{};
        if (steps > 0) {
            fetch(0);
            fetch(1);
            direct_wait<kLoads>();
#pragma unroll
            for (int i = 0; i < FM + FN; ++i) get(0, 0, 0, i);
            // (behind the last step loads bring zeros and fragments go unused: cheaper
            // than a second copy of the loop)
            for (int step = 0; step < steps; ++step) {
                const int cur = step & 1;
                run_part(0, cur, 1, no, 0);
                run_part(1, cur, 2, no, 0);
                run_part(0, cur, 3, no, 0);
                direct_wait<0>();
                da.at(step + 2);
                db.at(step + 2);
                run_part(1, cur ^ 1, 0, yes, cur);
            }
        }
        // A lane holds four columns of a row at a time: 32 x 32 results go through the
        // wave's own LDS, so that rows are written in runs.
        const int64_t row0 = WGRAD ? static_cast<int64_t>(e) * p.K + m0 : m0;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                put_block<F16>(p, slab, acc[i][j], row0 + wm + 32 * i, rows - wm - 32 * i,
                               n0 + wn + 32 * j, lane);
        // the next tile's loads go where this one's last fragments came from
        direct_wait<0>();
    }
}

template <bool F16, bool WGRAD, bool WLINE>
hipError_t launch_general(const GroupedParams &p, hipStream_t stream) {
    const int64_t tn = (p.N + 127) / 128, tk = (p.K + 127) / 128;
    const int64_t most = WGRAD ? p.E * tk * tn : (p.M / 128 + p.E + 1) * tn;
    const uint32_t grid = static_cast<uint32_t>(most < 1024 ? most : 1024);
    hipLaunchKernelGGL((general_kernel<F16, WGRAD, WLINE>), dim3(grid), dim3(256), 0, stream, p);
    return hipGetLastError();
}

template <bool F16, bool WGRAD, bool WLINE, int BM, int BN, int WM, int WN>
hipError_t launch_direct(const GroupedParams &p, hipStream_t stream) {
    constexpr int lds = direct_lds<BM, BN, WM, WN>();
    static_assert(lds <= kMaxLds, "as allow_lds allows");
    constexpr auto kernel = &direct_kernel<F16, WGRAD, WLINE, BM, BN, WM, WN>;
    if (hipError_t e = allow_lds<kernel>(lds); e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(256), dim3((BM / WM) * (BN / WN) * 64), lds, stream, p);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_grouped_t(const GroupedParams &p, hipStream_t stream) {
    // rows of whole pieces, of every operand that is loaded
    if (p.K % 8 == 0 && (p.N % 8 == 0 || (!p.wgrad && p.transpose))) {
        if (p.wgrad) return launch_direct<F16, true, true, 256, 256, 128, 128>(p, stream);
        return p.transpose ? launch_direct<F16, false, false, 256, 256, 128, 128>(p, stream)
                           : launch_direct<F16, false, true, 256, 256, 128, 128>(p, stream);
    }
    if (p.wgrad) return launch_general<F16, true, true>(p, stream);
    return p.transpose ? launch_general<F16, false, false>(p, stream)
                       : launch_general<F16, false, true>(p, stream);
}

}  // namespace

hipError_t launch_grouped(const GroupedParams &p, hipStream_t stream) {
    return p.f16 ? launch_grouped_t<true>(p, stream) : launch_grouped_t<false>(p, stream);
}

}  // namespace gfr
