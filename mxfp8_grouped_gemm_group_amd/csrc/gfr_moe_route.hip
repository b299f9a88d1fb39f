// Router: each token's experts from its logits, and the chosen (token, expert)
// pairs in expert order with the tokens' rows MX-quantised (the inputs of the
// grouped products).  include/gfr.h states the operator.
//
// A wave takes a token.  Lane l holds experts l V .. l V + V - 1 in registers
// (V = 1, 2, 4, 8 or 16 with E), and each of the k rounds takes the maximum
// over the wave (six DPP steps per word, no LDS), finds its lowest holder with a
// ballot and strikes it out there.  Choosing by the logits compares FP32; with a bias
// or expert groups the values compared are FP64, since two scores that differ
// by less than an FP32 rounding would otherwise change places.
// Weights are computed in FP64 and rounded once.
//
// With x, the pairs are sorted by expert, stably, by counting:
//   few tokens    one launch, one block per token: every block chooses for all
//                 tokens (cheaper than a launch that hands the choice over) and
//                 counts the pairs ahead of its own token's;
//   more tokens   route_kernel (choice, counts per chunk of tokens and
//                 expert), scan_kernel (a block per expert over the chunks; few
//                 chunks are summed by each block of the next instead),
//                 move_kernel (a block per chunk: ranks within it, rows).
// Moving rows bounds the long calls: each row is read once, quantised in
// registers and written to its k places in 16-byte stores.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gfr.h"
#include "gfr_device.h"
#include "gfr_layer.h"

namespace gfr {
namespace {

constexpr int kRouteWaves = 8;      // of a block of the long path, which takes
constexpr int kMaxChunk = 16;       // at most so many tokens (a chunk)
// One-launch path up to here: its blocks, one a token, each choose for all tokens,
// a wave a token.
constexpr int kFewTokens = 16;
constexpr int kFewChunks = 64;      // no scan launch up to here
constexpr int kMoveThreads = 256;

constexpr float kNegInf = -INFINITY;

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double x) {
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = dpp<CTRL, ROWS, 0xf, true>(0, static_cast<uint32_t>(b));
    const uint32_t hi = dpp<CTRL, ROWS, 0xf, true>(0, static_cast<uint32_t>(b >> 32));
    return __longlong_as_double(static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ double lane_value(double x, int lane) {
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
    return __longlong_as_double(static_cast<uint64_t>(hi) << 32 | lo);
}

// Over the wave: row shifts, then row broadcasts; lane 63 has the result.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = max(x, dpp<0x111, 0xf, 0xf, true>(0, x));
    x = max(x, dpp<0x112, 0xf, 0xf, true>(0, x));
    x = max(x, dpp<0x114, 0xf, 0xf, true>(0, x));
    x = max(x, dpp<0x118, 0xf, 0xf, true>(0, x));
    x = max(x, dpp<0x142, 0xa, 0xf, true>(0, x));
    x = max(x, dpp<0x143, 0xc, 0xf, true>(0, x));
    return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ double wave_sum(double x) {
    x += dpp_f64<0x111, 0xf>(x);
    x += dpp_f64<0x112, 0xf>(x);
    x += dpp_f64<0x114, 0xf>(x);
    x += dpp_f64<0x118, 0xf>(x);
    x += dpp_f64<0x142, 0xa>(x);
    x += dpp_f64<0x143, 0xc>(x);
    return lane_value(x, 63);
}

// Unsigned integers in the order of floats above -inf (0 stands for -inf and
// for what is struck out).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);     // -0 equals 0
    return x > kNegInf ? (b >> 31 ? ~b : b | 0x80000000u) : 0;
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
    return k == 0 ? kNegInf : __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t b = __double_as_longlong(x == 0.0 ? 0.0 : x);
    return x > static_cast<double>(kNegInf) ? (b >> 63 ? ~b : b | uint64_t{1} << 63) : 0;
}

// What is subtracted from logits ahead of exp: their largest, or 0 where none is live.
__device__ __forceinline__ double exponent_base(float top) {
    return top == kNegInf ? 0.0 : static_cast<double>(top);
}

// Strikes out the experts of all but the topk_group best groups.  Lane q adds
// up its group's two largest keys, and group q stays if fewer than topk_group
// groups are better (larger, or equal and of lower index).  The keys go through
// LDS (`s`, E doubles of this wave's own): all of them, or, where no lane holds
// experts of two groups, each lane's two largest (256 experts in 8 groups: 8
// reads instead of 32).
template <int V>
__device__ __forceinline__ void keep_groups(const RouteParams &p, double (&key)[V], double *s,
                                            int lane) {
    const int width = p.E / p.n_group;
    double first = kNegInf, second = kNegInf;
    __builtin_amdgcn_wave_barrier();
    if (V > 1 && width % V == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            second = fmax(second, fmin(first, key[v]));
            first = fmax(first, key[v]);
        }
        if (lane * V < p.E) s[2 * lane] = first, s[2 * lane + 1] = second;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int lanes = width / V;
        first = second = kNegInf;
        if (lane < p.n_group) {
#pragma unroll 4
            for (int i = 0; i < lanes; ++i) {
                const double a = s[2 * (lane * lanes + i)], b = s[2 * (lane * lanes + i) + 1];
                second = fmax(fmax(second, b), fmin(first, a));
                first = fmax(first, a);
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane * V + v < p.E) s[lane * V + v] = key[v];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (lane < p.n_group) {
#pragma unroll 4
            for (int i = 0; i < width; ++i) {
                const double d = s[lane * width + i];
                second = fmax(second, fmin(first, d));
                first = fmax(first, d);
            }
        }
    }
    const double value = first + (second > kNegInf ? second : 0.0);
    int better = 0;
    for (int q = 0; q < p.n_group; ++q) {
        const double other = lane_value(value, q);
        better += other > value || (other == value && q < lane);
    }
    const uint64_t kept = __ballot(lane < p.n_group && better < p.topk_group);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        if (e < p.E && !(kept >> (e / width) & 1)) key[v] = kNegInf;
    }
}

// A token's logits: lane l's V experts, -inf for what is not live.  (Loads
// without a branch between them, at clamped places: under conditions the
// compiler waits for each before the next.)
template <int V>
__device__ __forceinline__ void load_logits(const RouteParams &p, int t, int lane, float (&z)[V]) {
    const int64_t row = static_cast<int64_t>(t) * p.E;
    if (p.logits_bf16) {
        const uint16_t *at = static_cast<const uint16_t *>(p.logits) + row;
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = bf16_f32(at[min(lane * V + v, p.E - 1)]);
    } else {
        const float *at = static_cast<const float *>(p.logits) + row;
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = at[min(lane * V + v, p.E - 1)];
    }
#pragma unroll
    for (int v = 0; v < V; ++v)                        // NaN: not live
        z[v] = lane * V + v < p.E && z[v] > kNegInf ? z[v] : kNegInf;
}

// The choice of one token: lane j < k returns its j-th expert (-1: none) and
// weight.  WIDE: FP64 keys (bias or groups); s as keep_groups.  Keys are compared
// as ordered integers, an FP64 key's halves one after the other: a wave maximum
// of words is six instructions, one of doubles some thirty.  Scores, their sums and
// the weights are FP64 in both forms; without FP64 keys only the chosen ones are
// computed, a lane each.
template <int V, bool WIDE>
__device__ __forceinline__ void choose(const RouteParams &p, const float (&z)[V], int lane,
                                       double *s, int &id, float &weight) {
    uint32_t hi[V], lo[V];
    double score[V] = {};
    if (WIDE) {
        if (p.sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v) score[v] = 1.0 / (1.0 + exp(-static_cast<double>(z[v])));
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) m = max(m, ordered(z[v]));
            const double top = exponent_base(from_ordered(wave_max(m)));
            double sum = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += score[v] = exp(z[v] - top);
            sum = wave_sum(sum);
#pragma unroll
            for (int v = 0; v < V; ++v) score[v] /= sum;
        }
        float bias[V] = {};
        if (p.bias)
#pragma unroll
            for (int v = 0; v < V; ++v) bias[v] = p.bias[min(lane * V + v, p.E - 1)];
        double key[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double d = score[v] + bias[v];
            key[v] = z[v] > kNegInf && d > kNegInf ? d : kNegInf;
        }
        if (p.n_group > 1) keep_groups(p, key, s, lane);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint64_t o = ordered(key[v]);
            hi[v] = static_cast<uint32_t>(o >> 32);
            lo[v] = static_cast<uint32_t>(o);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) hi[v] = ordered(z[v]), lo[v] = 0;
    }
    id = -1;
    float logit = kNegInf, first = kNegInf;    // without WIDE: lane j's choice's, the largest
    double mine = 0, total = 0;
    for (int j = 0; j < p.k; ++j) {
        uint32_t h = hi[0], l = lo[0];
        double worth = score[0];
        int slot = 0;
#pragma unroll
        for (int v = 1; v < V; ++v)
            if (hi[v] > h || (WIDE && hi[v] == h && lo[v] > l))
                h = hi[v], l = lo[v], worth = score[v], slot = v;
        const uint32_t most = wave_max(h);
        if (most == 0) break;
        uint64_t holders = __ballot(h == most);
        if (WIDE && (holders & (holders - 1))) {     // several: by the low halves
            const uint32_t low = wave_max(h == most ? l : 0);
            holders = __ballot(h == most && l == low);
        }
        const int holder = __ffsll(static_cast<unsigned long long>(holders)) - 1;
        const int at = __builtin_amdgcn_readlane(slot, holder);
        if (lane == j) id = holder * V + at;
        if (WIDE) {
            const double value = lane_value(worth, holder);
            total += value;
            if (lane == j) mine = value;
        } else {
            if (j == 0) first = from_ordered(most);
            if (lane == j) logit = from_ordered(most);
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane == holder && v == at) hi[v] = lo[v] = 0;
    }
    if (!WIDE) {
        // softmax's denominator cancels under renormalize; so does exp(-first) of
        // sigmoids, which keeps far logits' scores from falling to zero together
        const double top = exponent_base(first), d = logit;
        if (!p.sigmoid)
            mine = exp(d - top);
        else if (p.renormalize && top < 0.0)
            mine = exp(d - top) / (1.0 + exp(d));
        else
            mine = 1.0 / (1.0 + exp(-d));
        if (id < 0) mine = 0.0;
        if (p.renormalize) {
            total = wave_sum(mine);
        } else if (!p.sigmoid) {
            double sum = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += exp(z[v] - top);
            mine /= wave_sum(sum);
        }
    }
    if (p.renormalize)   // a zero sum leaves zeros, a NaN goes through
        mine = total == 0.0 ? 0.0 : mine / total;
    weight = id < 0 ? 0.0f : static_cast<float>(mine * static_cast<double>(p.scaling));
}

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------

// Four floats times 2^-X as FP8 codes (to nearest, ties to even, saturating;
// NaN stays NaN), packed.
template <bool E5M2>
__device__ __forceinline__ uint32_t codes4(const float *v, float mul) {
    constexpr float kMax = E5M2 ? 57344.0f : 448.0f;
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[i] * mul;
        y[i] = a != a ? a : __builtin_amdgcn_fmed3f(a, -kMax, kMax);
    }
    int q = 0;
    if (E5M2) {
        q = __builtin_amdgcn_cvt_pk_bf8_f32(y[0], y[1], q, false);
        q = __builtin_amdgcn_cvt_pk_bf8_f32(y[2], y[3], q, true);
    } else {
        q = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], q, false);
        q = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], q, true);
    }
    return static_cast<uint32_t>(q);
}

// Token t's row quantised and written to rows pos[0 .. k) (row >= 0; ~row for
// a pair without an expert, which gets zeros).  Lane pairs hold a block of 32;
// `first` and `step` split the row's 16-element pieces over lanes, pairs
// kept together.
template <bool E5M2>
__device__ __forceinline__ void move_row(const RouteParams &p, int t, const int *pos, int first,
                                         int step) {
    constexpr int kEmax = E5M2 ? 15 : 8;
    const int pieces = p.H / 16, blocks = p.H / 32, per_row = 2 * ((p.H + 63) / 64);
    const uint16_t *src = p.x + static_cast<int64_t>(t) * p.H;
    for (int c = first; c < pieces; c += step) {
        const u4_t a = load<u4_t>(src + c * 16), b = load<u4_t>(src + c * 16 + 8);
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = i < 4 ? a[i] : b[i - 4];
            if (p.x_f16) {
                const h2_t h = __builtin_bit_cast(h2_t, w);
                v[2 * i] = static_cast<float>(h[0]);
                v[2 * i + 1] = static_cast<float>(h[1]);
            } else {
                v[2 * i] = __uint_as_float(w << 16);
                v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
            }
        }
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));   // drops NaN
        amax = fmaxf(amax, __uint_as_float(dpp<0xB1, 0xf, 0xf, true>(0, __float_as_uint(amax))));
        const int be = static_cast<int>(__float_as_uint(amax) >> 23);
        const int X = be == 0 ? -127 : max(be - 127 - kEmax, -127);
        const float mul = __uint_as_float(static_cast<uint32_t>(127 - X) << 23);
        u4_t q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = codes4<E5M2>(v + 4 * i, mul);
        const int blk = c >> 1;
        for (int j = 0; j < p.k; ++j) {
            const int at = pos[j];
            const bool live = at >= 0;
            const int64_t r = live ? at : ~at;
            *reinterpret_cast<u4_t *>(p.xin + r * p.H + c * 16) = live ? q : u4_t{0, 0, 0, 0};
            if (!(c & 1)) {
                uint8_t *sc = p.xin_scale + r * per_row + blk;
                sc[0] = live ? static_cast<uint8_t>(X + 127) : 0;
                if (blk == blocks - 1 && (blocks & 1)) sc[1] = 0;
            }
        }
    }
}

__device__ __forceinline__ void move_row_any(const RouteParams &p, int t, const int *pos,
                                             int first, int step) {
    if (p.e5m2)
        move_row<true>(p, t, pos, first, step);
    else
        move_row<false>(p, t, pos, first, step);
}

// ---------------------------------------------------------------------------
// Few tokens with x: one block of 16 waves per token.
// ---------------------------------------------------------------------------
template <int V, bool WIDE>
__global__ __launch_bounds__(1024) void route_few_kernel(RouteParams p) {
    extern __shared__ double keys[];            // WIDE with groups: 16 x E
    __shared__ int bucket[kFewTokens * GFR_MAX_TOPK];
    __shared__ int hist[GFR_MAX_EXPERTS];
    __shared__ int pos[GFR_MAX_TOPK];
    __shared__ float own_weight[GFR_MAX_TOPK];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int me = blockIdx.x, n = p.T * p.k;
    static_assert(kFewTokens <= 16, "a wave per token");
    if (wave < p.T) {
        int id;
        float weight, z[V];
        load_logits(p, wave, lane, z);
        choose<V, WIDE>(p, z, lane, WIDE ? keys + wave * p.E : nullptr, id, weight);
        if (lane < p.k) {
            bucket[wave * p.k + lane] = id < 0 ? p.E : id;
            if (wave == me) {
                own_weight[lane] = weight;
                p.ids[wave * p.k + lane] = id;
                p.weights[wave * p.k + lane] = weight;
            }
        }
    }
    if (me == 0)
        for (int e = threadIdx.x; e < p.E; e += 1024) hist[e] = 0;
    __syncthreads();
    // the place of each of this token's pairs: how many pairs go ahead of it
    for (int j = wave; j < p.k; j += 16) {
        const int q = me * p.k + j, b = bucket[q];
        int ahead = 0;
        for (int i = lane; i < n; i += 64) {
            const int o = bucket[i];
            ahead += o < b || (o == b && i < q);
        }
        ahead = static_cast<int>(wave_prefix(ahead));
        if (lane == 63) {
            pos[j] = b < p.E ? ahead : ~ahead;
            p.row_index[ahead] = me;
            p.logit[ahead] = own_weight[j];
        }
    }
    if (me == 0)
        for (int i = threadIdx.x; i < n; i += 1024)
            if (bucket[i] < p.E) atomicAdd(&hist[bucket[i]], 1);
    __syncthreads();
    if (me == 0)
        for (int e = threadIdx.x; e < p.E; e += 1024) p.group_list[e] = hist[e];
    move_row_any(p, me, pos, threadIdx.x, 1024);
}

// ---------------------------------------------------------------------------
// The choice alone, and the long path.
// ---------------------------------------------------------------------------

// A block's waves take `per_block` tokens; with counts, the pairs of the block
// per expert (bucket E: pairs without one) go to counts[bucket][block].
template <int V, bool WIDE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteParams p, int per_block) {
    extern __shared__ double keys[];            // WIDE with groups: waves x E
    __shared__ int hist[GFR_MAX_EXPERTS + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    if (p.counts) {
        for (int e = threadIdx.x; e <= p.E; e += blockDim.x) hist[e] = 0;
        __syncthreads();
    }
    const int t0 = blockIdx.x * per_block, t1 = min(t0 + per_block, p.T);
    for (int t = t0 + wave; t < t1; t += waves) {
        int id;
        float weight, z[V];
        load_logits(p, t, lane, z);
        choose<V, WIDE>(p, z, lane, WIDE ? keys + wave * p.E : nullptr, id, weight);
        if (lane < p.k) {
            const int64_t at = static_cast<int64_t>(t) * p.k + lane;
            p.ids[at] = id;
            p.weights[at] = weight;
            if (p.counts) atomicAdd(&hist[id < 0 ? p.E : id], 1);
        }
    }
    if (p.counts) {
        __syncthreads();
        for (int e = threadIdx.x; e <= p.E; e += blockDim.x)
            p.counts[static_cast<int64_t>(e) * gridDim.x + blockIdx.x] = hist[e];
    }
}

// counts[bucket][chunk] -> pairs of the bucket in earlier chunks, in place; a
// block per bucket.  group_list gets the totals.
__global__ __launch_bounds__(256) void scan_kernel(RouteParams p, int chunks) {
    __shared__ uint32_t totals[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x;
    int *c = p.counts + static_cast<int64_t>(e) * chunks;
    uint32_t carry = 0;
    for (int base = 0; base < chunks; base += 256) {
        const int i = base + threadIdx.x;
        const uint32_t v = i < chunks ? c[i] : 0;
        const uint32_t incl = wave_prefix(v);
        if (lane == 63) totals[wave] = incl;
        __syncthreads();
        uint32_t before = carry;
        for (int w = 0; w < 4; ++w) {
            if (w < wave) before += totals[w];
            carry += totals[w];
        }
        if (i < chunks) c[i] = before + incl - v;
        __syncthreads();
    }
    if (threadIdx.x == 0 && e < p.E) p.group_list[e] = carry;
}

// A block per chunk of tokens: where each bucket's pairs of this chunk begin
// (pairs of smaller experts, and of this one in earlier chunks), each pair's
// rank among the chunk's equals, then the rows.
// SCANNED: scan_kernel ran; otherwise (few chunks) every block sums the counts.
template <bool SCANNED>
__global__ __launch_bounds__(kMoveThreads) void move_kernel(RouteParams p, int chunk, int chunks) {
    __shared__ int start[GFR_MAX_EXPERTS + 1];
    __shared__ int bucket[kMaxChunk * GFR_MAX_TOPK];
    __shared__ int pos[kMaxChunk * GFR_MAX_TOPK];
    __shared__ uint32_t totals[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t0 = blockIdx.x * chunk, nt = min(chunk, p.T - t0), n = nt * p.k;
    const int64_t q0 = static_cast<int64_t>(t0) * p.k;
    for (int i = threadIdx.x; i < n; i += kMoveThreads) {
        const int id = p.ids[q0 + i];
        bucket[i] = id < 0 ? p.E : id;
    }
    uint32_t carry = 0;
    for (int base = 0; base <= p.E; base += kMoveThreads) {
        const int e = base + threadIdx.x;
        uint32_t v = 0, earlier = 0;
        if (e <= p.E) {
            const int *c = p.counts + static_cast<int64_t>(e) * chunks;
            if (SCANNED) {
                v = e < p.E ? static_cast<uint32_t>(p.group_list[e]) : 0;
                earlier = c[blockIdx.x];
            } else {
#pragma unroll 8
                for (int i = 0; i < chunks; ++i) {
                    const uint32_t n_i = c[i];
                    v += n_i;
                    earlier += i < static_cast<int>(blockIdx.x) ? n_i : 0;
                }
                if (e == p.E) v = 0;
                else if (blockIdx.x == 0 && blockIdx.y == 0) p.group_list[e] = v;
            }
        }
        const uint32_t incl = wave_prefix(v);
        if (lane == 63) totals[wave] = incl;
        __syncthreads();
        uint32_t before = carry;
        for (int w = 0; w < 4; ++w) {
            if (w < wave) before += totals[w];
            carry += totals[w];
        }
        if (e <= p.E) start[e] = before + incl - v + earlier;
        __syncthreads();
    }
    for (int i = threadIdx.x; i < n; i += kMoveThreads) {
        const int b = bucket[i];
        int rank = 0;
        for (int o = 0; o < i; ++o) rank += bucket[o] == b;
        const int at = start[b] + rank;
        pos[i] = b < p.E ? at : ~at;
        if (blockIdx.y == 0) {
            p.row_index[at] = t0 + i / p.k;
            p.logit[at] = p.weights[q0 + i];
        }
    }
    __syncthreads();
    for (int t = wave; t < nt; t += kMoveThreads / 64)
        move_row_any(p, t0 + t, pos + t * p.k, blockIdx.y * 64 + lane, gridDim.y * 64);
}

__global__ void clear_groups_kernel(int64_t *g, int n) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) g[i] = 0;
}

// Tokens per chunk: one per wave while that spreads them over the CUs, two (half
// the counts to scan) beyond.
int64_t chunk_of(int64_t T) { return T <= 4096 ? 8 : kMaxChunk; }

template <int V, bool WIDE>
hipError_t launch_route_t(const RouteParams &p, hipStream_t stream) {
    const size_t keys = WIDE && p.n_group > 1 ? sizeof(double) * p.E : 0;
    if (p.x && p.T <= kFewTokens) {
        // 16 waves' keys: at most 128 KB of LDS, at E = 1024
        constexpr auto kernel = &route_few_kernel<V, WIDE>;
        if (hipError_t e = allow_lds<kernel>(static_cast<int>(16 * keys)); e != hipSuccess)
            return e;
        hipLaunchKernelGGL(kernel, dim3(p.T), dim3(1024), 16 * keys, stream,
                           p);
        return hipGetLastError();
    }
    // the choice alone: single waves while they are few, so that each has a CU's
    // units to itself
    const int per_block = p.x || p.T > 4096 ? static_cast<int>(chunk_of(p.T)) : 1;
    const int waves = per_block < kRouteWaves ? per_block : kRouteWaves;
    const int blocks = (p.T + per_block - 1) / per_block;
    constexpr auto kernel = &route_kernel<V, WIDE>;
    if (hipError_t e = allow_lds<kernel>(static_cast<int>(waves * keys)); e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(64 * waves), waves * keys, stream, p, per_block);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || !p.x) return e;
    // few chunks: their rows' columns over several blocks each, and no scan
    const int pieces = (p.H / 16 + 63) / 64;
    int split = 1;
    while (blocks * split < 1024 && split * 2 <= pieces) split *= 2;
    if (blocks <= kFewChunks) {
        hipLaunchKernelGGL((move_kernel<false>), dim3(blocks, split), dim3(kMoveThreads), 0,
                           stream, p, per_block, blocks);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(scan_kernel, dim3(p.E + 1), dim3(256), 0, stream, p, blocks);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    hipLaunchKernelGGL((move_kernel<true>), dim3(blocks, split), dim3(kMoveThreads), 0, stream, p,
                       per_block, blocks);
    return hipGetLastError();
}

template <bool WIDE>
hipError_t launch_route_v(const RouteParams &p, hipStream_t stream) {
    if (p.E <= 64) return launch_route_t<1, WIDE>(p, stream);
    if (p.E <= 128) return launch_route_t<2, WIDE>(p, stream);
    if (p.E <= 256) return launch_route_t<4, WIDE>(p, stream);
    if (p.E <= 512) return launch_route_t<8, WIDE>(p, stream);
    return launch_route_t<16, WIDE>(p, stream);
}

}  // namespace

size_t route_workspace(int64_t T, int64_t E, int64_t k) {
    (void)k;
    if (T <= kFewTokens) return 0;
    const int64_t chunk = chunk_of(T);
    const size_t chunks = static_cast<size_t>((T + chunk - 1) / chunk);
    return (chunks * (E + 1) * sizeof(int) + 255) & ~static_cast<size_t>(255);
}

hipError_t launch_route(const RouteParams &p, hipStream_t stream) {
    if (p.T == 0) {
        if (!p.group_list) return hipSuccess;
        hipLaunchKernelGGL(clear_groups_kernel, dim3((p.E + 255) / 256), dim3(256), 0, stream,
                           p.group_list, p.E);
        return hipGetLastError();
    }
    return p.bias || p.n_group > 1 ? launch_route_v<true>(p, stream)
                                   : launch_route_v<false>(p, stream);
}

}  // namespace gfr
