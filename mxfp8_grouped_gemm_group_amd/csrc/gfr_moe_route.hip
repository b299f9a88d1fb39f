// Router: each token's experts from its logits, and the chosen (token, expert)
// pairs in expert order with the tokens' rows MX-quantised (the inputs of the
// grouped products).  include/gfr.h states the operator.
//
// A wave takes a token.  Lane l holds experts l V .. l V + V - 1 in registers
// (V = 1, 2, 4, 8 or 16 with E), and each of the k rounds takes the maximum
// over the wave (six DPP steps, no LDS), finds its lowest holder with a ballot
// and strikes it out there.  Choosing by the logits compares FP32; with a bias
// or expert groups the values compared are FP64, since two scores that differ
// by less than an FP32 rounding would otherwise change places.
//
// With x, the pairs are sorted by expert, stably, by counting:
//   few tokens    one launch, one block per token: every block chooses for all
//                 tokens (cheaper than a launch that hands the choice over) and
//                 counts the pairs ahead of its own token's;
//   more tokens   route_kernel (choice, counts per chunk of 16 tokens and
//                 expert), scan_kernel (a block per expert over the chunks),
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

constexpr int kChunk = 16;          // tokens per block of the long path
constexpr int kFewTokens = 64;      // one-launch path up to here
constexpr int kMoveThreads = 256;

// Waves of a route_kernel block: one per token of a chunk, or as many as V's
// registers leave.
constexpr int route_waves(int V) { return V == 16 ? 8 : kChunk; }

constexpr float kNegInf = -INFINITY;

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_max(float x) {
    const float y = __uint_as_float(
        dpp<CTRL, ROWS, 0xf, false>(__float_as_uint(kNegInf), __float_as_uint(x)));
    return fmaxf(x, y);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double x, double old) {
    const uint64_t b = __double_as_longlong(x), o = __double_as_longlong(old);
    const uint32_t lo = dpp<CTRL, ROWS, 0xf, false>(static_cast<uint32_t>(o),
                                                    static_cast<uint32_t>(b));
    const uint32_t hi = dpp<CTRL, ROWS, 0xf, false>(static_cast<uint32_t>(o >> 32),
                                                    static_cast<uint32_t>(b >> 32));
    return __longlong_as_double(static_cast<uint64_t>(hi) << 32 | lo);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_max(double x) {
    return fmax(x, dpp_f64<CTRL, ROWS>(x, static_cast<double>(kNegInf)));
}

__device__ __forceinline__ float lane_value(float x, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane));
}
__device__ __forceinline__ double lane_value(double x, int lane) {
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
    return __longlong_as_double(static_cast<uint64_t>(hi) << 32 | lo);
}

// Maximum over the wave (row shifts, then row broadcasts; lane 63 has it).
template <class K>
__device__ __forceinline__ K wave_max(K x) {
    x = dpp_max<0x111, 0xf>(x);
    x = dpp_max<0x112, 0xf>(x);
    x = dpp_max<0x114, 0xf>(x);
    x = dpp_max<0x118, 0xf>(x);
    x = dpp_max<0x142, 0xa>(x);
    x = dpp_max<0x143, 0xc>(x);
    return lane_value(x, 63);
}
__device__ __forceinline__ double wave_sum(double x) {
    x += dpp_f64<0x111, 0xf>(x, 0.0);
    x += dpp_f64<0x112, 0xf>(x, 0.0);
    x += dpp_f64<0x114, 0xf>(x, 0.0);
    x += dpp_f64<0x118, 0xf>(x, 0.0);
    x += dpp_f64<0x142, 0xa>(x, 0.0);
    x += dpp_f64<0x143, 0xc>(x, 0.0);
    return lane_value(x, 63);
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

// The choice of one token: lane j < k returns its j-th expert (-1: none) and
// weight.  WIDE: FP64 keys (bias or groups); s as keep_groups.
template <int V, bool WIDE>
__device__ __forceinline__ void choose(const RouteParams &p, int t, int lane, double *s, int &id,
                                       float &weight) {
    typedef typename std::conditional<WIDE, double, float>::type K;
    const int64_t row = static_cast<int64_t>(t) * p.E;
    float z[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        float l = kNegInf;
        if (e < p.E)
            l = p.logits_bf16 ? bf16_f32(static_cast<const uint16_t *>(p.logits)[row + e])
                              : static_cast<const float *>(p.logits)[row + e];
        z[v] = l > kNegInf ? l : kNegInf;   // NaN: not live
    }
    float top = 0.0f;
    if (!p.sigmoid) {
        top = z[0];
#pragma unroll
        for (int v = 1; v < V; ++v) top = fmaxf(top, z[v]);
        top = wave_max(top);
        if (top == kNegInf) top = 0.0f;
    }
    K key[V], score[V];
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (WIDE) {
            const double d = z[v];
            score[v] = p.sigmoid ? 1.0 / (1.0 + exp(-d)) : exp(d - top);
        } else {
            score[v] = p.sigmoid ? 1.0f / (1.0f + expf(-z[v])) : expf(z[v] - top);
        }
        sum += score[v];
    }
    // softmax's denominator; without FP64 keys and with renormalize it cancels
    K scale = 1;
    if (!p.sigmoid && (WIDE || !p.renormalize)) {
        sum = wave_sum(sum);
        if (WIDE) {
#pragma unroll
            for (int v = 0; v < V; ++v) score[v] = static_cast<K>(score[v] / sum);
        } else {
            scale = static_cast<K>(1.0 / sum);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (WIDE) {
            const int e = lane * V + v;
            const K d = score[v] + (p.bias && e < p.E ? static_cast<K>(p.bias[e]) : K(0));
            key[v] = z[v] > kNegInf && d > kNegInf ? d : K(kNegInf);
        } else {
            key[v] = z[v];
        }
    }
    if (WIDE && p.n_group > 1) {
        double d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = key[v];
        keep_groups(p, d, s, lane);
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = static_cast<K>(d[v]);
    }
    id = -1;
    K mine = 0, total = 0;
    for (int j = 0; j < p.k; ++j) {
        K best = key[0], worth = score[0];
        int slot = 0;
#pragma unroll
        for (int v = 1; v < V; ++v)
            if (key[v] > best) best = key[v], worth = score[v], slot = v;
        const K most = wave_max(best);
        if (!(most > K(kNegInf))) break;
        const int holder = __ffsll(static_cast<unsigned long long>(__ballot(best == most))) - 1;
        const int at = __builtin_amdgcn_readlane(slot, holder);
        const K value = lane_value(worth, holder);
        total += value;
        if (lane == j) id = holder * V + at, mine = value;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane == holder && v == at) key[v] = K(kNegInf);
    }
    if (p.renormalize)   // a zero sum leaves zeros, a NaN goes through
        mine = total == K(0) ? K(0) : mine / total;
    else
        mine *= scale;
    weight = id < 0 ? 0.0f : static_cast<float>(mine * static_cast<K>(p.scaling));
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
    __shared__ int own_id[GFR_MAX_TOPK];
    __shared__ float own_weight[GFR_MAX_TOPK];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int me = blockIdx.x, n = p.T * p.k;
    for (int t = wave; t < p.T; t += 16) {
        int id;
        float weight;
        choose<V, WIDE>(p, t, lane, WIDE ? keys + wave * p.E : nullptr, id, weight);
        if (lane < p.k) {
            bucket[t * p.k + lane] = id < 0 ? p.E : id;
            if (t == me) {
                own_id[lane] = id;
                own_weight[lane] = weight;
                p.ids[t * p.k + lane] = id;
                p.weights[t * p.k + lane] = weight;
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
__global__ __launch_bounds__(64 * route_waves(V)) void route_kernel(RouteParams p, int per_block) {
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
        float weight;
        choose<V, WIDE>(p, t, lane, WIDE ? keys + wave * p.E : nullptr, id, weight);
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
__global__ __launch_bounds__(kMoveThreads) void move_kernel(RouteParams p, int chunks) {
    __shared__ int start[GFR_MAX_EXPERTS + 1];
    __shared__ int bucket[kChunk * GFR_MAX_TOPK];
    __shared__ int pos[kChunk * GFR_MAX_TOPK];
    __shared__ uint32_t totals[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t0 = blockIdx.x * kChunk, nt = min(kChunk, p.T - t0), n = nt * p.k;
    const int64_t q0 = static_cast<int64_t>(t0) * p.k;
    for (int i = threadIdx.x; i < n; i += kMoveThreads) {
        const int id = p.ids[q0 + i];
        bucket[i] = id < 0 ? p.E : id;
    }
    uint32_t carry = 0;
    for (int base = 0; base <= p.E; base += kMoveThreads) {
        const int e = base + threadIdx.x;
        const uint32_t v = e < p.E ? static_cast<uint32_t>(p.group_list[e]) : 0;
        const uint32_t incl = wave_prefix(v);
        if (lane == 63) totals[wave] = incl;
        __syncthreads();
        uint32_t before = carry;
        for (int w = 0; w < 4; ++w) {
            if (w < wave) before += totals[w];
            carry += totals[w];
        }
        if (e <= p.E)
            start[e] = before + incl - v + p.counts[static_cast<int64_t>(e) * chunks + blockIdx.x];
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
    const int per_block = p.x || p.T > 4096 ? kChunk : 1;
    const int waves = per_block == 1 ? 1 : route_waves(V);
    const int blocks = (p.T + per_block - 1) / per_block;
    constexpr auto kernel = &route_kernel<V, WIDE>;
    if (hipError_t e = allow_lds<kernel>(static_cast<int>(waves * keys)); e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(64 * waves), waves * keys, stream, p, per_block);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || !p.x) return e;
    hipLaunchKernelGGL(scan_kernel, dim3(p.E + 1), dim3(256), 0, stream, p, blocks);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    // few chunks: their rows' columns over several blocks each
    const int pieces = (p.H / 16 + 63) / 64;
    int split = 1;
    while (blocks * split < 1024 && split * 2 <= pieces) split *= 2;
    hipLaunchKernelGGL(move_kernel, dim3(blocks, split), dim3(kMoveThreads), 0, stream, p, blocks);
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
    const size_t chunks = static_cast<size_t>(T + kChunk - 1) / kChunk;
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
