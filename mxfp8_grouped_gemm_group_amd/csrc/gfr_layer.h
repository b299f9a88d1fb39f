// Internal interface between the host API (gfr_layer_api.cpp) and the kernels
// of the dense product, the few-token experts, the router and the 16-bit grouped
// products and the adapters (gfr_linear.hip, gfr_moe_decode.hip, gfr_moe_route.hip,
// gfr_grouped.hip, gfr_lora.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace gfr {

// The kernel for a size (the tiled ones by their tile) and its K split.
struct LinearChoice {
    enum Kernel : int32_t { kRows, k256, k256x128, k128, k64 } kernel;
    int32_t split;             // 0: too large for a grid
};
LinearChoice linear_choice(int64_t M, int64_t N, int64_t K, int act);

struct LinearParams {
    const uint16_t *x;         // [M, K]
    const uint16_t *w;         // [N, K], or [2N, K] (swiglu)
    const void *bias;          // may be null
    const uint16_t *residual;  // may be null
    void *out;                 // [M, N]
    float *partial;            // split K: [split][M][columns, to a multiple of 8]
    int32_t bias_f32, out_f32, f16, act;
    int32_t wide;              // rows of out and residual are whole, aligned 16 bytes
    int32_t M, N, K;
    LinearChoice::Kernel kernel;
    int32_t split;             // 1: no partial sums
    int32_t keep_partial;      // 1: partial sums are the result; nothing joins them
};

hipError_t launch_linear(const LinearParams &p, hipStream_t stream);

// One of moe_decode's two products: the K chunks whose partial sums are kept
// apart, the column tiles each wave of a block takes, its waves, and whether
// these share one tile instead.
struct DecodePart {
    int32_t chunks, run, waves, shared;
};

struct DecodeParams {
    const uint16_t *x;         // [T, H] bf16
    const uint8_t *w13, *s13, *w2, *s2;
    const int32_t *ids;        // [T, k]
    const float *weights;      // [T, k]
    const uint16_t *shared;    // [T, N] bf16 or null
    void *out;                 // [T, N]
    int32_t *status;           // may be null
    float *gu;                 // [gate_up.chunks][T k][2I]: partial sums of x w13
    float *y;                  // [down.chunks][T k][N]: partial sums of h w2
    uint16_t *h;               // [3][T k][I]: silu(gate) * up as three bf16 terms, or null
    int64_t s13_e, s2_e;       // bytes between experts' scales (0: shared)
    float shared_w;
    int32_t out_f32;
    int32_t T, k, E, H, I, N;
    int32_t row_fragments;     // of 16 pairs, per group
    DecodePart gate_up, down;
};

// Workspace layout of moe_decode (256-byte aligned regions) and the products'
// shapes.
struct DecodeLayout {
    size_t gu, y, h, total;
    int32_t activate;          // h is made by a launch of its own
    int32_t row_fragments;
    DecodePart gate_up, down;
};
DecodeLayout decode_layout(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int64_t N,
                           int transpose_w13, int transpose_w2);
hipError_t launch_decode(const DecodeParams &p, int transpose_w13, int transpose_w2, int e5m2,
                         hipStream_t stream);

struct RouteParams {
    const void *logits;        // [T, E] f32 or bf16
    const float *bias;         // [E] or null
    int32_t *ids;              // [T, k]
    float *weights;            // [T, k]
    const uint16_t *x;         // [T, H] or null
    uint8_t *xin;              // [T k, H]
    uint8_t *xin_scale;        // [T k, 2 ceil(H / 64)]
    int64_t *group_list;       // [E]
    int32_t *row_index;        // [T k]
    float *logit;              // [T k]
    int32_t *counts;           // workspace: [E + 1][chunks]
    int32_t logits_bf16, x_f16, e5m2, sigmoid, renormalize;
    int32_t n_group, topk_group;
    float scaling;
    int32_t T, E, k, H;
};

// Workspace bytes of moe_route with x.
size_t route_workspace(int64_t T, int64_t E, int64_t k);
hipError_t launch_route(const RouteParams &p, hipStream_t stream);

// The kernel for a size of the 16-bit grouped products: whole rows of pieces straight to
// LDS, or the general one by its tile.
enum class GroupedKernel : int32_t { kDirect, k128, k64, k64Long };
GroupedKernel grouped_kernel(int wgrad, int transpose, int64_t M, int64_t E, int64_t K, int64_t N);

struct GroupedParams {
    const uint16_t *x;         // [M, K]
    const uint16_t *w;         // forward: [E, K, N] ([E, N, K] transposed); wgrad: [M, N]
    void *out;                 // forward: [M, N]; wgrad: [E, K, N]
    const int64_t *group_list; // [E]
    int32_t *status;           // may be null
    int32_t wgrad, transpose, cumsum;
    int32_t fill;              // forward: rows of no group are cleared
    int32_t accumulate;        // wgrad: out is added to
    int32_t f16, out_f32;
    int32_t wide;              // rows of out are whole, aligned 16 bytes
    int32_t turn;              // forward, [E, N, K]: column tiles begin at different steps of K
    GroupedKernel kernel;
    int32_t M, E, K, N;
};

hipError_t launch_grouped(const GroupedParams &p, hipStream_t stream);

struct LoraParams {
    const uint16_t *x;         // [M, K]
    const uint16_t *w;         // [N, K]
    const uint16_t *a;         // [L, r, K]
    const uint16_t *b;         // [L, N, r]
    const int32_t *ids;        // [M]
    const float *scaling;      // [L] or null
    const void *bias;          // [N] or null
    const uint16_t *residual;  // [M, N] or null
    void *out;                 // [M, N]
    int32_t *status;           // may be null
    float *inner;              // workspace, few rows or F16: [M][r], scaled
    float *dense;              // workspace, many rows: [M / 32][N / 32] of 32 x 32 sums as
                               // lanes have them; few rows: [M][N], or the K splits' sums
    uint16_t *terms;           // workspace, many rows of bf16: [M][3][r], scaled
    int32_t *codes;            // workspace, many rows: [M / 32], the adapter of 32 rows
    LinearChoice choice;
    int32_t tiles;             // many rows
    int32_t bias_f32, out_f32, f16;
    int32_t M, N, K, L, r;
};

// Workspace layout of lora_linear (256-byte aligned regions; inner or terms at 0).
struct LoraLayout {
    size_t codes, dense, total;
    int32_t tiles;             // many rows: dense tiles that take expansions in their sum
    LinearChoice choice;       // few rows: of the dense product
};
LoraLayout lora_layout(int64_t M, int64_t N, int64_t K, int64_t r);
hipError_t launch_lora(const LoraParams &p, hipStream_t stream);

}  // namespace gfr
