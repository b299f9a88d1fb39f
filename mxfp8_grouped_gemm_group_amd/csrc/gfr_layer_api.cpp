// Host side of the descriptor calls for the rest of the MoE block: gfr_linear,
// gfr_moe_decode, gfr_moe_route, gfr_grouped_linear and its weights' gradient,
// gfr_lora_linear (include/gfr.h).  As in gfr_api.cpp every error
// is returned before anything is enqueued, no device memory is read and
// nothing is synchronised.
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "gfr.h"
#include "gfr_checks.h"
#include "gfr_layer.h"

namespace {

// Of moe_route: 16 a block of 512 threads, and a grid has at most 2^32 threads.
constexpr int64_t kMaxTokens = int64_t{1} << 26;

// Workspace of `need` bytes in opts.
int check_workspace(const gfr_options *opts, size_t need) {
    if (need == 0) return GFR_OK;
    if (!opts || !opts->workspace || opts->workspace_bytes < need)
        return GFR_ERR_WORKSPACE_TOO_SMALL;
    return aligned(opts->workspace, 256) ? GFR_OK : GFR_ERR_BAD_ALIGNMENT;
}

int resolve_linear(const gfr_tensor *x, const gfr_tensor *w, const gfr_tensor *bias,
                   const gfr_tensor *residual, int activation, const gfr_tensor *out,
                   gfr::LinearParams &p) {
    if (!x || !w || !out) return GFR_ERR_NULL_ARG;
    if (activation < GFR_ACT_NONE || activation > GFR_ACT_SWIGLU) return GFR_ERR_BAD_ARG;
    GFR_TRY(check_desc(x, {2}, {GFR_DT_BF16, GFR_DT_F16}));
    GFR_TRY(check_desc(w, {2}, {x->dtype}));
    GFR_TRY(check_desc(out, {2}, {x->dtype, GFR_DT_F32}));
    const int64_t M = x->shape[0], K = x->shape[1], rows = w->shape[0];
    if (activation == GFR_ACT_SWIGLU && rows % 2 != 0) return GFR_ERR_BAD_SHAPE;
    const int64_t N = activation == GFR_ACT_SWIGLU ? rows / 2 : rows;
    if (K < 1 || w->shape[1] != K || !shape_is(out, {M, N})) return GFR_ERR_BAD_SHAPE;
    if (present(bias)) {
        GFR_TRY(check_desc(bias, {1}, {x->dtype, GFR_DT_F32}));
        if (!shape_is(bias, {rows})) return GFR_ERR_BAD_SHAPE;
    }
    if (present(residual)) {
        GFR_TRY(check_desc(residual, {2}, {x->dtype}));
        if (!shape_is(residual, {M, N})) return GFR_ERR_BAD_SHAPE;
    }
    if (M > int64_t{1} << 30 || rows > int64_t{1} << 30 || K > int64_t{1} << 21)
        return GFR_ERR_UNSUPPORTED;
    if (!aligned(x->data, 16) || !aligned(w->data, 16) || !aligned(out->data, 8) ||
        (present(bias) && !aligned(bias->data, 8)) ||
        (present(residual) && !aligned(residual->data, 8)))
        return GFR_ERR_BAD_ALIGNMENT;
    p.x = static_cast<const uint16_t *>(x->data);
    p.w = static_cast<const uint16_t *>(w->data);
    p.bias = present(bias) ? bias->data : nullptr;
    p.residual = present(residual) ? static_cast<const uint16_t *>(residual->data) : nullptr;
    p.out = out->data;
    p.bias_f32 = present(bias) && bias->dtype == GFR_DT_F32;
    p.out_f32 = out->dtype == GFR_DT_F32;
    p.f16 = x->dtype == GFR_DT_F16;
    p.act = activation;
    p.wide = N % 8 == 0 && aligned(out->data, 16) &&
             (!present(residual) || aligned(residual->data, 16));
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    const gfr::LinearChoice choice = gfr::linear_choice(M, N, K, activation);
    p.kernel = choice.kernel;
    p.split = choice.split;
    return p.split > 0 ? GFR_OK : GFR_ERR_UNSUPPORTED;
}

size_t linear_bytes(const gfr::LinearParams &p) {
    if (p.split <= 1 || p.M == 0 || p.N == 0) return 0;
    const size_t pitch = (static_cast<size_t>(p.N) + 7) / 8 * 8;
    const size_t rows = p.act == GFR_ACT_SWIGLU ? 2 * pitch : pitch;
    return (sizeof(float) * p.split * p.M * rows + 255) & ~static_cast<size_t>(255);
}

int check_decode_sizes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int64_t N) {
    if (T < 0 || k < 1 || E < 1 || H < 1 || I < 1 || N < 0) return GFR_ERR_BAD_SHAPE;
    if (T > GFR_DECODE_MAX_TOKENS || k > GFR_MAX_TOPK || T * k > 1024 || E > GFR_MAX_EXPERTS ||
        H % 64 != 0 || I % 64 != 0 || N % 64 != 0)
        return GFR_ERR_UNSUPPORTED;
    // an expert's weights are addressed by 32-bit offsets
    if (H > kMaxRows || I > kMaxRows || N > kMaxRows || 2 * H * I > kMaxRows || I * N > kMaxRows)
        return GFR_ERR_UNSUPPORTED;
    return GFR_OK;
}

// [E, K, N] weights ([E, N, K] transposed) and their scales against K and the
// expert count; N comes back.
int resolve_weights(const gfr_tensor *w, const gfr_tensor *scale, int transpose, int64_t E,
                    int64_t K, int64_t &N, int64_t &scale_e) {
    if (transpose != 0 && transpose != 1) return GFR_ERR_BAD_ARG;
    GFR_TRY(check_desc(scale, {3, 4}, kScaleTypes));
    if (w->shape[0] != E || w->shape[transpose ? 2 : 1] != K) return GFR_ERR_BAD_SHAPE;
    N = w->shape[transpose ? 1 : 2];
    const int64_t kb = (K + 63) / 64, s0 = transpose ? N : kb, s1 = transpose ? kb : N;
    const bool per_expert = scale->ndim == 4;
    if (per_expert ? !shape_is(scale, {E, s0, s1, 2}) : !shape_is(scale, {s0, s1, 2}))
        return GFR_ERR_BAD_SHAPE;
    scale_e = per_expert ? kb * N * 2 : 0;
    return GFR_OK;
}

// The arguments that the grouped product and its weights' gradient share: x [M, K],
// group_list [E] and where E, M and the other width N fit.
int resolve_groups(const gfr_tensor *x, const gfr_tensor *group_list, int group_list_type,
                   int transpose_w, int flag, int64_t E, int64_t N, const gfr_tensor *out,
                   const gfr_options *opts, gfr::GroupedParams &p) {
    if ((group_list_type != GFR_GROUP_LIST_CUMSUM && group_list_type != GFR_GROUP_LIST_COUNT) ||
        (transpose_w != 0 && transpose_w != 1) || (flag != 0 && flag != 1))
        return GFR_ERR_BAD_ARG;
    GFR_TRY(check_desc(group_list, {1}, {GFR_DT_I64}));
    if (!shape_is(group_list, {E})) return GFR_ERR_BAD_SHAPE;
    const int64_t M = x->shape[0], K = x->shape[1];
    if (E < 1 || E > GFR_MAX_EXPERTS || M > int64_t{1} << 30 || K > int64_t{1} << 21 ||
        N > int64_t{1} << 21)
        return GFR_ERR_UNSUPPORTED;
    if (!aligned(x->data, 16) || !aligned(out->data, 16) || !aligned(group_list->data, 8))
        return GFR_ERR_BAD_ALIGNMENT;
    p.group_list = static_cast<const int64_t *>(group_list->data);
    p.cumsum = group_list_type == GFR_GROUP_LIST_CUMSUM;
    p.status = opts ? opts->status_dev : nullptr;
    p.out = out->data;
    p.f16 = x->dtype == GFR_DT_F16;
    p.out_f32 = out->dtype == GFR_DT_F32;
    p.M = static_cast<int32_t>(M);
    p.E = static_cast<int32_t>(E);
    return GFR_OK;
}

int check_lora_sizes(int64_t M, int64_t N, int64_t K, int64_t r) {
    if (M < 0 || N < 0 || K < 1) return GFR_ERR_BAD_SHAPE;
    if (r < 1 || r > GFR_MAX_RANK || M > int64_t{1} << 26 || N > int64_t{1} << 30 ||
        K > int64_t{1} << 21)
        return GFR_ERR_UNSUPPORTED;
    // (a grid has at most 2^32 threads, here a wave for four of a row's ranks)
    if (M * ((r + 3) / 4) > int64_t{1} << 25) return GFR_ERR_UNSUPPORTED;
    return gfr::linear_choice(M, N, K, GFR_ACT_NONE).split > 0 ? GFR_OK : GFR_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int gfr_linear_workspace_size(const gfr_tensor *x, const gfr_tensor *w, const gfr_tensor *bias,
                              const gfr_tensor *residual, int activation, const gfr_tensor *out,
                              size_t *bytes) {
    if (!bytes) return GFR_ERR_NULL_ARG;
    gfr::LinearParams p{};
    GFR_TRY(resolve_linear(x, w, bias, residual, activation, out, p));
    *bytes = linear_bytes(p);
    return GFR_OK;
}

int gfr_linear(const gfr_tensor *x, const gfr_tensor *w, const gfr_tensor *bias,
               const gfr_tensor *residual, int activation, const gfr_tensor *out, void *stream,
               const gfr_options *opts) {
    gfr::LinearParams p{};
    GFR_TRY(resolve_linear(x, w, bias, residual, activation, out, p));
    if (p.M == 0 || p.N == 0) return GFR_OK;
    GFR_TRY(check_workspace(opts, linear_bytes(p)));
    if (p.split > 1) p.partial = static_cast<float *>(opts->workspace);
    return gfr::launch_linear(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GFR_OK
                                                                                 : GFR_ERR_HIP;
}

int gfr_moe_decode_workspace_size(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I,
                                  int64_t N, int transpose_w13, int transpose_w2, size_t *bytes) {
    if (!bytes) return GFR_ERR_NULL_ARG;
    if ((transpose_w13 != 0 && transpose_w13 != 1) || (transpose_w2 != 0 && transpose_w2 != 1))
        return GFR_ERR_BAD_ARG;
    GFR_TRY(check_decode_sizes(T, k, E, H, I, N));
    *bytes = T > 0 && N > 0
                 ? gfr::decode_layout(T, k, E, H, I, N, transpose_w13, transpose_w2).total
                 : 0;
    return GFR_OK;
}

int gfr_moe_decode(const gfr_tensor *x, const gfr_tensor *w13, const gfr_tensor *scale13,
                   const gfr_tensor *w2, const gfr_tensor *scale2, const gfr_tensor *topk_ids,
                   const gfr_tensor *topk_weights, const gfr_tensor *shared_input,
                   float shared_input_weight, const gfr_tensor *out, int transpose_w13,
                   int transpose_w2, void *stream, const gfr_options *opts) {
    if (!x || !w13 || !scale13 || !w2 || !scale2 || !topk_ids || !topk_weights || !out)
        return GFR_ERR_NULL_ARG;
    GFR_TRY(check_desc(x, {2}, {GFR_DT_BF16}));
    GFR_TRY(check_desc(w13, {3}, {GFR_DT_FP8_E4M3FN, GFR_DT_FP8_E5M2}));
    GFR_TRY(check_desc(w2, {3}, {w13->dtype}));
    GFR_TRY(check_desc(topk_ids, {2}, {GFR_DT_I32}));
    GFR_TRY(check_desc(topk_weights, {2}, {GFR_DT_F32}));
    GFR_TRY(check_desc(out, {2}, {GFR_DT_BF16, GFR_DT_F32}));
    gfr::DecodeParams p{};
    const int64_t T = x->shape[0], H = x->shape[1], E = w13->shape[0], k = topk_ids->shape[1];
    int64_t N2 = 0, N = 0;
    GFR_TRY(resolve_weights(w13, scale13, transpose_w13, E, H, N2, p.s13_e));
    if (N2 % 2 != 0) return GFR_ERR_BAD_SHAPE;
    const int64_t I = N2 / 2;
    GFR_TRY(resolve_weights(w2, scale2, transpose_w2, E, I, N, p.s2_e));
    if (!shape_is(topk_ids, {T, k}) || !shape_is(topk_weights, {T, k}) || !shape_is(out, {T, N}))
        return GFR_ERR_BAD_SHAPE;
    if (present(shared_input)) {
        GFR_TRY(check_desc(shared_input, {2}, {GFR_DT_BF16}));
        if (!shape_is(shared_input, {T, N})) return GFR_ERR_BAD_SHAPE;
    }
    GFR_TRY(check_decode_sizes(T, k, E, H, I, N));
    if (T == 0 || N == 0) return GFR_OK;
    for (const gfr_tensor *t : {x, w13, scale13, w2, scale2, topk_ids, topk_weights, out})
        if (!aligned(t->data, 16)) return GFR_ERR_BAD_ALIGNMENT;
    if (present(shared_input) && !aligned(shared_input->data, 16)) return GFR_ERR_BAD_ALIGNMENT;
    const gfr::DecodeLayout d =
        gfr::decode_layout(T, k, E, H, I, N, transpose_w13, transpose_w2);
    GFR_TRY(check_workspace(opts, d.total));
    char *ws = static_cast<char *>(opts->workspace);
    p.x = static_cast<const uint16_t *>(x->data);
    p.w13 = static_cast<const uint8_t *>(w13->data);
    p.s13 = static_cast<const uint8_t *>(scale13->data);
    p.w2 = static_cast<const uint8_t *>(w2->data);
    p.s2 = static_cast<const uint8_t *>(scale2->data);
    p.ids = static_cast<const int32_t *>(topk_ids->data);
    p.weights = static_cast<const float *>(topk_weights->data);
    p.shared = present(shared_input) ? static_cast<const uint16_t *>(shared_input->data) : nullptr;
    p.shared_w = shared_input_weight;
    p.out = out->data;
    p.out_f32 = out->dtype == GFR_DT_F32;
    p.status = opts->status_dev;
    p.gu = reinterpret_cast<float *>(ws + d.gu);
    p.y = reinterpret_cast<float *>(ws + d.y);
    p.h = d.activate ? reinterpret_cast<uint16_t *>(ws + d.h) : nullptr;
    p.row_fragments = d.row_fragments;
    p.gate_up = d.gate_up;
    p.down = d.down;
    p.T = static_cast<int32_t>(T);
    p.k = static_cast<int32_t>(k);
    p.E = static_cast<int32_t>(E);
    p.H = static_cast<int32_t>(H);
    p.I = static_cast<int32_t>(I);
    p.N = static_cast<int32_t>(N);
    return gfr::launch_decode(p, transpose_w13, transpose_w2, w13->dtype == GFR_DT_FP8_E5M2,
                              static_cast<hipStream_t>(stream)) == hipSuccess
               ? GFR_OK
               : GFR_ERR_HIP;
}

int gfr_moe_route_workspace_size(int64_t T, int64_t E, int64_t k, size_t *bytes) {
    if (!bytes) return GFR_ERR_NULL_ARG;
    if (T < 0 || E < 1 || k < 1 || k > E) return GFR_ERR_BAD_SHAPE;
    if (E > GFR_MAX_EXPERTS || k > GFR_MAX_TOPK || T > kMaxTokens || T * k > kMaxRows)
        return GFR_ERR_UNSUPPORTED;
    *bytes = gfr::route_workspace(T, E, k);
    return GFR_OK;
}

int gfr_moe_route(const gfr_tensor *logits, const gfr_tensor *bias, int scoring, int n_group,
                  int topk_group, int renormalize, float scaling, const gfr_tensor *topk_ids,
                  const gfr_tensor *topk_weights, const gfr_tensor *x, const gfr_tensor *xin,
                  const gfr_tensor *xin_scale, const gfr_tensor *group_list,
                  const gfr_tensor *row_index, const gfr_tensor *logit, void *stream,
                  const gfr_options *opts) {
    if (!logits || !topk_ids || !topk_weights) return GFR_ERR_NULL_ARG;
    if (scoring != GFR_SCORE_SOFTMAX && scoring != GFR_SCORE_SIGMOID) return GFR_ERR_BAD_ARG;
    if (renormalize != 0 && renormalize != 1) return GFR_ERR_BAD_ARG;
    GFR_TRY(check_desc(logits, {2}, {GFR_DT_F32, GFR_DT_BF16}));
    GFR_TRY(check_desc(topk_ids, {2}, {GFR_DT_I32}));
    GFR_TRY(check_desc(topk_weights, {2}, {GFR_DT_F32}));
    const int64_t T = logits->shape[0], E = logits->shape[1], k = topk_ids->shape[1];
    if (E < 1 || k < 1 || k > E) return GFR_ERR_BAD_SHAPE;
    if (!shape_is(topk_ids, {T, k}) || !shape_is(topk_weights, {T, k})) return GFR_ERR_BAD_SHAPE;
    if (present(bias)) {
        GFR_TRY(check_desc(bias, {1}, {GFR_DT_F32}));
        if (!shape_is(bias, {E})) return GFR_ERR_BAD_SHAPE;
        if (!aligned(bias->data, 4)) return GFR_ERR_BAD_ALIGNMENT;
    }
    if (E > GFR_MAX_EXPERTS || k > GFR_MAX_TOPK || T > kMaxTokens || T * k > kMaxRows)
        return GFR_ERR_UNSUPPORTED;
    if (n_group < 1 || n_group > 64 || E % n_group != 0 || topk_group < 1 || topk_group > n_group)
        return GFR_ERR_BAD_ARG;
    gfr::RouteParams p{};
    if (x) {
        if (!xin || !xin_scale || !group_list || !row_index || !logit) return GFR_ERR_NULL_ARG;
        GFR_TRY(check_desc(x, {2}, {GFR_DT_BF16, GFR_DT_F16}));
        GFR_TRY(check_desc(xin, {2}, {GFR_DT_FP8_E4M3FN, GFR_DT_FP8_E5M2}));
        GFR_TRY(check_desc(xin_scale, {3}, kScaleTypes));
        GFR_TRY(check_desc(group_list, {1}, {GFR_DT_I64}));
        GFR_TRY(check_desc(row_index, {1}, {GFR_DT_I32}));
        GFR_TRY(check_desc(logit, {1}, {GFR_DT_F32}));
        const int64_t H = x->shape[1];
        if (x->shape[0] != T || H < 1 || !shape_is(xin, {T * k, H}) ||
            !shape_is(xin_scale, {T * k, (H + 63) / 64, 2}) || !shape_is(group_list, {E}) ||
            !shape_is(row_index, {T * k}) || !shape_is(logit, {T * k}))
            return GFR_ERR_BAD_SHAPE;
        if (H % 32 != 0 || H > kMaxRows) return GFR_ERR_UNSUPPORTED;
        if (!aligned(x->data, 16) || !aligned(xin->data, 16) || !aligned(group_list->data, 8) ||
            !aligned(row_index->data, 4) || !aligned(logit->data, 4))
            return GFR_ERR_BAD_ALIGNMENT;
        p.x = static_cast<const uint16_t *>(x->data);
        p.xin = static_cast<uint8_t *>(xin->data);
        p.xin_scale = static_cast<uint8_t *>(xin_scale->data);
        p.group_list = static_cast<int64_t *>(group_list->data);
        p.row_index = static_cast<int32_t *>(row_index->data);
        p.logit = static_cast<float *>(logit->data);
        p.x_f16 = x->dtype == GFR_DT_F16;
        p.e5m2 = xin->dtype == GFR_DT_FP8_E5M2;
        p.H = static_cast<int32_t>(H);
        const size_t need = gfr::route_workspace(T, E, k);
        GFR_TRY(check_workspace(opts, need));
        if (need) p.counts = static_cast<int32_t *>(opts->workspace);
    } else if (xin || xin_scale || group_list || row_index || logit) {
        return GFR_ERR_NULL_ARG;
    }
    if (!aligned(logits->data, logits->dtype == GFR_DT_F32 ? 4 : 2) ||
        !aligned(topk_ids->data, 4) || !aligned(topk_weights->data, 4))
        return GFR_ERR_BAD_ALIGNMENT;
    p.logits = logits->data;
    p.logits_bf16 = logits->dtype == GFR_DT_BF16;
    p.bias = present(bias) ? static_cast<const float *>(bias->data) : nullptr;
    p.ids = static_cast<int32_t *>(topk_ids->data);
    p.weights = static_cast<float *>(topk_weights->data);
    p.sigmoid = scoring == GFR_SCORE_SIGMOID;
    p.renormalize = renormalize;
    p.n_group = n_group;
    p.topk_group = topk_group;
    p.scaling = scaling;
    p.T = static_cast<int32_t>(T);
    p.E = static_cast<int32_t>(E);
    p.k = static_cast<int32_t>(k);
    return gfr::launch_route(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GFR_OK
                                                                                : GFR_ERR_HIP;
}

int gfr_grouped_linear(const gfr_tensor *x, const gfr_tensor *w, const gfr_tensor *group_list,
                       int group_list_type, int transpose_w, int fill, const gfr_tensor *out,
                       void *stream, const gfr_options *opts) {
    if (!x || !w || !group_list || !out) return GFR_ERR_NULL_ARG;
    GFR_TRY(check_desc(x, {2}, {GFR_DT_BF16, GFR_DT_F16}));
    GFR_TRY(check_desc(w, {3}, {x->dtype}));
    GFR_TRY(check_desc(out, {2}, {x->dtype, GFR_DT_F32}));
    const int64_t M = x->shape[0], K = x->shape[1], E = w->shape[0];
    const int64_t N = w->shape[transpose_w ? 1 : 2];
    gfr::GroupedParams p{};
    if (K < 1 || w->shape[transpose_w ? 2 : 1] != K || !shape_is(out, {M, N}))
        return GFR_ERR_BAD_SHAPE;
    GFR_TRY(resolve_groups(x, group_list, group_list_type, transpose_w, fill, E, N, out, opts, p));
    if (!aligned(w->data, 16)) return GFR_ERR_BAD_ALIGNMENT;
    if (M == 0 || N == 0) return GFR_OK;
    p.x = static_cast<const uint16_t *>(x->data);
    p.w = static_cast<const uint16_t *>(w->data);
    p.K = static_cast<int32_t>(K);
    p.N = static_cast<int32_t>(N);
    p.transpose = transpose_w;
    p.kernel = gfr::grouped_kernel(0, transpose_w, M, E, K, N);
    p.turn = transpose_w && M <= 128 * E;
    p.fill = fill;
    p.wide = N % 8 == 0;
    // (tiles are counted in 32 bits)
    if ((M / 64 + E + 2) * ((N + 63) / 64) > kMaxRows) return GFR_ERR_UNSUPPORTED;
    return gfr::launch_grouped(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GFR_OK
                                                                                  : GFR_ERR_HIP;
}

int gfr_grouped_linear_wgrad(const gfr_tensor *x, const gfr_tensor *dy,
                             const gfr_tensor *group_list, int group_list_type, int transpose_w,
                             int accumulate, const gfr_tensor *out, void *stream,
                             const gfr_options *opts) {
    if (!x || !dy || !group_list || !out) return GFR_ERR_NULL_ARG;
    GFR_TRY(check_desc(x, {2}, {GFR_DT_BF16, GFR_DT_F16}));
    GFR_TRY(check_desc(dy, {2}, {x->dtype}));
    GFR_TRY(check_desc(out, {3}, {x->dtype, GFR_DT_F32}));
    const int64_t M = x->shape[0], K = x->shape[1], N = dy->shape[1], E = out->shape[0];
    if (dy->shape[0] != M || !(transpose_w ? shape_is(out, {E, N, K}) : shape_is(out, {E, K, N})))
        return GFR_ERR_BAD_SHAPE;
    gfr::GroupedParams p{};
    GFR_TRY(resolve_groups(x, group_list, group_list_type, transpose_w, accumulate, E, N, out, opts,
                           p));
    if (!aligned(dy->data, 16)) return GFR_ERR_BAD_ALIGNMENT;
    if (K == 0 || N == 0 || (M == 0 && accumulate)) return GFR_OK;
    // the gradient of transposed weights is that of the other product, dy^T x
    const gfr_tensor *rows = transpose_w ? dy : x, *columns = transpose_w ? x : dy;
    p.x = static_cast<const uint16_t *>(rows->data);
    p.w = static_cast<const uint16_t *>(columns->data);
    p.K = static_cast<int32_t>(rows->shape[1]);
    p.N = static_cast<int32_t>(columns->shape[1]);
    p.wgrad = 1;
    p.accumulate = accumulate;
    p.kernel = gfr::grouped_kernel(1, 0, M, E, p.K, p.N);
    p.wide = p.N % 8 == 0;
    if (E * ((K + 63) / 64) * ((N + 63) / 64) > kMaxRows) return GFR_ERR_UNSUPPORTED;
    return gfr::launch_grouped(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GFR_OK
                                                                                  : GFR_ERR_HIP;
}

int gfr_lora_linear_workspace_size(int64_t M, int64_t N, int64_t K, int64_t r, size_t *bytes) {
    if (!bytes) return GFR_ERR_NULL_ARG;
    GFR_TRY(check_lora_sizes(M, N, K, r));
    *bytes = M > 0 && N > 0 ? gfr::lora_layout(M, N, K, r).total : 0;
    return GFR_OK;
}

int gfr_lora_linear(const gfr_tensor *x, const gfr_tensor *w, const gfr_tensor *bias,
                    const gfr_tensor *residual, const gfr_tensor *lora_a,
                    const gfr_tensor *lora_b, const gfr_tensor *adapter_ids,
                    const gfr_tensor *scaling, const gfr_tensor *out, void *stream,
                    const gfr_options *opts) {
    if (!lora_a || !lora_b || !adapter_ids) return GFR_ERR_NULL_ARG;
    gfr::LinearParams d{};
    GFR_TRY(resolve_linear(x, w, bias, residual, GFR_ACT_NONE, out, d));
    GFR_TRY(check_desc(lora_a, {3}, {x->dtype}));
    GFR_TRY(check_desc(lora_b, {3}, {x->dtype}));
    GFR_TRY(check_desc(adapter_ids, {1}, {GFR_DT_I32}));
    const int64_t M = d.M, N = d.N, K = d.K, L = lora_a->shape[0], r = lora_a->shape[1];
    if (lora_a->shape[2] != K || !shape_is(lora_b, {L, N, r}) || !shape_is(adapter_ids, {M}))
        return GFR_ERR_BAD_SHAPE;
    if (present(scaling)) {
        GFR_TRY(check_desc(scaling, {1}, {GFR_DT_F32}));
        if (!shape_is(scaling, {L})) return GFR_ERR_BAD_SHAPE;
        if (!aligned(scaling->data, 4)) return GFR_ERR_BAD_ALIGNMENT;
    }
    GFR_TRY(check_lora_sizes(M, N, K, r));
    if (L < 1 || L > int64_t{1} << 20) return GFR_ERR_UNSUPPORTED;
    if (!aligned(lora_a->data, 16) || !aligned(lora_b->data, 16) || !aligned(adapter_ids->data, 4))
        return GFR_ERR_BAD_ALIGNMENT;
    if (M == 0 || N == 0) return GFR_OK;
    const gfr::LoraLayout l = gfr::lora_layout(M, N, K, r);
    GFR_TRY(check_workspace(opts, l.total));
    char *ws = static_cast<char *>(opts->workspace);
    gfr::LoraParams p{};
    p.x = d.x;
    p.w = d.w;
    p.a = static_cast<const uint16_t *>(lora_a->data);
    p.b = static_cast<const uint16_t *>(lora_b->data);
    p.ids = static_cast<const int32_t *>(adapter_ids->data);
    p.scaling = present(scaling) ? static_cast<const float *>(scaling->data) : nullptr;
    p.bias = d.bias;
    p.residual = d.residual;
    p.out = d.out;
    p.status = opts->status_dev;
    p.inner = reinterpret_cast<float *>(ws);
    p.terms = reinterpret_cast<uint16_t *>(ws);
    p.codes = reinterpret_cast<int32_t *>(ws + l.codes);
    p.tiles = l.tiles;
    p.dense = reinterpret_cast<float *>(ws + l.dense);
    p.choice = l.choice;
    p.bias_f32 = d.bias_f32;
    p.out_f32 = d.out_f32;
    p.f16 = d.f16;
    p.M = d.M;
    p.N = d.N;
    p.K = d.K;
    p.L = static_cast<int32_t>(L);
    p.r = static_cast<int32_t>(r);
    return gfr::launch_lora(p, static_cast<hipStream_t>(stream)) == hipSuccess ? GFR_OK
                                                                               : GFR_ERR_HIP;
}

}  // extern "C"
