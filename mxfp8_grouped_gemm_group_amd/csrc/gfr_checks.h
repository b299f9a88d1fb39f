// Descriptor checks shared by the API sources (gfr_api.cpp, gfr_layer_api.cpp).
#pragma once

#include <stdint.h>

#include <initializer_list>

#include "gfr.h"

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// An optional tensor is absent when its descriptor or its data is NULL
// (with no element, NULL data is a present but empty tensor).
inline bool present(const gfr_tensor *t) { return t && t->data; }

inline int64_t numel(const gfr_tensor *t) {
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
    return n;
}

// Rank in `ranks` (GFR_ERR_BAD_RANK), no negative extent (GFR_ERR_BAD_SHAPE),
// dtype in `dtypes` (GFR_ERR_BAD_DTYPE), data present when the tensor holds
// any element (GFR_ERR_NULL_ARG).
inline int check_desc(const gfr_tensor *t, std::initializer_list<int> ranks,
               std::initializer_list<int> dtypes) {
    if (!t) return GFR_ERR_NULL_ARG;
    bool rank_ok = false;
    for (int r : ranks) rank_ok |= t->ndim == r;
    if (!rank_ok || t->ndim < 1 || t->ndim > 4) return GFR_ERR_BAD_RANK;
    for (int i = 0; i < t->ndim; ++i)
        if (t->shape[i] < 0) return GFR_ERR_BAD_SHAPE;
    bool dtype_ok = false;
    for (int d : dtypes) dtype_ok |= t->dtype == d;
    if (!dtype_ok) return GFR_ERR_BAD_DTYPE;
    if (!t->data && numel(t) > 0) return GFR_ERR_NULL_ARG;
    return GFR_OK;
}

inline bool shape_is(const gfr_tensor *t, std::initializer_list<int64_t> s) {
    if (static_cast<size_t>(t->ndim) != s.size()) return false;
    int i = 0;
    for (int64_t v : s)
        if (t->shape[i++] != v) return false;
    return true;
}

#define GFR_TRY(expr)                  \
    do {                               \
        const int rc_ = (expr);        \
        if (rc_ != GFR_OK) return rc_; \
    } while (0)

const std::initializer_list<int> kScaleTypes = {GFR_DT_E8M0, GFR_DT_U8};

}  // namespace
