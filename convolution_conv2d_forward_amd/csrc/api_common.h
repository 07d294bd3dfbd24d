// Argument checks shared by the ABI layers of include/attention.h and
// include/decoder.h.  Host code only.
#pragma once

#include <algorithm>
#include <cstring>
#include <new>
#include <utility>

#include "conv2d_internal.h"

namespace conv2d {

constexpr int64_t kMaxRows = 0x7fffffff;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

inline int64_t elem_size(int32_t dtype) { return dtype == CONV_DTYPE_F32 ? 4 : 2; }

inline bool is_bool(int32_t v) { return v == 0 || v == 1; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

inline conv_status_t check_dtype(int32_t dtype) {
    if (dtype == CONV_DTYPE_I8) return fail(CONV_ERR_UNSUPPORTED, "dtype I8: these operators are F32 and BF16");
    if (dtype != CONV_DTYPE_F32 && dtype != CONV_DTYPE_BF16)
        return fail(CONV_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    return CONV_OK;
}

// A row stride that defaults to the row's length.
inline conv_status_t resolve_stride(int64_t& stride, int64_t len, const char* what) {
    if (stride == 0) stride = len;
    if (stride < 0 || stride > kMaxStride)
        return fail(CONV_ERR_INVALID_ARG, "%s = %lld outside 0 .. 2^40", what, (long long)stride);
    if (stride < len)
        return fail(CONV_ERR_INCOMPATIBLE_SHAPES, "%s = %lld is below the row's %lld elements", what,
                    (long long)stride, (long long)len);
    return CONV_OK;
}

// n steps of `stride` elements reach beyond what 64-bit byte offsets are
// checked for here (2^44 elements; no device holds that much).
inline bool too_far(int64_t n, int64_t stride) { return stride > 0 && n > ((int64_t)1 << 44) / stride; }

// n rows of `len` elements at `stride`.
inline View rows_view(const void* p, int64_t n, int64_t stride, int64_t len, int64_t es) {
    return View{(uintptr_t)p, n, stride * es, len * es};
}

inline View flat_view(const void* p, int64_t bytes) { return View{(uintptr_t)p, p && bytes > 0 ? 1 : 0, 0, bytes}; }

template <typename D>
conv_status_t make_desc(const D& proto, D** out) {
    D* d = new (std::nothrow) D(proto);
    if (!d) return fail(CONV_ERR_HIP, "out of host memory");
    *out = d;
    return ok();
}

// Whether a tensor's dimensions lie within each other, so that no two elements
// share memory: each stride reaches past all that the smaller ones span.
inline bool nested(const int64_t* s, int64_t batch, int64_t len, int64_t heads, int64_t d) {
    std::pair<int64_t, int64_t> dims[3] = {{s[0], batch}, {s[1], len}, {s[2], heads}};
    std::sort(dims, dims + 3);
    int64_t span = d;
    for (const auto& [stride, n] : dims) {
        if (n <= 1) continue;
        if (stride < span) return false;
        span += (n - 1) * stride;
    }
    return true;
}

}  // namespace conv2d
