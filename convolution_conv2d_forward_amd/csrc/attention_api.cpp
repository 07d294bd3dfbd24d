// C ABI of include/attention.h: descriptors, argument checks, dispatch.  Host
// code only.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <new>
#include <utility>

#include "attention_internal.h"

using namespace conv2d;

struct linear_desc {
    linear_params_t p;
};

struct qk_rope_desc {
    qk_rope_params_t p;
    double turns[ROPE_MAX_PAIRS];
};

struct attention_desc {
    attention_params_t p;
};

namespace {

constexpr int64_t kMaxRows = 0x7fffffff;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

int64_t elem_size(int32_t dtype) { return dtype == CONV_DTYPE_F32 ? 4 : 2; }

bool is_bool(int32_t v) { return v == 0 || v == 1; }

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

conv_status_t check_dtype(int32_t dtype) {
    if (dtype == CONV_DTYPE_I8) return fail(CONV_ERR_UNSUPPORTED, "dtype I8: these operators are F32 and BF16");
    if (dtype != CONV_DTYPE_F32 && dtype != CONV_DTYPE_BF16)
        return fail(CONV_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    return CONV_OK;
}

// A row stride that defaults to the row's length.
conv_status_t resolve_stride(int64_t& stride, int64_t len, const char* what) {
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
bool too_far(int64_t n, int64_t stride) { return stride > 0 && n > ((int64_t)1 << 44) / stride; }

// n rows of `len` elements at `stride`.
View rows_view(const void* p, int64_t n, int64_t stride, int64_t len, int64_t es) {
    return View{(uintptr_t)p, n, stride * es, len * es};
}

View flat_view(const void* p, int64_t bytes) { return View{(uintptr_t)p, p && bytes > 0 ? 1 : 0, 0, bytes}; }

template <typename D>
conv_status_t make_desc(const D& proto, D** out) {
    D* d = new (std::nothrow) D(proto);
    if (!d) return fail(CONV_ERR_HIP, "out of host memory");
    *out = d;
    return ok();
}

LinearArgs linear_args(const linear_params_t& p, int64_t rows, const void* x, const void* w, const float* bias,
                       const void* residual, void* y) {
    const int64_t es = elem_size(p.dtype), chunk = 16 / es;
    LinearArgs a;
    memset(&a, 0, sizeof(a));
    a.x = x; a.w = w; a.y = y;
    a.bias = p.has_bias ? bias : nullptr;
    a.residual = p.has_residual ? residual : nullptr;
    a.xs = p.x_stride; a.ys = p.y_stride; a.rs = p.residual_stride;
    a.m = (int32_t)rows; a.k = p.k; a.n = p.n;
    a.act = p.act_type; a.act_a = p.act_type == CONV_ACT_RELU ? 0.0f : p.act_params[0]; a.act_b = p.act_params[1];
    if ((p.x_stride > p.k ? p.x_stride : p.k) * es * 256 < (int64_t)1 << 32) {
        const auto rows_at = [&](int64_t bytes) {
            return p.k * es % bytes == 0 && p.x_stride * es % bytes == 0 && ((uintptr_t)x | (uintptr_t)w) % bytes == 0;
        };
        a.vec = rows_at(16) ? 16 : rows_at(4) ? 4 : 0;
    }
    const auto out_ok = [&](const void* q, int64_t stride) {
        return stride % chunk == 0 && aligned16(q);
    };
    a.vec_out = p.n % 8 == 0 && out_ok(y, p.y_stride) && (!p.has_residual || out_ok(residual, p.residual_stride)) &&
                (!p.has_bias || aligned16(bias));
    return a;
}

// Turns a position of each rotated pair.  The formulas are the header's.
void rope_turns(const qk_rope_params_t& p, double* turns) {
    const double pi = 3.14159265358979323846;
    const double r = p.rotary_dim, lt = std::log(p.theta);
    const auto index = [&](double n) { return r * std::log(p.original_len / (2 * pi * n)) / (2 * lt); };
    double lo = 0, hi = 0;
    if (p.scaling == ROPE_SCALING_YARN) {
        lo = std::fmax(std::floor(index(p.beta_fast)), 0.0);
        hi = std::fmin(std::ceil(index(p.beta_slow)), r - 1);
    }
    for (int i = 0; i < p.rotary_dim / 2; ++i) {
        double f = std::pow(p.theta, -2.0 * i / r);
        if (p.scaling == ROPE_SCALING_LINEAR) {
            f /= p.factor;
        } else if (p.scaling == ROPE_SCALING_YARN) {
            const double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            f = f * (1 - ramp) + f / p.factor * ramp;
        }
        turns[i] = f / (2 * pi);
    }
}

AttnArgs attn_args(const attention_params_t& p, int64_t batch, int64_t q_len, int64_t kv_len) {
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    memcpy(a.q_s, p.q_strides, sizeof(a.q_s));
    memcpy(a.k_s, p.k_strides, sizeof(a.k_s));
    memcpy(a.v_s, p.v_strides, sizeof(a.v_s));
    memcpy(a.o_s, p.out_strides, sizeof(a.o_s));
    a.batch = (int32_t)batch; a.q_len = (int32_t)q_len; a.kv_len = (int32_t)kv_len;
    a.heads_q = p.heads_q; a.heads_kv = p.heads_kv; a.group = p.heads_q / p.heads_kv; a.d = p.head_dim;
    a.causal = p.causal; a.window = p.window;
    a.rows = (int32_t)(q_len * a.group);
    a.scale = p.scale; a.softcap = p.softcap;
    return a;
}

constexpr int64_t kMaxLen = (int64_t)1 << 30;

conv_status_t check_attn_sizes(const attention_params_t& p, int64_t batch, int64_t q_len, int64_t kv_len) {
    if (batch < 0 || q_len < 0 || kv_len < 0) return fail(CONV_ERR_INVALID_ARG, "negative batch, q_len or kv_len");
    if (q_len > kMaxLen || kv_len > kMaxLen || batch > kMaxLen)
        return fail(CONV_ERR_INVALID_ARG, "batch, q_len or kv_len beyond 2^30");
    if (q_len * (p.heads_q / p.heads_kv) > kMaxLen)
        return fail(CONV_ERR_UNSUPPORTED, "q_len times the queries of a key head beyond 2^30");
    if (batch * p.heads_kv > kMaxRows) return fail(CONV_ERR_UNSUPPORTED, "batch times heads_kv beyond 2^31");
    const int64_t* all[4] = {p.q_strides, p.k_strides, p.v_strides, p.out_strides};
    for (int t = 0; t < 4; ++t)
        if (too_far(batch, all[t][0]) || too_far(t == 0 || t == 3 ? q_len : kv_len, all[t][1]) ||
            too_far(p.heads_q, all[t][2]))
            return fail(CONV_ERR_UNSUPPORTED, "a tensor reaches beyond 2^44 elements");
    return CONV_OK;
}

// The plan's grid: sequences may be divided over launches, one may not.
conv_status_t check_attn_grid(const AttnArgs& a, const AttnPlan& p) {
    if (sequence_workgroups(a, p) > most_workgroups(256))
        return fail(CONV_ERR_UNSUPPORTED, "a sequence's grid beyond 2^24 - 1 workgroups");
    return CONV_OK;
}

// From a tensor's first element to its last.
View span_view(const void* ptr, const int64_t* s, int64_t batch, int64_t len, int64_t heads, int64_t d, int64_t es) {
    if (!ptr || batch == 0 || len == 0) return View{(uintptr_t)ptr, 0, 0, 0};
    return View{(uintptr_t)ptr, 1, 0, ((batch - 1) * s[0] + (len - 1) * s[1] + (heads - 1) * s[2] + d) * es};
}

// Whether a tensor's dimensions lie within each other, so that no two elements
// share memory: each stride reaches past all that the smaller ones span.
bool nested(const int64_t* s, int64_t batch, int64_t len, int64_t heads, int64_t d) {
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

}  // namespace

extern "C" {

// ------------------------------------------------------------- linear ----

void linear_params_init(linear_params_t* p) {
    if (!p) return;
    memset(p, 0, sizeof(*p));
    p->act_params[0] = p->act_params[1] = NAN;
}

conv_status_t linear_desc_create(const linear_params_t* pp, linear_desc_t* out) {
    if (!pp || !out) return fail(CONV_ERR_INVALID_ARG, "null params or out");
    *out = nullptr;
    linear_params_t p = *pp;
    conv_status_t st = check_dtype(p.dtype);
    if (st != CONV_OK) return st;
    if (p.k < 1 || p.k > 1 << 24 || p.n < 1 || p.n > 1 << 24)
        return fail(CONV_ERR_INVALID_ARG, "k = %d and n = %d must be 1 .. 2^24", p.k, p.n);
    if (!is_bool(p.has_bias) || !is_bool(p.has_residual))
        return fail(CONV_ERR_INVALID_ARG, "has_bias and has_residual are 0 or 1");
    switch (p.act_type) {
    case CONV_ACT_NONE: case CONV_ACT_RELU: case LINEAR_ACT_SILU: case LINEAR_ACT_GELU: case LINEAR_ACT_GELU_TANH:
        break;
    case CONV_ACT_LEAKY_RELU:
        if (std::isnan(p.act_params[0])) p.act_params[0] = 0.01f;
        if (!std::isfinite(p.act_params[0])) return fail(CONV_ERR_INVALID_ARG, "non-finite LeakyReLU alpha");
        break;
    case CONV_ACT_CLIP:
        if (std::isnan(p.act_params[0])) p.act_params[0] = -FLT_MAX;
        if (std::isnan(p.act_params[1])) p.act_params[1] = FLT_MAX;
        if (p.act_params[0] > p.act_params[1]) return fail(CONV_ERR_INVALID_ARG, "clip lo > hi");
        break;
    case CONV_ACT_PRELU:
        return fail(CONV_ERR_UNSUPPORTED, "linear_forward has no PReLU");
    default:
        return fail(CONV_ERR_INVALID_ARG, "unknown activation %d", p.act_type);
    }
    if ((st = resolve_stride(p.x_stride, p.k, "x_stride")) != CONV_OK) return st;
    if ((st = resolve_stride(p.y_stride, p.n, "y_stride")) != CONV_OK) return st;
    if ((st = resolve_stride(p.residual_stride, p.n, "residual_stride")) != CONV_OK) return st;
    return make_desc(linear_desc{p}, out);
}

void linear_desc_destroy(linear_desc_t d) { delete d; }

const char* linear_desc_kernel_name(linear_desc_t d, int64_t rows) {
    if (!d || rows < 0 || rows > kMaxRows) return "";
    const void* p = (const void*)(uintptr_t)4096;
    return linear_kernel_name(d->p.dtype, linear_args(d->p, rows, p, p, (const float*)p, p, (void*)p));
}

conv_status_t linear_forward(linear_desc_t d, int64_t rows, const void* x, const void* w, const float* bias,
                             const void* residual, void* y, void* stream) {
    if (!d) return fail(CONV_ERR_INVALID_ARG, "null descriptor");
    const linear_params_t& p = d->p;
    if (rows < 0 || rows > kMaxRows) return fail(CONV_ERR_INVALID_ARG, "rows = %lld", (long long)rows);
    if (rows == 0) return ok();
    if (!x || !w || !y) return fail(CONV_ERR_INVALID_ARG, "null x, w or y");
    if (too_far(rows, p.x_stride) || too_far(rows, p.y_stride) || (p.has_residual && too_far(rows, p.residual_stride)))
        return fail(CONV_ERR_UNSUPPORTED, "a tensor reaches beyond 2^44 elements");
    if (p.has_bias && !bias) return fail(CONV_ERR_INVALID_ARG, "has_bias set but bias is null");
    if (p.has_residual && !residual) return fail(CONV_ERR_INVALID_ARG, "has_residual set but residual is null");
    const int64_t es = elem_size(p.dtype);
    if (((uintptr_t)x | (uintptr_t)w | (uintptr_t)y | (p.has_residual ? (uintptr_t)residual : 0)) & (uintptr_t)(es - 1))
        return fail(CONV_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
    if (p.has_bias && ((uintptr_t)bias & 3)) return fail(CONV_ERR_INVALID_ARG, "bias is not aligned to 4 bytes");
    const View yv = rows_view(y, rows, p.y_stride, p.n, es);
    if (views_overlap(yv, rows_view(x, rows, p.x_stride, p.k, es))) return fail(CONV_ERR_ALIAS, "y overlaps x");
    if (views_overlap(yv, flat_view(w, (int64_t)p.n * p.k * es))) return fail(CONV_ERR_ALIAS, "y overlaps w");
    if (p.has_bias && views_overlap(yv, flat_view(bias, 4 * (int64_t)p.n)))
        return fail(CONV_ERR_ALIAS, "y overlaps the bias");
    if (p.has_residual && !(residual == y && p.residual_stride == p.y_stride) &&
        views_overlap(yv, rows_view(residual, rows, p.residual_stride, p.n, es)))
        return fail(CONV_ERR_ALIAS, "y overlaps the residual without being it");
    const LinearArgs a = linear_args(p, rows, x, w, bias, residual, y);
    return hip_status(launch_linear(p.dtype, a, (hipStream_t)stream), "linear");
}

// ------------------------------------------------------------ qk_rope ----

void qk_rope_params_init(qk_rope_params_t* p) {
    if (!p) return;
    memset(p, 0, sizeof(*p));
    p->theta = 10000.0;
    p->factor = 1.0;
    p->beta_fast = 32.0;
    p->beta_slow = 1.0;
    p->eps = 1e-6f;
}

conv_status_t qk_rope_desc_create(const qk_rope_params_t* pp, qk_rope_desc_t* out) {
    if (!pp || !out) return fail(CONV_ERR_INVALID_ARG, "null params or out");
    *out = nullptr;
    qk_rope_desc d;
    memset(&d, 0, sizeof(d));
    d.p = *pp;
    qk_rope_params_t& p = d.p;
    conv_status_t st = check_dtype(p.dtype);
    if (st != CONV_OK) return st;
    if (p.heads_q < 1 || p.heads_kv < 1 || p.heads_q > 1 << 16 || p.heads_kv > 1 << 16)
        return fail(CONV_ERR_INVALID_ARG, "heads_q = %d, heads_kv = %d must be 1 .. 2^16", p.heads_q, p.heads_kv);
    if (p.head_dim < 1) return fail(CONV_ERR_INVALID_ARG, "head_dim = %d", p.head_dim);
    if (p.head_dim > 2 * ROPE_MAX_PAIRS) return fail(CONV_ERR_UNSUPPORTED, "head_dim = %d beyond 256", p.head_dim);
    if (p.rotary_dim == 0) p.rotary_dim = p.head_dim;
    if (p.rotary_dim < 0 || p.rotary_dim % 2) return fail(CONV_ERR_INVALID_ARG, "rotary_dim = %d must be even", p.rotary_dim);
    if (p.rotary_dim > p.head_dim)
        return fail(CONV_ERR_INCOMPATIBLE_SHAPES, "rotary_dim = %d beyond head_dim = %d", p.rotary_dim, p.head_dim);
    if (p.layout != ROPE_HALF && p.layout != ROPE_INTERLEAVED)
        return fail(CONV_ERR_INVALID_ARG, "unknown layout %d", p.layout);
    if (p.scaling < ROPE_SCALING_NONE || p.scaling > ROPE_SCALING_YARN)
        return fail(CONV_ERR_INVALID_ARG, "unknown scaling %d", p.scaling);
    if (!is_bool(p.has_norm)) return fail(CONV_ERR_INVALID_ARG, "has_norm is 0 or 1");
    if (!(p.eps >= 0) || !std::isfinite(p.eps)) return fail(CONV_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!(p.theta > 1) || !std::isfinite(p.theta)) return fail(CONV_ERR_INVALID_ARG, "theta must be finite and > 1");
    if (!(p.factor >= 1) || !std::isfinite(p.factor)) return fail(CONV_ERR_INVALID_ARG, "factor must be finite and >= 1");
    if (!(p.attn_factor >= 0) || !std::isfinite(p.attn_factor))
        return fail(CONV_ERR_INVALID_ARG, "attn_factor must be finite and >= 0");
    if (p.scaling == ROPE_SCALING_YARN &&
        (p.original_len < 1 || !(p.beta_fast > 0) || !(p.beta_slow > 0) || !std::isfinite(p.beta_fast) ||
         !std::isfinite(p.beta_slow)))
        return fail(CONV_ERR_INVALID_ARG, "YARN needs original_len >= 1 and finite beta_fast, beta_slow > 0");
    if (p.attn_factor == 0) p.attn_factor = p.scaling == ROPE_SCALING_YARN ? 0.1 * std::log(p.factor) + 1 : 1.0;
    const int64_t hd = p.head_dim;
    if ((st = resolve_stride(p.qkv_stride, (p.heads_q + 2 * (int64_t)p.heads_kv) * hd, "qkv_stride")) != CONV_OK) return st;
    if ((st = resolve_stride(p.q_stride, p.heads_q * hd, "q_stride")) != CONV_OK) return st;
    if ((st = resolve_stride(p.k_stride, p.heads_kv * hd, "k_stride")) != CONV_OK) return st;
    if ((st = resolve_stride(p.v_stride, p.heads_kv * hd, "v_stride")) != CONV_OK) return st;
    rope_turns(p, d.turns);
    return make_desc(d, out);
}

void qk_rope_desc_destroy(qk_rope_desc_t d) { delete d; }

conv_status_t qk_rope_forward(qk_rope_desc_t d, int64_t tokens, const void* qkv, const float* q_gamma,
                              const float* k_gamma, const int32_t* positions, const int32_t* slots,
                              int64_t cache_rows, void* q, void* k, void* v, void* stream) {
    if (!d) return fail(CONV_ERR_INVALID_ARG, "null descriptor");
    const qk_rope_params_t& p = d->p;
    if (tokens < 0 || tokens > kMaxRows || cache_rows < 0 || cache_rows > kMaxRows)
        return fail(CONV_ERR_INVALID_ARG, "tokens = %lld, cache_rows = %lld", (long long)tokens, (long long)cache_rows);
    if (tokens == 0) return ok();
    if (!qkv || !positions || !q || !k) return fail(CONV_ERR_INVALID_ARG, "null qkv, positions, q or k");
    if (p.has_norm && (!q_gamma || !k_gamma)) return fail(CONV_ERR_INVALID_ARG, "has_norm set but a gamma is null");
    if (!slots && cache_rows < tokens)
        return fail(CONV_ERR_INCOMPATIBLE_SHAPES, "%lld cache rows for %lld tokens without slots",
                    (long long)cache_rows, (long long)tokens);
    const int64_t es = elem_size(p.dtype), hd = p.head_dim;
    if (((uintptr_t)qkv | (uintptr_t)q | (uintptr_t)k | (uintptr_t)v) & (uintptr_t)(es - 1))
        return fail(CONV_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
    if (((uintptr_t)positions | (uintptr_t)slots | (p.has_norm ? (uintptr_t)q_gamma | (uintptr_t)k_gamma : 0)) & 3)
        return fail(CONV_ERR_INVALID_ARG, "positions, slots or a gamma is not aligned to 4 bytes");
    const int64_t krows = slots ? cache_rows : tokens;
    if (too_far(tokens, p.qkv_stride) || too_far(tokens, p.q_stride) || too_far(krows, p.k_stride) ||
        too_far(krows, p.v_stride))
        return fail(CONV_ERR_UNSUPPORTED, "a tensor reaches beyond 2^44 elements");
    const View in = rows_view(qkv, tokens, p.qkv_stride, (p.heads_q + 2 * (int64_t)p.heads_kv) * hd, es);
    const View qv = rows_view(q, tokens, p.q_stride, p.heads_q * hd, es);
    const View kv = rows_view(k, krows, p.k_stride, p.heads_kv * hd, es);
    const View vv = rows_view(v, v ? krows : 0, p.v_stride, p.heads_kv * hd, es);
    if (!(q == qkv && p.q_stride == p.qkv_stride) && views_overlap(qv, in))
        return fail(CONV_ERR_ALIAS, "q overlaps qkv without being it");
    if (views_overlap(kv, in) || views_overlap(vv, in)) return fail(CONV_ERR_ALIAS, "k or v overlaps qkv");
    if (views_overlap(qv, kv) || views_overlap(qv, vv) || views_overlap(kv, vv))
        return fail(CONV_ERR_ALIAS, "two outputs overlap");
    const View small[4] = {flat_view(positions, 4 * tokens), flat_view(slots, 4 * tokens),
                           flat_view(p.has_norm ? q_gamma : nullptr, 4 * hd),
                           flat_view(p.has_norm ? k_gamma : nullptr, 4 * hd)};
    for (const View& s : small)
        if (views_overlap(s, qv) || views_overlap(s, kv) || views_overlap(s, vv))
            return fail(CONV_ERR_ALIAS, "an output overlaps positions, slots or a gamma");
    RopeArgs a;
    memset(&a, 0, sizeof(a));
    a.qkv = qkv; a.positions = positions; a.slots = slots; a.q = q; a.k = k; a.v = v;
    a.q_gamma = p.has_norm ? q_gamma : nullptr;
    a.k_gamma = p.has_norm ? k_gamma : nullptr;
    a.qkv_s = p.qkv_stride; a.q_s = p.q_stride; a.k_s = p.k_stride; a.v_s = p.v_stride;
    a.cache_rows = krows;
    a.tokens = (int32_t)tokens; a.heads_q = p.heads_q; a.heads_kv = p.heads_kv;
    a.d = p.head_dim; a.r = p.rotary_dim; a.eps = p.eps; a.attn_factor = (float)p.attn_factor;
    a.turns = d->turns;
    const int64_t chunk = 16 / es;
    const bool vec = aligned16(qkv) && aligned16(q) && aligned16(k) && aligned16(v) &&
                     (!p.has_norm || (aligned16(q_gamma) && aligned16(k_gamma))) && p.head_dim % 8 == 0 &&
                     p.rotary_dim % 8 == 0 && p.qkv_stride % chunk == 0 && p.q_stride % chunk == 0 &&
                     p.k_stride % chunk == 0 && p.v_stride % chunk == 0;
    return hip_status(launch_qk_rope(p.dtype, p.layout, vec, a, (hipStream_t)stream), "qk_rope");
}

// ---------------------------------------------------------- attention ----

void attention_params_init(attention_params_t* p) {
    if (!p) return;
    memset(p, 0, sizeof(*p));
    p->scale = NAN;
}

conv_status_t attention_desc_create(const attention_params_t* pp, attention_desc_t* out) {
    if (!pp || !out) return fail(CONV_ERR_INVALID_ARG, "null params or out");
    *out = nullptr;
    attention_params_t p = *pp;
    conv_status_t st = check_dtype(p.dtype);
    if (st != CONV_OK) return st;
    if (p.heads_q < 1 || p.heads_kv < 1 || p.heads_q > 1 << 16)
        return fail(CONV_ERR_INVALID_ARG, "heads_q = %d, heads_kv = %d must be 1 .. 2^16", p.heads_q, p.heads_kv);
    if (p.heads_q % p.heads_kv)
        return fail(CONV_ERR_INCOMPATIBLE_SHAPES, "heads_kv = %d does not divide heads_q = %d", p.heads_kv, p.heads_q);
    if (p.head_dim < 1) return fail(CONV_ERR_INVALID_ARG, "head_dim = %d", p.head_dim);
    const int64_t chunk = 16 / elem_size(p.dtype);
    if (p.head_dim > 256 || p.head_dim % chunk)
        return fail(CONV_ERR_UNSUPPORTED, "head_dim = %d is not a multiple of %d up to 256", p.head_dim, (int)chunk);
    if (!is_bool(p.causal) || !is_bool(p.has_slopes)) return fail(CONV_ERR_INVALID_ARG, "causal and has_slopes are 0 or 1");
    if (p.window < 0) return fail(CONV_ERR_INVALID_ARG, "window = %d", p.window);
    if (!(p.softcap >= 0) || !std::isfinite(p.softcap)) return fail(CONV_ERR_INVALID_ARG, "softcap must be finite and >= 0");
    if (std::isnan(p.scale)) p.scale = 1.0f / std::sqrt((float)p.head_dim);
    if (!std::isfinite(p.scale)) return fail(CONV_ERR_INVALID_ARG, "non-finite scale");
    const int64_t* all[4] = {p.q_strides, p.k_strides, p.v_strides, p.out_strides};
    for (int t = 0; t < 4; ++t) {
        for (int i = 0; i < 3; ++i) {
            const int64_t s = all[t][i];
            if (s < 0 || s > kMaxStride) return fail(CONV_ERR_INVALID_ARG, "a stride outside 0 .. 2^40");
            if (s % chunk) return fail(CONV_ERR_UNSUPPORTED, "a stride is not a multiple of 16 bytes");
            if (t == 3 && s < p.head_dim)
                return fail(CONV_ERR_INCOMPATIBLE_SHAPES, "an output stride is below head_dim");
        }
    }
    return make_desc(attention_desc{p}, out);
}

void attention_desc_destroy(attention_desc_t d) { delete d; }

conv_status_t attention_workspace_bytes(attention_desc_t d, int64_t batch, int64_t q_len, int64_t kv_len,
                                        int64_t* bytes) {
    if (!d || !bytes) return fail(CONV_ERR_INVALID_ARG, "null descriptor or bytes");
    const conv_status_t st = check_attn_sizes(d->p, batch, q_len, kv_len);
    if (st != CONV_OK) return st;
    *bytes = 0;
    if (batch == 0 || q_len == 0) return ok();
    const AttnArgs a = attn_args(d->p, batch, q_len, kv_len);
    const AttnPlan plan = plan_attention(d->p.dtype, a);
    if (check_attn_grid(a, plan) != CONV_OK) return CONV_ERR_UNSUPPORTED;
    *bytes = plan.ws_bytes;
    return ok();
}

conv_status_t attention_forward(attention_desc_t d, int64_t batch, int64_t q_len, int64_t kv_len, const void* q,
                                const void* k, const void* v, const int32_t* q_lens, const int32_t* kv_lens,
                                const int32_t* prefix_lens, const int32_t* doc_offsets, int32_t n_docs,
                                const float* slopes, void* out, void* workspace, int64_t workspace_bytes,
                                void* stream) {
    if (!d) return fail(CONV_ERR_INVALID_ARG, "null descriptor");
    const attention_params_t& p = d->p;
    const conv_status_t st = check_attn_sizes(p, batch, q_len, kv_len);
    if (st != CONV_OK) return st;
    if (batch == 0 || q_len == 0) return ok();
    if (!q || !out || (kv_len > 0 && (!k || !v))) return fail(CONV_ERR_INVALID_ARG, "null q, k, v or out");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(workspace))
        return fail(CONV_ERR_INVALID_ARG, "a tensor or the workspace is not aligned to 16 bytes");
    if (((uintptr_t)q_lens | (uintptr_t)kv_lens | (uintptr_t)prefix_lens | (uintptr_t)doc_offsets | (uintptr_t)slopes) & 3)
        return fail(CONV_ERR_INVALID_ARG, "lengths, offsets or slopes are not aligned to 4 bytes");
    if (p.has_slopes && !slopes) return fail(CONV_ERR_INVALID_ARG, "has_slopes set but slopes is null");
    if (doc_offsets && n_docs < 1) return fail(CONV_ERR_INVALID_ARG, "doc_offsets with n_docs = %d", n_docs);
    AttnArgs a = attn_args(p, batch, q_len, kv_len);
    const AttnPlan plan = plan_attention(p.dtype, a);
    if (check_attn_grid(a, plan) != CONV_OK) return CONV_ERR_UNSUPPORTED;
    if (plan.ws_bytes > 0 && (!workspace || workspace_bytes < plan.ws_bytes))
        return fail(CONV_ERR_INVALID_ARG, "a workspace of %lld bytes is needed", (long long)plan.ws_bytes);
    const int64_t es = elem_size(p.dtype);
    const View ov = span_view(out, p.out_strides, batch, q_len, p.heads_q, p.head_dim, es);
    const View wv = flat_view(workspace, plan.ws_bytes);
    const View in[8] = {span_view(q, p.q_strides, batch, q_len, p.heads_q, p.head_dim, es),
                        span_view(k, p.k_strides, batch, kv_len, p.heads_kv, p.head_dim, es),
                        span_view(v, p.v_strides, batch, kv_len, p.heads_kv, p.head_dim, es),
                        flat_view(q_lens, 4 * batch),
                        flat_view(kv_lens, 4 * batch),
                        flat_view(prefix_lens, 4 * batch),
                        flat_view(doc_offsets, 4 * batch * ((int64_t)n_docs + 1)),
                        flat_view(p.has_slopes ? slopes : nullptr, 4 * (int64_t)p.heads_q)};
    if (!nested(p.out_strides, batch, q_len, p.heads_q, p.head_dim))
        return fail(CONV_ERR_ALIAS, "rows of out share memory");
    if (views_overlap(ov, wv)) return fail(CONV_ERR_ALIAS, "out overlaps the workspace");
    for (const View& iv : in)
        if (views_overlap(ov, iv) || views_overlap(wv, iv))
            return fail(CONV_ERR_ALIAS, "out or the workspace overlaps an input");
    a.q = q; a.k = k; a.v = v; a.out = out;
    a.q_lens = q_lens; a.kv_lens = kv_lens; a.prefix_lens = prefix_lens;
    a.doc_offsets = doc_offsets; a.n_docs = doc_offsets ? n_docs : 0;
    a.slopes = p.has_slopes ? slopes : nullptr;
    a.ws = plan.ws_bytes > 0 ? (float*)workspace : nullptr;
    a.row_tiles = plan.row_tiles; a.splits = plan.splits;
    return hip_status(launch_attention(p.dtype, plan, a, (hipStream_t)stream), "attention");
}

}  // extern "C"
