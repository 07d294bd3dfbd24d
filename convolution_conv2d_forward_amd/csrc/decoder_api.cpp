// C ABI of include/decoder.h: descriptors, argument checks, dispatch.  Host
// code only.
#include <cmath>
#include <cstring>

#include "api_common.h"
#include "decoder_internal.h"

using namespace conv2d;

struct kv_cache_desc {
    kv_cache_params_t p;
};

struct paged_attention_desc {
    paged_attention_params_t p;
};

struct block_norm_desc {
    block_norm_params_t p;
};

namespace {

constexpr int64_t kMaxLen = (int64_t)1 << 30;

conv_status_t check_cache_dtype(int32_t dtype, int32_t cache) {
    const conv_status_t st = check_dtype(dtype);
    if (st != CONV_OK) return st;
    if (cache != dtype && cache != KV_CACHE_E4M3) {
        if (cache == CONV_DTYPE_F32 || cache == CONV_DTYPE_BF16 || cache == CONV_DTYPE_I8)
            return fail(CONV_ERR_UNSUPPORTED, "a cache is of the call's dtype or E4M3");
        return fail(CONV_ERR_INVALID_ARG, "unknown cache_dtype %d", cache);
    }
    return CONV_OK;
}

int64_t cache_elem_size(int32_t cache) { return cache == KV_CACHE_E4M3 ? 1 : elem_size(cache); }

// (page, token, head) strides that default to dense ones.
conv_status_t resolve_page_strides(int64_t* s, int64_t page_size, int64_t heads, int64_t len, const char* what) {
    if (s[0] == 0 && s[1] == 0 && s[2] == 0) {
        s[2] = len;
        s[1] = heads * len;
        s[0] = page_size * s[1];
    }
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] > kMaxStride)
            return fail(CONV_ERR_INVALID_ARG, "%s outside 0 .. 2^40", what);
    return CONV_OK;
}

bool pages_too_far(const int64_t* s, int64_t n_pages, int64_t page_size, int64_t heads) {
    return too_far(n_pages, s[0]) || too_far(page_size, s[1]) || too_far(heads, s[2]);
}

// Elements from the first to the last one of `n_pages` pages, all heads.
int64_t pages_span(const int64_t* s, int64_t n_pages, int64_t page_size, int64_t heads, int64_t len) {
    return (n_pages - 1) * s[0] + (page_size - 1) * s[1] + (heads - 1) * s[2] + len;
}

// The pages' bytes: page by page where the pages lie apart (another tensor's
// may lie between them), else from the first to the last.
View pages_view(const void* p, const int64_t* s, int64_t n_pages, int64_t page_size, int64_t heads, int64_t len,
                int64_t es) {
    if (!p || n_pages == 0) return View{(uintptr_t)p, 0, 0, 0};
    const int64_t inner = pages_span(s, 1, page_size, heads, len);
    if (n_pages > 1 && s[0] >= inner) return View{(uintptr_t)p, n_pages, s[0] * es, inner * es};
    return View{(uintptr_t)p, 1, 0, pages_span(s, n_pages, page_size, heads, len) * es};
}

// A tensor of rows of `len` bytes at three strides (bytes), and its view.
struct Grid {
    uintptr_t base;
    int64_t stride[3], n[3], len;
    View view;
};

Grid pages_grid(const void* p, const int64_t* s, int64_t n_pages, int64_t page_size, int64_t heads, int64_t len, int64_t es) {
    return Grid{(uintptr_t)p, {s[0] * es, s[1] * es, s[2] * es}, {n_pages, page_size, heads}, len * es,
                pages_view(p, s, n_pages, page_size, heads, len, es)};
}

// Whether rows of two grids of the same strides and counts overlap, `delta` bytes
// apart: dimension by dimension from the largest stride on, those differences of
// the two indices that the smaller strides can still make up for.  They are three
// at most where the dimensions lie within each other.
bool rows_meet(const std::pair<int64_t, int64_t>* dims, int count, int64_t delta, int64_t a_len, int64_t b_len) {
    if (count == 0) return delta < a_len && -delta < b_len;
    const auto [stride, n] = dims[0];
    int64_t inner = 0;
    for (int i = 1; i < count; ++i) inner += dims[i].first * (dims[i].second - 1);
    const auto floor_div = [](int64_t x, int64_t d) { return x >= 0 ? x / d : -((-x + d - 1) / d); };
    int64_t lo = -floor_div(inner + b_len - 1 + delta, stride), hi = floor_div(inner + a_len - 1 - delta, stride);
    if (lo < -(n - 1)) lo = -(n - 1);
    if (hi > n - 1) hi = n - 1;
    for (int64_t i = lo; i <= hi; ++i)
        if (rows_meet(dims + 1, count - 1, delta + i * stride, a_len, b_len)) return true;
    return false;
}

// Whether two tensors, each with its dimensions within each other, share memory.
// Exact where they have the same strides in bytes, as tensors that are interleaved
// in one buffer have; otherwise by their views.
bool grids_overlap(const Grid& a, const Grid& b) {
    if (!views_overlap(a.view, b.view)) return false;
    std::pair<int64_t, int64_t> dims[3];
    int count = 0;
    for (int i = 0; i < 3; ++i) {
        if (a.n[i] != b.n[i]) return true;
        if (a.n[i] <= 1) continue;
        if (a.stride[i] != b.stride[i]) return true;
        dims[count++] = {a.stride[i], a.n[i]};
    }
    std::sort(dims, dims + count, [](const auto& x, const auto& y) { return x.first > y.first; });
    return rows_meet(dims, count, (int64_t)(b.base - a.base), a.len, b.len);
}

PageStrides page_strides(const int64_t* s) { return PageStrides{s[0], s[1], s[2]}; }

bool misaligned(const void* p, int64_t bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) != 0; }

KvArgs kv_args(const kv_cache_params_t& p, int64_t n_pages, const void* k_pages, const void* v_pages,
               const uint8_t* k_scales, const uint8_t* v_scales, const void* k, const void* v) {
    KvArgs a;
    memset(&a, 0, sizeof(a));
    a.k = k; a.v = v; a.k_pages = k_pages; a.v_pages = v_pages;
    const bool e4m3 = p.cache_dtype == KV_CACHE_E4M3;
    a.k_scales = e4m3 ? k_scales : nullptr;
    a.v_scales = e4m3 ? v_scales : nullptr;
    a.k_s = p.k_stride; a.v_s = p.v_stride;
    a.ks = page_strides(p.k_page_strides); a.vs = page_strides(p.v_page_strides); a.ss = page_strides(p.scale_strides);
    a.n_pages = (int32_t)n_pages; a.heads = p.heads_kv; a.d = p.head_dim;
    a.page_size = make_divu32((uint32_t)p.page_size);
    return a;
}

// Whether rows can be moved 8 elements at a time.
bool kv_vec(const kv_cache_params_t& p, const KvArgs& a) {
    const int64_t es = elem_size(p.dtype), cs = cache_elem_size(p.cache_dtype);
    const int64_t wide = es * 8 < 16 ? es * 8 : 16, cwide = cs * 8 < 16 ? cs * 8 : 16;
    const auto ok16 = [](const void* q, std::initializer_list<int64_t> strides, int64_t size, int64_t bytes) {
        if (misaligned(q, bytes)) return false;
        for (int64_t s : strides)
            if (s * size % bytes) return false;
        return true;
    };
    return p.head_dim % 8 == 0 && ok16(a.k, {a.k_s, a.k_bs}, es, wide) && ok16(a.v, {a.v_s, a.v_bs}, es, wide) &&
           ok16(a.k_pages, {a.ks.page, a.ks.token, a.ks.head}, cs, cwide) &&
           ok16(a.v_pages, {a.vs.page, a.vs.token, a.vs.head}, cs, cwide);
}

// The checks that kv_cache_store and kv_cache_load share.
conv_status_t check_kv(const kv_cache_params_t& p, int64_t n_pages, const void* k_pages, const void* v_pages,
                       const uint8_t* k_scales, const uint8_t* v_scales, const void* k, const void* v) {
    if (!k || !v) return fail(CONV_ERR_INVALID_ARG, "null k or v");
    if (n_pages > 0 && (!k_pages || !v_pages)) return fail(CONV_ERR_INVALID_ARG, "null k_pages or v_pages");
    const bool e4m3 = p.cache_dtype == KV_CACHE_E4M3;
    if (e4m3 && n_pages > 0 && (!k_scales || !v_scales))
        return fail(CONV_ERR_INVALID_ARG, "an E4M3 cache needs k_scales and v_scales");
    const int64_t es = elem_size(p.dtype), cs = cache_elem_size(p.cache_dtype);
    if (misaligned(k, es) || misaligned(v, es) || misaligned(k_pages, cs) || misaligned(v_pages, cs))
        return fail(CONV_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
    if (pages_too_far(p.k_page_strides, n_pages, p.page_size, p.heads_kv) ||
        pages_too_far(p.v_page_strides, n_pages, p.page_size, p.heads_kv) ||
        (e4m3 && pages_too_far(p.scale_strides, n_pages, p.page_size, p.heads_kv)))
        return fail(CONV_ERR_UNSUPPORTED, "a tensor reaches beyond 2^44 elements");
    return CONV_OK;
}

struct KvGrids {
    Grid pages[4];   // keys, values, their scales
    int n;
};

KvGrids kv_grids(const kv_cache_params_t& p, int64_t n_pages, const void* k_pages, const void* v_pages,
                 const uint8_t* k_scales, const uint8_t* v_scales) {
    const int64_t cs = cache_elem_size(p.cache_dtype), ps = p.page_size, h = p.heads_kv, d = p.head_dim;
    KvGrids v{{pages_grid(k_pages, p.k_page_strides, n_pages, ps, h, d, cs),
               pages_grid(v_pages, p.v_page_strides, n_pages, ps, h, d, cs),
               pages_grid(k_scales, p.scale_strides, n_pages, ps, h, 1, 1),
               pages_grid(v_scales, p.scale_strides, n_pages, ps, h, 1, 1)},
              p.cache_dtype == KV_CACHE_E4M3 ? 4 : 2};
    return v;
}

PagedArgs paged_args(const paged_attention_params_t& p, int64_t tokens, int64_t batch, int64_t max_pages,
                     int64_t n_pages) {
    PagedArgs a;
    memset(&a, 0, sizeof(a));
    a.q_s = p.q_stride; a.o_s = p.out_stride;
    const int64_t cs = cache_elem_size(p.cache_dtype);
    const auto units = [&](const int64_t* s, int64_t size, int64_t per) {
        return PageUnits{(uint32_t)(s[0] * size / per), (uint32_t)(s[1] * size / per)};
    };
    a.k_u = units(p.k_page_strides, cs, 16); a.v_u = units(p.v_page_strides, cs, 16);
    a.s_u = units(p.scale_strides, 1, 1);
    a.k_head = p.k_page_strides[2] * cs; a.v_head = p.v_page_strides[2] * cs; a.s_head = p.scale_strides[2];
    a.tokens = (int32_t)tokens; a.batch = (int32_t)batch;
    a.max_pages = (int32_t)max_pages; a.n_pages = (int32_t)n_pages;
    a.heads_q = p.heads_q; a.heads_kv = p.heads_kv; a.group = p.heads_q / p.heads_kv; a.d = p.head_dim;
    a.window = p.window; a.sinks = p.sinks;
    a.page_size = make_divu32((uint32_t)p.page_size);
    a.group_div = make_divu32((uint32_t)a.group);
    a.scale = p.scale; a.softcap = p.softcap;
    return a;
}

conv_status_t check_paged_sizes(const paged_attention_params_t& p, int64_t tokens, int64_t batch, int64_t max_pages) {
    if (tokens < 0 || batch < 0 || max_pages < 0) return fail(CONV_ERR_INVALID_ARG, "negative tokens, batch or max_pages");
    if (tokens > kMaxLen || batch > kMaxLen || max_pages > kMaxLen || max_pages * p.page_size > kMaxLen)
        return fail(CONV_ERR_INVALID_ARG, "tokens, batch or max_pages * page_size beyond 2^30");
    if (tokens * (p.heads_q / p.heads_kv) > kMaxLen)
        return fail(CONV_ERR_UNSUPPORTED, "tokens times the queries of a key head beyond 2^30");
    if (too_far(tokens, p.q_stride) || too_far(tokens, p.out_stride) || too_far(batch, max_pages))
        return fail(CONV_ERR_UNSUPPORTED, "a tensor reaches beyond 2^44 elements");
    return CONV_OK;
}

}  // namespace

extern "C" {

// ----------------------------------------------------------- kv_cache ----

void kv_cache_params_init(kv_cache_params_t* p) {
    if (!p) return;
    memset(p, 0, sizeof(*p));
}

conv_status_t kv_cache_desc_create(const kv_cache_params_t* pp, kv_cache_desc_t* out) {
    if (!pp || !out) return fail(CONV_ERR_INVALID_ARG, "null params or out");
    *out = nullptr;
    kv_cache_params_t p = *pp;
    conv_status_t st = check_cache_dtype(p.dtype, p.cache_dtype);
    if (st != CONV_OK) return st;
    if (p.heads_kv < 1 || p.heads_kv > 1 << 16) return fail(CONV_ERR_INVALID_ARG, "heads_kv = %d must be 1 .. 2^16", p.heads_kv);
    if (p.head_dim < 1) return fail(CONV_ERR_INVALID_ARG, "head_dim = %d", p.head_dim);
    if (p.head_dim > 256) return fail(CONV_ERR_UNSUPPORTED, "head_dim = %d beyond 256", p.head_dim);
    if (p.page_size < 1 || p.page_size > 1 << 16)
        return fail(CONV_ERR_INVALID_ARG, "page_size = %d must be 1 .. 2^16", p.page_size);
    const int64_t row = (int64_t)p.heads_kv * p.head_dim;
    if ((st = resolve_stride(p.k_stride, row, "k_stride")) != CONV_OK) return st;
    if ((st = resolve_stride(p.v_stride, row, "v_stride")) != CONV_OK) return st;
    for (int64_t s : {p.k_batch_stride, p.v_batch_stride})
        if (s < 0 || s > kMaxStride) return fail(CONV_ERR_INVALID_ARG, "a batch stride outside 0 .. 2^40");
    const int64_t d = p.head_dim;
    if ((st = resolve_page_strides(p.k_page_strides, p.page_size, p.heads_kv, d, "k_page_strides")) != CONV_OK ||
        (st = resolve_page_strides(p.v_page_strides, p.page_size, p.heads_kv, d, "v_page_strides")) != CONV_OK ||
        (st = resolve_page_strides(p.scale_strides, p.page_size, p.heads_kv, 1, "scale_strides")) != CONV_OK)
        return st;
    for (int i = 0; i < 3; ++i)
        if (p.k_page_strides[i] < d || p.v_page_strides[i] < d || p.scale_strides[i] < 1)
            return fail(CONV_ERR_INCOMPATIBLE_SHAPES, "a page stride is below head_dim, or a scale's is 0");
    return make_desc(kv_cache_desc{p}, out);
}

void kv_cache_desc_destroy(kv_cache_desc_t d) { delete d; }

conv_status_t kv_cache_store(kv_cache_desc_t desc, int64_t tokens, const void* k, const void* v, const int32_t* slots,
                             int64_t n_pages, void* k_pages, void* v_pages, uint8_t* k_scales, uint8_t* v_scales,
                             void* stream) {
    if (!desc) return fail(CONV_ERR_INVALID_ARG, "null descriptor");
    const kv_cache_params_t& p = desc->p;
    if (tokens < 0 || tokens > kMaxRows || n_pages < 0 || n_pages > kMaxRows || n_pages * p.page_size > kMaxRows)
        return fail(CONV_ERR_INVALID_ARG, "tokens = %lld or n_pages = %lld", (long long)tokens, (long long)n_pages);
    if (tokens == 0) return ok();
    conv_status_t st = check_kv(p, n_pages, k_pages, v_pages, k_scales, v_scales, k, v);
    if (st != CONV_OK) return st;
    if (!slots) return fail(CONV_ERR_INVALID_ARG, "null slots");
    if (misaligned(slots, 4)) return fail(CONV_ERR_INVALID_ARG, "slots is not aligned to 4 bytes");
    if (too_far(tokens, p.k_stride) || too_far(tokens, p.v_stride))
        return fail(CONV_ERR_UNSUPPORTED, "a tensor reaches beyond 2^44 elements");
    const bool e4m3 = p.cache_dtype == KV_CACHE_E4M3;
    const int64_t ps = p.page_size, h = p.heads_kv, hd = p.head_dim, es = elem_size(p.dtype);
    if (!nested(p.k_page_strides, n_pages, ps, h, hd) || !nested(p.v_page_strides, n_pages, ps, h, hd) ||
        (e4m3 && !nested(p.scale_strides, n_pages, ps, h, 1)))
        return fail(CONV_ERR_ALIAS, "elements of the pages share memory");
    const KvGrids out = kv_grids(p, n_pages, k_pages, v_pages, k_scales, v_scales);
    const View in[3] = {rows_view(k, tokens, p.k_stride, h * hd, es), rows_view(v, tokens, p.v_stride, h * hd, es),
                        flat_view(slots, 4 * tokens)};
    for (int i = 0; i < out.n; ++i) {
        for (const View& iv : in)
            if (views_overlap(out.pages[i].view, iv)) return fail(CONV_ERR_ALIAS, "pages or scales overlap an input");
        for (int j = 0; j < i; ++j)
            if (grids_overlap(out.pages[i], out.pages[j])) return fail(CONV_ERR_ALIAS, "pages or scales overlap each other");
    }
    if (n_pages == 0) return ok();   // no slot to store to
    KvArgs a = kv_args(p, n_pages, k_pages, v_pages, k_scales, v_scales, k, v);
    a.slots = slots;
    a.tokens = (int32_t)tokens;
    return hip_status(launch_kv_store(p.dtype, e4m3, kv_vec(p, a), a, (hipStream_t)stream), "kv_cache_store");
}

conv_status_t kv_cache_load(kv_cache_desc_t desc, int64_t batch, int64_t kv_len, int64_t max_pages,
                            const int32_t* page_table, const int32_t* kv_lens, int64_t n_pages, const void* k_pages,
                            const void* v_pages, const uint8_t* k_scales, const uint8_t* v_scales, void* k, void* v,
                            void* stream) {
    if (!desc) return fail(CONV_ERR_INVALID_ARG, "null descriptor");
    const kv_cache_params_t& p = desc->p;
    if (batch < 0 || kv_len < 0 || max_pages < 0 || n_pages < 0)
        return fail(CONV_ERR_INVALID_ARG, "negative batch, kv_len, max_pages or n_pages");
    if (batch > kMaxLen || kv_len > kMaxLen || max_pages > kMaxLen || max_pages * p.page_size > kMaxLen ||
        n_pages > kMaxRows || n_pages * p.page_size > kMaxRows)
        return fail(CONV_ERR_INVALID_ARG, "batch, kv_len or max_pages * page_size beyond 2^30, or n_pages * page_size beyond 2^31");
    if (batch == 0 || kv_len == 0 || max_pages == 0) return ok();
    conv_status_t st = check_kv(p, n_pages, k_pages, v_pages, k_scales, v_scales, k, v);
    if (st != CONV_OK) return st;
    if (!page_table) return fail(CONV_ERR_INVALID_ARG, "null page_table");
    if (misaligned(page_table, 4) || misaligned(kv_lens, 4))
        return fail(CONV_ERR_INVALID_ARG, "page_table or kv_lens is not aligned to 4 bytes");
    const int64_t h = p.heads_kv, hd = p.head_dim, es = elem_size(p.dtype);
    if (too_far(kv_len, p.k_stride) || too_far(kv_len, p.v_stride) || too_far(batch, max_pages))
        return fail(CONV_ERR_UNSUPPORTED, "a tensor reaches beyond 2^44 elements");
    const int64_t kb = p.k_batch_stride ? p.k_batch_stride : kv_len * p.k_stride;
    const int64_t vb = p.v_batch_stride ? p.v_batch_stride : kv_len * p.v_stride;
    if (too_far(batch, kb) || too_far(batch, vb))
        return fail(CONV_ERR_UNSUPPORTED, "a tensor reaches beyond 2^44 elements");
    const int64_t ks[3] = {kb, p.k_stride, hd}, vs[3] = {vb, p.v_stride, hd};
    if (!nested(ks, batch, kv_len, h, hd) || !nested(vs, batch, kv_len, h, hd))
        return fail(CONV_ERR_ALIAS, "rows of k or v share memory");
    const KvGrids in = kv_grids(p, n_pages, k_pages, v_pages, k_scales, v_scales);
    // Row by row where all rows are equally far apart, else sequence by
    // sequence, or from the first to the last element.
    const auto grid = [&](const void* q, const int64_t* s) {
        Grid g{(uintptr_t)q, {s[0] * es, s[1] * es, 0}, {batch, kv_len, 1}, h * hd * es, {}};
        const int64_t inner = (kv_len - 1) * s[1] + h * hd;
        g.view = batch == 1 || s[0] == kv_len * s[1] ? rows_view(q, batch * kv_len, s[1], h * hd, es)
                 : s[0] >= inner                     ? View{(uintptr_t)q, batch, s[0] * es, inner * es}
                                                     : View{(uintptr_t)q, 1, 0, ((batch - 1) * s[0] + inner) * es};
        return g;
    };
    const Grid out[2] = {grid(k, ks), grid(v, vs)};
    const View small[2] = {flat_view(page_table, 4 * batch * max_pages), flat_view(kv_lens, 4 * batch)};
    if (grids_overlap(out[0], out[1])) return fail(CONV_ERR_ALIAS, "k overlaps v");
    for (const Grid& o : out) {
        for (int i = 0; i < in.n; ++i)
            if (views_overlap(o.view, in.pages[i].view)) return fail(CONV_ERR_ALIAS, "k or v overlaps the pages or their scales");
        for (const View& s : small)
            if (views_overlap(o.view, s)) return fail(CONV_ERR_ALIAS, "k or v overlaps page_table or kv_lens");
    }
    if (n_pages == 0) return ok();   // no page to read
    KvArgs a = kv_args(p, n_pages, k_pages, v_pages, k_scales, v_scales, k, v);
    a.page_table = page_table; a.kv_lens = kv_lens;
    a.k_bs = kb; a.v_bs = vb;
    a.batch = (int32_t)batch; a.max_pages = (int32_t)max_pages;
    a.kv_len = (int32_t)(kv_len < max_pages * p.page_size ? kv_len : max_pages * p.page_size);
    const bool e4m3 = p.cache_dtype == KV_CACHE_E4M3;
    return hip_status(launch_kv_load(p.dtype, e4m3, kv_vec(p, a), a, (hipStream_t)stream), "kv_cache_load");
}

// ---------------------------------------------------- paged attention ----

void paged_attention_params_init(paged_attention_params_t* p) {
    if (!p) return;
    memset(p, 0, sizeof(*p));
    p->scale = NAN;
}

conv_status_t paged_attention_desc_create(const paged_attention_params_t* pp, paged_attention_desc_t* out) {
    if (!pp || !out) return fail(CONV_ERR_INVALID_ARG, "null params or out");
    *out = nullptr;
    paged_attention_params_t p = *pp;
    conv_status_t st = check_cache_dtype(p.dtype, p.cache_dtype);
    if (st != CONV_OK) return st;
    if (p.heads_q < 1 || p.heads_kv < 1 || p.heads_q > 1 << 16)
        return fail(CONV_ERR_INVALID_ARG, "heads_q = %d, heads_kv = %d must be 1 .. 2^16", p.heads_q, p.heads_kv);
    if (p.heads_q % p.heads_kv)
        return fail(CONV_ERR_INCOMPATIBLE_SHAPES, "heads_kv = %d does not divide heads_q = %d", p.heads_kv, p.heads_q);
    if (p.head_dim < 1) return fail(CONV_ERR_INVALID_ARG, "head_dim = %d", p.head_dim);
    // Elements of 16 bytes of q, and of the pages.
    const int64_t chunk = 16 / elem_size(p.dtype), unit = 16 / cache_elem_size(p.cache_dtype);
    if (p.head_dim > 256 || p.head_dim % unit)
        return fail(CONV_ERR_UNSUPPORTED, "head_dim = %d is not a multiple of %d up to 256", p.head_dim, (int)unit);
    if (p.page_size < 1 || p.page_size > 1 << 16)
        return fail(CONV_ERR_INVALID_ARG, "page_size = %d must be 1 .. 2^16", p.page_size);
    if (p.window < 0 || p.sinks < 0) return fail(CONV_ERR_INVALID_ARG, "window = %d, sinks = %d", p.window, p.sinks);
    if (!(p.softcap >= 0) || !std::isfinite(p.softcap)) return fail(CONV_ERR_INVALID_ARG, "softcap must be finite and >= 0");
    if (std::isnan(p.scale)) p.scale = 1.0f / std::sqrt((float)p.head_dim);
    if (!std::isfinite(p.scale)) return fail(CONV_ERR_INVALID_ARG, "non-finite scale");
    const int64_t d = p.head_dim;
    if ((st = resolve_stride(p.q_stride, p.heads_q * d, "q_stride")) != CONV_OK) return st;
    if ((st = resolve_stride(p.out_stride, p.heads_q * d, "out_stride")) != CONV_OK) return st;
    if ((st = resolve_page_strides(p.k_page_strides, p.page_size, p.heads_kv, d, "k_page_strides")) != CONV_OK ||
        (st = resolve_page_strides(p.v_page_strides, p.page_size, p.heads_kv, d, "v_page_strides")) != CONV_OK ||
        (st = resolve_page_strides(p.scale_strides, p.page_size, p.heads_kv, 1, "scale_strides")) != CONV_OK)
        return st;
    if (p.q_stride % chunk || p.out_stride % chunk)
        return fail(CONV_ERR_UNSUPPORTED, "a token stride is not a multiple of 16 bytes");
    for (int i = 0; i < 3; ++i)
        if (p.k_page_strides[i] % unit || p.v_page_strides[i] % unit)
            return fail(CONV_ERR_UNSUPPORTED, "a page stride is not a multiple of %d elements", (int)unit);
    return make_desc(paged_attention_desc{p}, out);
}

void paged_attention_desc_destroy(paged_attention_desc_t d) { delete d; }

conv_status_t paged_attention_workspace_bytes(paged_attention_desc_t d, int64_t tokens, int64_t batch,
                                              int64_t max_pages, int64_t* bytes) {
    if (!d || !bytes) return fail(CONV_ERR_INVALID_ARG, "null descriptor or bytes");
    const conv_status_t st = check_paged_sizes(d->p, tokens, batch, max_pages);
    if (st != CONV_OK) return st;
    *bytes = 0;
    if (tokens == 0 || batch == 0) return ok();
    const PagedArgs a = paged_args(d->p, tokens, batch, max_pages, 0);
    *bytes = plan_paged_attention(d->p.dtype, d->p.cache_dtype == KV_CACHE_E4M3, a).ws_bytes;
    return ok();
}

conv_status_t paged_attention_forward(paged_attention_desc_t d, int64_t tokens, int64_t batch, int64_t max_pages,
                                      const void* q, const int32_t* q_offsets, const int32_t* kv_lens,
                                      const int32_t* page_table, int64_t n_pages, const void* k_pages,
                                      const void* v_pages, const uint8_t* k_scales, const uint8_t* v_scales, void* out,
                                      void* workspace, int64_t workspace_bytes, void* stream) {
    if (!d) return fail(CONV_ERR_INVALID_ARG, "null descriptor");
    const paged_attention_params_t& p = d->p;
    const conv_status_t st = check_paged_sizes(p, tokens, batch, max_pages);
    if (st != CONV_OK) return st;
    if (n_pages < 0 || n_pages > kMaxRows || n_pages * p.page_size > kMaxRows)
        return fail(CONV_ERR_INVALID_ARG, "n_pages = %lld", (long long)n_pages);
    if (tokens == 0 || batch == 0) return ok();
    const bool e4m3 = p.cache_dtype == KV_CACHE_E4M3;
    if (!q || !out || !q_offsets || !kv_lens) return fail(CONV_ERR_INVALID_ARG, "null q, out, q_offsets or kv_lens");
    if (max_pages > 0 && !page_table) return fail(CONV_ERR_INVALID_ARG, "null page_table");
    if (n_pages > 0 && (!k_pages || !v_pages || (e4m3 && (!k_scales || !v_scales))))
        return fail(CONV_ERR_INVALID_ARG, "null pages, or scales of an E4M3 cache");
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned16(k_pages) || !aligned16(v_pages))
        return fail(CONV_ERR_INVALID_ARG, "a tensor or the workspace is not aligned to 16 bytes");
    if (misaligned(q_offsets, 4) || misaligned(kv_lens, 4) || misaligned(page_table, 4))
        return fail(CONV_ERR_INVALID_ARG, "q_offsets, kv_lens or page_table is not aligned to 4 bytes");
    const int64_t ps = p.page_size, h = p.heads_kv, hd = p.head_dim, es = elem_size(p.dtype), cs = cache_elem_size(p.cache_dtype);
    if (n_pages > 0) {
        const auto far = [&](const int64_t* s, int64_t len, int64_t per) {
            return pages_too_far(s, n_pages, ps, h) || pages_span(s, n_pages, ps, h, len) / per >= (int64_t)1 << 32;
        };
        if (far(p.k_page_strides, hd, 16 / cs) || far(p.v_page_strides, hd, 16 / cs) || (e4m3 && far(p.scale_strides, 1, 1)))
            return fail(CONV_ERR_UNSUPPORTED, "pages reach beyond 2^36 bytes, or their scales beyond 2^32");
    }
    PagedArgs a = paged_args(p, tokens, batch, max_pages, n_pages);
    const PagedPlan plan = plan_paged_attention(p.dtype, e4m3, a);
    if (plan.ws_bytes > 0 && (!workspace || workspace_bytes < plan.ws_bytes))
        return fail(CONV_ERR_INVALID_ARG, "a workspace of %lld bytes is needed", (long long)plan.ws_bytes);
    if (n_pages == 0) a.max_pages = 0;   // no key to see
    const View wv = flat_view(workspace, plan.ws_bytes);
    const View ov = rows_view(out, tokens, p.out_stride, p.heads_q * hd, es);
    const View in[8] = {rows_view(q, tokens, p.q_stride, p.heads_q * hd, es),
                        flat_view(q_offsets, 4 * (batch + 1)),
                        flat_view(kv_lens, 4 * batch),
                        flat_view(page_table, 4 * batch * max_pages),
                        pages_view(k_pages, p.k_page_strides, n_pages, ps, h, hd, cs),
                        pages_view(v_pages, p.v_page_strides, n_pages, ps, h, hd, cs),
                        pages_view(e4m3 ? k_scales : nullptr, p.scale_strides, n_pages, ps, h, 1, 1),
                        pages_view(e4m3 ? v_scales : nullptr, p.scale_strides, n_pages, ps, h, 1, 1)};
    if (views_overlap(ov, wv)) return fail(CONV_ERR_ALIAS, "out overlaps the workspace");
    for (const View& iv : in)
        if (views_overlap(ov, iv) || views_overlap(wv, iv))
            return fail(CONV_ERR_ALIAS, "out or the workspace overlaps an input");
    a.q = q; a.out = out; a.q_offsets = q_offsets; a.kv_lens = kv_lens; a.page_table = page_table;
    a.k = k_pages; a.v = v_pages;
    a.ks = e4m3 ? k_scales : nullptr;
    a.vs = e4m3 ? v_scales : nullptr;
    a.ws = plan.ws_bytes > 0 ? workspace : nullptr;
    a.tiles = plan.tiles; a.parts = plan.parts; a.long_blocks = plan.long_blocks;
    a.group_heads = plan.group_heads; a.head_groups = a.heads_kv / plan.group_heads;
    return hip_status(launch_paged_attention(p.dtype, e4m3, plan, a, (hipStream_t)stream), "paged_attention");
}

// --------------------------------------------------------- block norm ----

void block_norm_params_init(block_norm_params_t* p) {
    if (!p) return;
    memset(p, 0, sizeof(*p));
    p->residual_scale = p->block_scale = 1.0f;
    p->eps = 1e-6f;
}

conv_status_t block_norm_desc_create(const block_norm_params_t* pp, block_norm_desc_t* out) {
    if (!pp || !out) return fail(CONV_ERR_INVALID_ARG, "null params or out");
    *out = nullptr;
    block_norm_params_t p = *pp;
    conv_status_t st = check_dtype(p.dtype);
    if (st != CONV_OK) return st;
    if (p.width < 1) return fail(CONV_ERR_INVALID_ARG, "width = %d", p.width);
    if (p.width > NORM_MAX_WIDTH) return fail(CONV_ERR_UNSUPPORTED, "width = %d beyond %d", p.width, NORM_MAX_WIDTH);
    for (int32_t kind : {p.post_norm, p.pre_norm})
        if (kind < BLOCK_NORM_NONE || kind > BLOCK_NORM_LAYER) return fail(CONV_ERR_INVALID_ARG, "unknown norm %d", kind);
    if (!is_bool(p.has_post_beta) || !is_bool(p.has_pre_beta) || !is_bool(p.has_gate))
        return fail(CONV_ERR_INVALID_ARG, "has_post_beta, has_pre_beta and has_gate are 0 or 1");
    if ((p.has_post_beta && p.post_norm == BLOCK_NORM_NONE) || (p.has_pre_beta && p.pre_norm == BLOCK_NORM_NONE))
        return fail(CONV_ERR_INVALID_ARG, "a beta without its norm");
    if (p.gate_rows < 0) return fail(CONV_ERR_INVALID_ARG, "gate_rows = %d", p.gate_rows);
    if (!std::isfinite(p.residual_scale) || !std::isfinite(p.block_scale))
        return fail(CONV_ERR_INVALID_ARG, "non-finite residual_scale or block_scale");
    if (!(p.eps >= 0) || !std::isfinite(p.eps)) return fail(CONV_ERR_INVALID_ARG, "eps must be finite and >= 0");
    const struct { int64_t& s; const char* what; } strides[5] = {{p.y_stride, "y_stride"}, {p.x_stride, "x_stride"},
        {p.residual_stride, "residual_stride"}, {p.out_stride, "out_stride"}, {p.gate_stride, "gate_stride"}};
    for (const auto& s : strides)
        if ((st = resolve_stride(s.s, p.width, s.what)) != CONV_OK) return st;
    return make_desc(block_norm_desc{p}, out);
}

void block_norm_desc_destroy(block_norm_desc_t d) { delete d; }

conv_status_t block_norm_forward(block_norm_desc_t d, int64_t rows, const void* y, const void* x, const void* gate,
                                 const float* post_gamma, const float* post_beta, const float* pre_gamma,
                                 const float* pre_beta, void* residual, void* out, void* stream) {
    if (!d) return fail(CONV_ERR_INVALID_ARG, "null descriptor");
    const block_norm_params_t& p = d->p;
    if (rows < 0 || rows > kMaxRows) return fail(CONV_ERR_INVALID_ARG, "rows = %lld", (long long)rows);
    if (rows == 0) return ok();
    const bool post = p.post_norm != BLOCK_NORM_NONE, pre = p.pre_norm != BLOCK_NORM_NONE;
    if (!p.has_gate) gate = nullptr;
    if (!post) post_gamma = nullptr;
    if (!p.has_post_beta) post_beta = nullptr;
    if (!pre) pre_gamma = nullptr;
    if (!p.has_pre_beta) pre_beta = nullptr;
    if (!pre) out = nullptr;
    if (!y || !x || !residual || (pre && !out)) return fail(CONV_ERR_INVALID_ARG, "null y, x, residual or out");
    if ((p.has_gate && !gate) || (post && !post_gamma) || (pre && !pre_gamma) || (p.has_post_beta && !post_beta) ||
        (p.has_pre_beta && !pre_beta))
        return fail(CONV_ERR_INVALID_ARG, "null gate, gamma or beta");
    const int64_t es = elem_size(p.dtype), w = p.width;
    for (const void* t : {y, x, gate, (const void*)residual, (const void*)out})
        if (misaligned(t, es)) return fail(CONV_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
    for (const float* t : {post_gamma, post_beta, pre_gamma, pre_beta})
        if (misaligned(t, 4)) return fail(CONV_ERR_INVALID_ARG, "a gamma or beta is not aligned to 4 bytes");
    const int64_t gates = p.gate_rows ? (rows + p.gate_rows - 1) / p.gate_rows : 1;
    if (too_far(rows, p.y_stride) || too_far(rows, p.x_stride) || too_far(rows, p.residual_stride) ||
        (pre && too_far(rows, p.out_stride)) || (gate && too_far(gates, p.gate_stride)))
        return fail(CONV_ERR_UNSUPPORTED, "a tensor reaches beyond 2^44 elements");
    const View rv = rows_view(residual, rows, p.residual_stride, w, es), ov = rows_view(out, pre ? rows : 0, p.out_stride, w, es);
    const View yv = rows_view(y, rows, p.y_stride, w, es), xv = rows_view(x, rows, p.x_stride, w, es);
    if (views_overlap(rv, ov)) return fail(CONV_ERR_ALIAS, "residual overlaps out");
    const auto same = [](const void* a, int64_t sa, const void* b, int64_t sb) { return a == b && sa == sb; };
    if ((!same(residual, p.residual_stride, x, p.x_stride) && views_overlap(rv, xv)) ||
        (!same(residual, p.residual_stride, y, p.y_stride) && views_overlap(rv, yv)))
        return fail(CONV_ERR_ALIAS, "residual overlaps x or y without being it");
    if ((!same(out, p.out_stride, y, p.y_stride) && views_overlap(ov, yv)) || views_overlap(ov, xv))
        return fail(CONV_ERR_ALIAS, "out overlaps x, or y without being it");
    const View small[5] = {rows_view(gate, gate ? gates : 0, p.gate_stride, w, es), flat_view(post_gamma, 4 * w),
                           flat_view(post_beta, 4 * w), flat_view(pre_gamma, 4 * w), flat_view(pre_beta, 4 * w)};
    for (const View& s : small)
        if (views_overlap(s, rv) || views_overlap(s, ov)) return fail(CONV_ERR_ALIAS, "an output overlaps the gate, a gamma or a beta");
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.y = y; a.x = x; a.gate = gate; a.residual = residual; a.out = out;
    a.post_gamma = post_gamma; a.post_beta = post_beta; a.pre_gamma = pre_gamma; a.pre_beta = pre_beta;
    a.y_s = p.y_stride; a.x_s = p.x_stride; a.r_s = p.residual_stride; a.o_s = p.out_stride; a.g_s = p.gate_stride;
    a.rows = (int32_t)rows; a.width = p.width; a.post = p.post_norm; a.pre = p.pre_norm;
    if (p.gate_rows) a.gate_rows = make_divu32((uint32_t)p.gate_rows);
    a.residual_scale = p.residual_scale; a.block_scale = p.block_scale; a.eps = p.eps;
    const int64_t chunk = 16 / es;
    const auto at16 = [&](const void* t, int64_t stride) { return !t || (aligned16(t) && stride % chunk == 0); };
    const bool vec = p.width % 8 == 0 && at16(y, p.y_stride) && at16(x, p.x_stride) && at16(gate, p.gate_stride) &&
                     at16(residual, p.residual_stride) && at16(out, p.out_stride) && aligned16(post_gamma) &&
                     aligned16(post_beta) && aligned16(pre_gamma) && aligned16(pre_beta);
    return hip_status(launch_block_norm(p.dtype, vec, a, (hipStream_t)stream), "block_norm");
}

}  // extern "C"
