// Softmax attention of new tokens over the pages of a cache.
#include "attention_common.h"
#include "decoder_internal.h"
#include "e4m3.h"

namespace conv2d {

namespace {

// A wave a (new token, head): a key at a time, a lane every 64th element.
template <typename T, bool E4>
__global__ __launch_bounds__(256) void paged_any(PagedArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t all = (int64_t)a.tokens * a.heads_q;
    for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < all; w += (int64_t)gridDim.x * 4) {
        const int t = (int)(w / a.heads_q), hq = (int)(w - (int64_t)t * a.heads_q), hk = hq / a.group;
        // The last sequence that starts at or before t.
        int b = 0, end = a.batch + 1;
        while (b < end) {
            const int mid = (b + end) >> 1;
            if (a.q_offsets[mid] <= t)
                b = mid + 1;
            else
                end = mid;
        }
        --b;
        if (b < 0 || b >= a.batch) continue;
        const int first = max(a.q_offsets[b], 0), nq = min(a.q_offsets[b + 1], a.tokens) - first;
        const int nk = min(max(a.kv_lens[b], 0), a.max_pages * (int)a.page_size.d);
        if (t - first >= nq) continue;
        const int p = nk - nq + (t - first);
        float q[4], o[4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = lane + 64 * i < a.d ? to_f32(((const T*)a.q)[t * a.q_s + (int64_t)hq * a.d + lane + 64 * i]) : 0.0f;
        float top = -INFINITY, total = 0.0f;
        for (int j = 0; j <= p; ++j) {
            if (a.window && p - j >= a.window && j >= a.sinks) {
                j = p - a.window;
                continue;
            }
            const uint32_t n = divu((uint32_t)j, a.page_size), token = (uint32_t)j - n * a.page_size.d;
            const int page = a.page_table[(int64_t)b * a.max_pages + n];
            if (page < 0 || page >= a.n_pages) continue;
            const auto row = [&](const void* pages, const PageStrides& s, const uint8_t* scales, float (&x)[4]) {
                const int64_t at = page * s.page + (int64_t)token * s.token + hk * s.head;
                float scale = 1.0f;
                if (E4) scale = scale_value(scales[page * a.s_s.page + (int64_t)token * a.s_s.token + hk * a.s_s.head]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = lane + 64 * i;
                    x[i] = 0.0f;
                    if (e < a.d) x[i] = E4 ? decode1(((const uint8_t*)pages)[at + e], scale) : to_f32(((const T*)pages)[at + e]);
                }
            };
            float x[4], dot[1] = {0.0f};
            row(a.k, a.k_s, a.ks, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) dot[0] += q[i] * x[i];
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) dot[0] += __shfl_xor(dot[0], m, 64);
            ScoreP sp;
            sp.cap = a.softcap;
            sp.scale = a.softcap > 0.0f ? cap_scale(a.scale, a.softcap) : a.scale * kLog2e;
            scores<T>(sp, dot);
            const float now = fmaxf(top, dot[0]), fade = __builtin_amdgcn_exp2f(top - (now == -INFINITY ? 0.0f : now));
            const float weight = __builtin_amdgcn_exp2f(dot[0] - (now == -INFINITY ? 0.0f : now));
            top = now;
            total = total * fade + weight;
            row(a.v, a.v_s, a.vs, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = o[i] * fade + weight * x[i];
        }
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 64 * i < a.d) ((T*)a.out)[t * a.o_s + (int64_t)hq * a.d + lane + 64 * i] = from_f32<T>(o[i] * inv);
    }
}

template <typename T, bool E4>
hipError_t run(const PagedArgs& a, hipStream_t s) {
    const int64_t most = (int64_t)device_cu_count() * 64, n = ((int64_t)a.tokens * a.heads_q + 3) / 4;
    paged_any<T, E4><<<dim3((uint32_t)(n < most ? n : most)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_attention(int32_t dtype, bool e4m3, const PagedArgs& a, hipStream_t s) {
    if (dtype == CONV_DTYPE_F32) return e4m3 ? run<float, true>(a, s) : run<float, false>(a, s);
    return e4m3 ? run<bf16, true>(a, s) : run<bf16, false>(a, s);
}

}  // namespace conv2d
