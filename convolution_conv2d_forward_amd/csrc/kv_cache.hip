// Keys and values to the pages of a cache, and back.
#include "decoder_internal.h"
#include "e4m3.h"

namespace conv2d {

namespace {

// A slot's place in pages of the strides s.
__device__ __forceinline__ int64_t slot_at(const PageStrides& s, uint32_t page, uint32_t token, int head) {
    return (int64_t)page * s.page + (int64_t)token * s.token + (int64_t)head * s.head;
}

// Any head size, stride and alignment: a wave a (token, head) of the keys or
// the values, a lane an element at a time.
template <typename T, bool E4>
__global__ __launch_bounds__(256) void kv_store_any(KvArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t rows = (int64_t)a.tokens * a.heads * 2;
    for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < rows; w += (int64_t)gridDim.x * 4) {
        const bool is_v = w & 1;
        const int64_t t = (w >> 1) / a.heads;
        const int h = (int)((w >> 1) - t * a.heads);
        const int slot = a.slots[t];
        if (slot < 0 || slot >= a.n_pages * (int)a.page_size.d) continue;
        const uint32_t page = divu((uint32_t)slot, a.page_size), token = (uint32_t)slot - page * a.page_size.d;
        const T* x = (const T*)(is_v ? a.v : a.k) + t * (is_v ? a.v_s : a.k_s) + (int64_t)h * a.d;
        const int64_t at = slot_at(is_v ? a.vs : a.ks, page, token, h);
        void* pages = (void*)(is_v ? a.v_pages : a.k_pages);
        if constexpr (E4) {
            float top = 0.0f;
            for (int e = lane; e < a.d; e += 64) top = fmaxf(top, finite_size(to_f32(x[e])));
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
            const uint32_t s = scale_of(top);
            for (int e = lane; e < a.d; e += 64)
                ((uint8_t*)pages)[at + e] = (uint8_t)encode2(to_f32(x[e]), 0.0f, scale_inverse(s), 0, false);
            if (lane == 0) ((uint8_t*)(is_v ? a.v_scales : a.k_scales))[slot_at(a.ss, page, token, h)] = (uint8_t)s;
        } else {
            for (int e = lane; e < a.d; e += 64) ((T*)pages)[at + e] = x[e];
        }
    }
}

template <typename T, bool E4>
__global__ __launch_bounds__(256) void kv_load_any(KvArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t rows = (int64_t)a.batch * a.kv_len * a.heads * 2;
    for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < rows; w += (int64_t)gridDim.x * 4) {
        const bool is_v = w & 1;
        const int64_t token_i = (w >> 1) / a.heads;
        const int h = (int)((w >> 1) - token_i * a.heads);
        const int b = (int)(token_i / a.kv_len), i = (int)(token_i - (int64_t)b * a.kv_len);
        if (a.kv_lens && i >= a.kv_lens[b]) continue;
        const uint32_t n = divu((uint32_t)i, a.page_size), token = (uint32_t)i - n * a.page_size.d;
        const int page = a.page_table[(int64_t)b * a.max_pages + n];
        if (page < 0 || page >= a.n_pages) continue;
        T* x = (T*)(is_v ? a.v : a.k) + b * (is_v ? a.v_bs : a.k_bs) + i * (is_v ? a.v_s : a.k_s) + (int64_t)h * a.d;
        const void* pages = is_v ? a.v_pages : a.k_pages;
        const int64_t at = slot_at(is_v ? a.vs : a.ks, page, token, h);
        if constexpr (E4) {
            const float s = scale_value((is_v ? a.v_scales : a.k_scales)[slot_at(a.ss, page, token, h)]);
            for (int e = lane; e < a.d; e += 64) x[e] = from_f32<T>(decode1(((const uint8_t*)pages)[at + e], s));
        } else {
            for (int e = lane; e < a.d; e += 64) x[e] = ((const T*)pages)[at + e];
        }
    }
}

// Workgroups for so many waves: enough to fill the chip, each with several.
uint32_t grid_of(int64_t waves) {
    const int64_t most = (int64_t)device_cu_count() * 64, n = (waves + 3) / 4;
    return (uint32_t)(n < most ? n : most);
}

template <typename T, bool E4>
hipError_t store(bool vec, const KvArgs& a, hipStream_t s) {
    kv_store_any<T, E4><<<dim3(grid_of((int64_t)a.tokens * a.heads * 2)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool E4>
hipError_t load(bool vec, const KvArgs& a, hipStream_t s) {
    kv_load_any<T, E4><<<dim3(grid_of((int64_t)a.batch * a.kv_len * a.heads * 2)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_store(int32_t dtype, bool e4m3, bool vec, const KvArgs& a, hipStream_t s) {
    if (dtype == CONV_DTYPE_F32) return e4m3 ? store<float, true>(vec, a, s) : store<float, false>(vec, a, s);
    return e4m3 ? store<bf16, true>(vec, a, s) : store<bf16, false>(vec, a, s);
}

hipError_t launch_kv_load(int32_t dtype, bool e4m3, bool vec, const KvArgs& a, hipStream_t s) {
    if (dtype == CONV_DTYPE_F32) return e4m3 ? load<float, true>(vec, a, s) : load<float, false>(vec, a, s);
    return e4m3 ? load<bf16, true>(vec, a, s) : load<bf16, false>(vec, a, s);
}

}  // namespace conv2d
