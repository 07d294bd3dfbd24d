// Keys and values to the pages of a cache, and back.
#include <type_traits>

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

// 8 elements of T, moved as they are.
template <typename T>
using Raw8 = uint32_t __attribute__((ext_vector_type(2 * sizeof(T)), aligned(16)));

// Rows of 8 elements a lane: a wave takes a token's rows (keys of all heads,
// then values), or UN times as many of them as fit in its lanes, LPH lanes
// each, all loads in flight at once; blockIdx.y says which.  Bound by bytes:
// 16384 tokens of 8 heads of 128 bf16 to codes take 19.3 us (5.2 TB/s), 26446
// back 25.9 (6.3).  Stores pass by the L2s: through them 22.4 and 40.3.  UN = 4:
// 19.9 and 26.9, 1: 27.7 and 51 (through the L2s).
constexpr int UN = 2;

// This lane's i-th row: whether there is one, its head, and whether it is a
// value's.
template <int LPH>
__device__ __forceinline__ bool row_of(const KvArgs& a, int i, int& h, bool& is_v) {
    const int lane = threadIdx.x & 63, row = ((int)blockIdx.y * UN + i) * (64 / LPH) + lane / LPH;
    is_v = row >= a.heads;
    h = is_v ? row - a.heads : row;
    return row < 2 * a.heads && (lane & (LPH - 1)) * 8 < a.d;
}

template <typename T, bool E4, int LPH>
__global__ __launch_bounds__(256) void kv_store_vec(KvArgs a) {
    const int lane = threadIdx.x & 63, e = (lane & (LPH - 1)) * 8;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.tokens; t += (int64_t)gridDim.x * 4) {
        const int slot = a.slots[t];
        if (slot < 0 || slot >= a.n_pages * (int)a.page_size.d) continue;
        const uint32_t page = divu((uint32_t)slot, a.page_size), token = (uint32_t)slot - page * a.page_size.d;
        typedef T V __attribute__((ext_vector_type(8)));
        Raw8<T> x[UN];
        int h[UN];
        bool is_v[UN], on[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            on[i] = row_of<LPH>(a, i, h[i], is_v[i]);
            const T* p = (const T*)(is_v[i] ? a.v : a.k) + t * (is_v[i] ? a.v_s : a.k_s) + (int64_t)h[i] * a.d + e;
            x[i] = 0;
            if (on[i]) x[i] = *(const Raw8<T>*)p;
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            void* pages = (void*)(is_v[i] ? a.v_pages : a.k_pages);
            const int64_t at = slot_at(is_v[i] ? a.vs : a.ks, page, token, h[i]) + e;
            if constexpr (E4) {
                const f32x8 v = __builtin_convertvector(__builtin_bit_cast(V, x[i]), f32x8);
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_size(v[j]));
#pragma unroll
                for (int m = 1; m < LPH; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
                const uint32_t s = scale_of(top);
                const float inverse = scale_inverse(s);
                const u32x2 codes{encode4(f32x4{v[0], v[1], v[2], v[3]}, inverse), encode4(f32x4{v[4], v[5], v[6], v[7]}, inverse)};
                if (on[i]) __builtin_nontemporal_store(codes, (u32x2*)((uint8_t*)pages + at));
                if (on[i] && e == 0)
                    ((uint8_t*)(is_v[i] ? a.v_scales : a.k_scales))[slot_at(a.ss, page, token, h[i])] = (uint8_t)s;
            } else if (on[i]) {
                __builtin_nontemporal_store(x[i], (Raw8<T>*)((T*)pages + at));
            }
        }
    }
}

template <typename T, bool E4, int LPH>
__global__ __launch_bounds__(256) void kv_load_vec(KvArgs a) {
    const int lane = threadIdx.x & 63, e = (lane & (LPH - 1)) * 8;
    for (int b = blockIdx.z; b < a.batch; b += gridDim.z) {
        const int len = a.kv_lens ? min(a.kv_lens[b], a.kv_len) : a.kv_len;
        for (int t = (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6); t < len; t += (int)gridDim.x * 4) {
            const uint32_t n = divu((uint32_t)t, a.page_size), token = (uint32_t)t - n * a.page_size.d;
            const int page = a.page_table[(int64_t)b * a.max_pages + n];
            if (page < 0 || page >= a.n_pages) continue;
            typedef typename std::conditional<E4, u32x2, Raw8<T>>::type X;
            X x[UN];
            uint32_t s[UN];
            int h[UN];
            bool is_v[UN], on[UN];
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                on[i] = row_of<LPH>(a, i, h[i], is_v[i]);
                const char* pages = (const char*)(is_v[i] ? a.v_pages : a.k_pages);
                const int64_t at = slot_at(is_v[i] ? a.vs : a.ks, page, token, h[i]) + e;
                if (!on[i]) continue;
                x[i] = *(const X*)(pages + at * (E4 ? 1 : (int)sizeof(T)));
                if (E4) s[i] = (is_v[i] ? a.v_scales : a.k_scales)[slot_at(a.ss, page, token, h[i])];
            }
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                if (!on[i]) continue;
                T* p = (T*)(is_v[i] ? a.v : a.k) + b * (is_v[i] ? a.v_bs : a.k_bs) + t * (is_v[i] ? a.v_s : a.k_s) +
                       (int64_t)h[i] * a.d + e;
                if constexpr (!E4) {
                    __builtin_nontemporal_store(x[i], (Raw8<T>*)p);
                } else if constexpr (sizeof(T) == 2) {
                    __builtin_nontemporal_store(decode(x[i], scale_value(s[i]), T{}), (u32x4*)p);
                } else {
                    __builtin_nontemporal_store(decode(x[i][0], scale_value(s[i]), T{}), (u32x4*)p);
                    __builtin_nontemporal_store(decode(x[i][1], scale_value(s[i]), T{}), (u32x4*)p + 1);
                }
            }
        }
    }
}

// A grid's workgroups, whatever its dimensions, at most.
constexpr int64_t kMostGrid = (int64_t)1 << 22;

// Workgroups for so many waves: as many as run at once, or fewer.
uint32_t grid_of(int64_t waves) {
    const int64_t most = (int64_t)device_cu_count() * 8, n = (waves + 3) / 4;
    return (uint32_t)(n < most ? n : most);
}

template <typename T, bool E4, int LPH>
hipError_t store_vec(const KvArgs& a, hipStream_t s) {
    const int parts = (2 * a.heads + 64 / LPH * UN - 1) / (64 / LPH * UN);
    const uint32_t x = grid_of(a.tokens), most = (uint32_t)(kMostGrid / parts);
    kv_store_vec<T, E4, LPH><<<dim3(x < most ? x : most, (uint32_t)parts), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool E4>
hipError_t store(bool vec, const KvArgs& a, hipStream_t s) {
    if (vec) {
        if (a.d <= 32) return store_vec<T, E4, 4>(a, s);
        if (a.d <= 64) return store_vec<T, E4, 8>(a, s);
        if (a.d <= 128) return store_vec<T, E4, 16>(a, s);
        return store_vec<T, E4, 32>(a, s);
    }
    kv_store_any<T, E4><<<dim3(grid_of((int64_t)a.tokens * a.heads * 2)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool E4, int LPH>
hipError_t load_vec(const KvArgs& a, hipStream_t s) {
    const int parts = (2 * a.heads + 64 / LPH * UN - 1) / (64 / LPH * UN);
    const uint32_t all = grid_of(a.kv_len), each = (uint32_t)(kMostGrid / parts), x = all < each ? all : each;
    const uint32_t most = each / x, z = (uint32_t)a.batch < most ? (uint32_t)a.batch : most;
    kv_load_vec<T, E4, LPH><<<dim3(x, (uint32_t)parts, z < 65535 ? z : 65535), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool E4>
hipError_t load(bool vec, const KvArgs& a, hipStream_t s) {
    if (vec) {
        if (a.d <= 32) return load_vec<T, E4, 4>(a, s);
        if (a.d <= 64) return load_vec<T, E4, 8>(a, s);
        if (a.d <= 128) return load_vec<T, E4, 16>(a, s);
        return load_vec<T, E4, 32>(a, s);
    }
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
