// The norm behind a block, its gate and the scaled residual, and the norm
// before the next block, a row at a time.
#include <cfloat>

#include "decoder_internal.h"
#include "seq_common.h"

namespace conv2d {

namespace {

// A piece of a row, V elements: 8 at a 16-byte boundary, or one.
template <typename T, int V>
using Raw = T __attribute__((ext_vector_type(V), aligned(V == 8 ? 16 : sizeof(T))));
template <int V>
using Piece = float __attribute__((ext_vector_type(V)));

template <int V, typename T>
__device__ __forceinline__ Piece<V> values(Raw<T, V> r) {
    return __builtin_convertvector(r, Piece<V>);
}
template <int V, typename T>
__device__ __forceinline__ Raw<T, V> load(const T* p) {
    return *(const Raw<T, V>*)p;
}
template <int V, typename T>
__device__ __forceinline__ void store(T* p, Piece<V> v) {
    *(Raw<T, V>*)p = __builtin_convertvector(v, Raw<T, V>);
}

// Sum over a workgroup of NW waves, in all threads; `part` is read until each
// thread's next barrier.
template <int NW>
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    if (NW == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) s += part[i];
    return s;
}

// A row's squares may leave fp32's range where the row does not: then they are
// formed of the row times a power of two.  2^-80 brings the largest squares and sums
// of 32768 elements into range, 2^64 the least ones (which count only where no
// eps outweighs them).
constexpr float kDown = 0x1p-80f, kUp = 0x1p64f;
__device__ __forceinline__ bool out_of_range(float total, float eps) {
    return !(total < INFINITY) || (total < 0x1p-80f && eps < 0x1p-100f);
}
// What eps is next to the squares of a row times `scale`; above zero where it is,
// so that a row without spread stays 0.
__device__ __forceinline__ float scaled_eps(float eps, float scale) {
    return eps > 0.0f ? fmaxf(eps * scale * scale, FLT_MIN) : 0.0f;
}

// NW waves a row, whose pieces stay in registers, CP of them a thread: every
// element is read once and written once, and a row's mean is known before the
// squares around it are summed.  With up to 8 elements a thread a workgroup
// takes row after row, the next one's loads in flight, and keeps the gammas and
// betas: read for each row they are, from L2, twice the bytes of a bf16 row
// between two LAYER norms.  8192 rows of 4096 bf16 between two of them take 59
// us (4.5 TB/s), with a workgroup a row 65; with 24 waves on a CU instead of 16
// 68, with 16 waves a row 104.
template <typename T, int V, int NW, int CP>
__global__ __launch_bounds__(64 * NW) void block_norm(NormArgs a) {
    __shared__ float part[4][NW];
    const int tid = threadIdx.x;
    const float inv_n = 1.0f / (float)a.width;
    constexpr bool HOLD = V * CP <= 8;
    constexpr int HC = HOLD ? CP : 1;
    // A piece's first element, and whether it is in the row.
    int base = tid * V;
    const auto at = [&](int c) { return base + c * (64 * NW * V); };
    const auto on = [&](int c) { return at(c) < a.width; };
    const auto vector = [&](int which, bool is_beta, int c) {
        const float* v = which ? (is_beta ? a.pre_beta : a.pre_gamma) : (is_beta ? a.post_beta : a.post_gamma);
        return v && on(c) ? load<V>(v + at(c)) : Piece<V>(is_beta ? 0.0f : 1.0f);
    };
    Piece<V> kept[2][2][HC];   // gammas and betas of both norms
    if constexpr (HOLD) {
#pragma unroll
        for (int c = 0; c < CP; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) kept[i >> 1][i & 1][c] = vector(i >> 1, i & 1, c);
    }
    // The norm of the pieces in place.
    const auto norm = [&](Piece<V> (&p)[CP], int kind, int which) {
        float unit = 1.0f;
        if (kind == BLOCK_NORM_LAYER) {
            const auto sum = [&](float scale) {
                float s = 0.0f;
#pragma unroll
                for (int c = 0; c < CP; ++c)
#pragma unroll
                    for (int i = 0; i < V; ++i) s += scale * p[c][i];   // zeros past the row
                return block_sum<NW>(s, part[2 * which]);
            };
            // Halves: an element less the mean may be beyond fp32's range.
            unit = 0.5f;
            float half_mean = sum(1.0f) * inv_n * 0.5f;
            if (!(fabsf(half_mean) < INFINITY)) {
                if (NW > 1) __syncthreads();   // the sums have been read
                half_mean = sum(kDown) * inv_n * (0.5f / kDown);
            }
#pragma unroll
            for (int c = 0; c < CP; ++c) p[c] = on(c) ? 0.5f * p[c] - half_mean : Piece<V>(0.0f);
        }
        const auto squares = [&](float scale) {
            float sq = 0.0f;
#pragma unroll
            for (int c = 0; c < CP; ++c)
#pragma unroll
                for (int i = 0; i < V; ++i) sq += (scale * p[c][i]) * (scale * p[c][i]);
            return block_sum<NW>(sq, part[2 * which + 1]);
        };
        float total = squares(1.0f), scale = 1.0f;
        if (out_of_range(total, a.eps)) {
            scale = total < 1.0f ? kUp : kDown;
            if (NW > 1) __syncthreads();   // the sums have been read
            total = squares(scale);
        }
        const float r = scale / sqrtf(total * inv_n + scaled_eps(a.eps, unit * scale));
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            if constexpr (HOLD)
                p[c] = p[c] * r * kept[which][0][c] + kept[which][1][c];
            else
                p[c] = p[c] * r * vector(which, false, c) + vector(which, true, c);
        }
    };
    const auto y_of = [&](int64_t row, int c) { return load<V>((const T*)a.y + row * a.y_s + at(c)); };
    const auto x_of = [&](int64_t row, int c) { return load<V>((const T*)a.x + row * a.x_s + at(c)); };
    const auto gate_of = [&](int64_t row, int c) {
        return load<V>((const T*)a.gate + (a.gate_rows.d ? (int64_t)divu((uint32_t)row, a.gate_rows) * a.g_s : 0) + at(c));
    };
    Raw<T, V> y[HC] = {}, x[HC] = {}, gate[HC] = {};
    const auto fetch = [&](int64_t row) {
        if constexpr (HOLD) {
            if (row >= a.rows) return;
#pragma unroll
            for (int c = 0; c < CP; ++c) {
                if (!on(c)) continue;
                y[c] = y_of(row, c);
                x[c] = x_of(row, c);
                if (a.gate) gate[c] = gate_of(row, c);
            }
        }
    };
    fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (NW > 1 && row != blockIdx.x) __syncthreads();   // the last row's sums have been read
        if (!HOLD) asm volatile("" : "+v"(base));           // no place is kept in registers across the rows
        Piece<V> u[CP], rx[HC], g[HC];
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            if constexpr (HOLD) {
                u[c] = values<V, T>(y[c]);
                rx[c] = values<V, T>(x[c]);
                g[c] = values<V, T>(gate[c]);
            } else {
                u[c] = on(c) ? values<V, T>(y_of(row, c)) : Piece<V>(0.0f);
            }
        }
        fetch(row + gridDim.x);
        if (a.post) norm(u, a.post, 0);
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            if (!on(c)) {
                u[c] = Piece<V>(0.0f);
                continue;
            }
            if constexpr (!HOLD) {
                rx[0] = values<V, T>(x_of(row, c));
                if (a.gate) g[0] = values<V, T>(gate_of(row, c));
            }
            if (a.gate) u[c] *= g[HOLD ? c : 0];
            u[c] = a.residual_scale * rx[HOLD ? c : 0] + a.block_scale * u[c];
            store<V>((T*)a.residual + row * a.r_s + at(c), u[c]);   // this thread has read all that it overwrites
        }
        if (!a.pre) continue;
        norm(u, a.pre, 1);
#pragma unroll
        for (int c = 0; c < CP; ++c)
            if (on(c)) store<V>((T*)a.out + row * a.o_s + at(c), u[c]);
    }
}

// Wide rows at any alignment: 1024 threads a row, which lies in LDS in fp32.
template <typename T>
__global__ __launch_bounds__(1024) void block_norm_wide(NormArgs a) {
    __shared__ float v[NORM_MAX_WIDTH];
    __shared__ float part[4][16];
    const int tid = threadIdx.x;
    const float inv_n = 1.0f / (float)a.width;
    // Each thread keeps to its own elements.
    const auto norm = [&](int kind, const float* gamma, const float* beta, float (*sums)[16]) {
        float mean, total, eps = a.eps;
        for (bool again = false;; again = true) {
            mean = 0.0f;
            if (kind == BLOCK_NORM_LAYER) {
                float s = 0.0f;
                for (int e = tid; e < a.width; e += 1024) s += v[e];
                mean = block_sum<16>(s, sums[0]) * inv_n;
            }
            float sq = 0.0f;
            for (int e = tid; e < a.width; e += 1024) sq += (v[e] - mean) * (v[e] - mean);
            total = block_sum<16>(sq, sums[1]);
            if (again || !out_of_range(total, eps)) break;
            const float scale = total < 1.0f ? kUp : kDown;
            for (int e = tid; e < a.width; e += 1024) v[e] *= scale;
            eps = scaled_eps(eps, scale);
            __syncthreads();   // the sums have been read
        }
        const float r = 1.0f / sqrtf(total * inv_n + eps);
        for (int e = tid; e < a.width; e += 1024) v[e] = (v[e] - mean) * r * gamma[e] + (beta ? beta[e] : 0.0f);
    };
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (row != blockIdx.x) __syncthreads();   // the last row's sums have been read
        const T *y = (const T*)a.y + row * a.y_s, *x = (const T*)a.x + row * a.x_s;
        const T* gate = (const T*)a.gate + (a.gate_rows.d ? (int64_t)divu((uint32_t)row, a.gate_rows) * a.g_s : 0);
        for (int e = tid; e < a.width; e += 1024) v[e] = to_f32(y[e]);
        if (a.post) norm(a.post, a.post_gamma, a.post_beta, part);
        for (int e = tid; e < a.width; e += 1024) {
            const float u = a.gate ? v[e] * to_f32(gate[e]) : v[e];
            v[e] = a.residual_scale * to_f32(x[e]) + a.block_scale * u;
            ((T*)a.residual)[row * a.r_s + e] = from_f32<T>(v[e]);
        }
        if (!a.pre) continue;
        norm(a.pre, a.pre_gamma, a.pre_beta, part + 2);
        for (int e = tid; e < a.width; e += 1024) ((T*)a.out)[row * a.o_s + e] = from_f32<T>(v[e]);
    }
}

template <typename T, int V, int NW, int CP>
hipError_t run(const NormArgs& a, hipStream_t s) {
    const int64_t most = (int64_t)device_cu_count() * (NW > 8 ? 1 : 16 / NW);   // 16 waves a CU
    block_norm<T, V, NW, CP><<<dim3((uint32_t)(a.rows < most ? a.rows : most)), dim3(64 * NW), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t run(bool vec, const NormArgs& a, hipStream_t s) {
    if (!vec) {
        if (a.width <= 1024) return run<T, 1, 4, 4>(a, s);
        if (a.width <= 8192) return run<T, 1, 16, 8>(a, s);
        const int64_t most = device_cu_count();   // a row takes most of a CU's LDS
        block_norm_wide<T><<<dim3((uint32_t)(a.rows < most ? a.rows : most)), dim3(1024), 0, s>>>(a);
        return hipGetLastError();
    }
    if (a.width <= 512) return run<T, 8, 1, 1>(a, s);
    if (a.width <= 1024) return run<T, 8, 2, 1>(a, s);
    if (a.width <= 2048) return run<T, 8, 4, 1>(a, s);
    if (a.width <= 4096) return run<T, 8, 8, 1>(a, s);
    if (a.width <= 8192) return run<T, 8, 16, 1>(a, s);
    if (a.width <= 16384) return run<T, 8, 16, 2>(a, s);
    return run<T, 8, 16, 4>(a, s);
}

}  // namespace

hipError_t launch_block_norm(int32_t dtype, bool vec, const NormArgs& a, hipStream_t s) {
    return dtype == CONV_DTYPE_F32 ? run<float>(vec, a, s) : run<bf16>(vec, a, s);
}

}  // namespace conv2d
