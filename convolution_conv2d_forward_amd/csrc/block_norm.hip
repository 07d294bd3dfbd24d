// The norm behind a block, its gate and the scaled residual, and the norm
// before the next block, a row at a time.
#include "decoder_internal.h"
#include "seq_common.h"

namespace conv2d {

namespace {

// A piece of a row: 8 elements at a 16-byte boundary, or one.
template <int V>
struct Piece {
    float v[V];
    template <typename T>
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (V == 8) {
            const f32x8 r = load8(p);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = r[i];
        } else {
            v[0] = to_f32(*p);
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (V == 8) {
            f32x8 r;
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = v[i];
            store8(p, r);
        } else {
            *p = from_f32<T>(v[0]);
        }
    }
};

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

// NW waves a row, whose pieces stay in registers, CP of them a thread: every
// element is read once and written once, and a row's mean is known before the
// squares around it are summed.
template <typename T, int V, int NW, int CP>
__global__ __launch_bounds__(64 * NW) void block_norm(NormArgs a) {
    __shared__ float part[4][NW];
    const int tid = threadIdx.x;
    const float inv_n = 1.0f / (float)a.width;
    // The norm of the pieces in place; `part` holds two sums.
    const auto norm = [&](Piece<V> (&p)[CP], int kind, const float* gamma, const float* beta, float (*sums)[NW]) {
        float mean = 0.0f;
        if (kind == BLOCK_NORM_LAYER) {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < CP; ++c)
#pragma unroll
                for (int i = 0; i < V; ++i) s += p[c].v[i];   // zeros past the row
            mean = block_sum<NW>(s, sums[0]) * inv_n;
        }
        float sq = 0.0f;
#pragma unroll
        for (int c = 0; c < CP; ++c)
            if ((tid + c * 64 * NW) * V < a.width) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    p[c].v[i] -= mean;
                    sq += p[c].v[i] * p[c].v[i];
                }
            }
        const float r = 1.0f / sqrtf(block_sum<NW>(sq, sums[1]) * inv_n + a.eps);
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            const int e = (tid + c * 64 * NW) * V;
            if (e >= a.width) continue;
            Piece<V> g, b{};
            g.load(gamma + e);
            if (beta) b.load(beta + e);
#pragma unroll
            for (int i = 0; i < V; ++i) p[c].v[i] = p[c].v[i] * r * g.v[i] + b.v[i];
        }
    };
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (NW > 1 && row != blockIdx.x) __syncthreads();   // the last row's sums have been read
        const T *y = (const T*)a.y + row * a.y_s, *x = (const T*)a.x + row * a.x_s;
        const T* gate = (const T*)a.gate + (a.gate_rows.d ? (int64_t)divu((uint32_t)row, a.gate_rows) * a.g_s : 0);
        Piece<V> u[CP] = {}, rx[CP] = {};
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            const int e = (tid + c * 64 * NW) * V;
            if (e >= a.width) continue;
            u[c].load(y + e);
            rx[c].load(x + e);
        }
        if (a.post) norm(u, a.post, a.post_gamma, a.post_beta, part);
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            const int e = (tid + c * 64 * NW) * V;
            if (e >= a.width) continue;
            if (a.gate) {
                Piece<V> g;
                g.load(gate + e);
#pragma unroll
                for (int i = 0; i < V; ++i) u[c].v[i] *= g.v[i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) u[c].v[i] = a.residual_scale * rx[c].v[i] + a.block_scale * u[c].v[i];
            u[c].store((T*)a.residual + row * a.r_s + e);   // this thread has read all that it overwrites
        }
        if (!a.pre) continue;
        norm(u, a.pre, a.pre_gamma, a.pre_beta, part + 2);
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            const int e = (tid + c * 64 * NW) * V;
            if (e < a.width) u[c].store((T*)a.out + row * a.o_s + e);
        }
    }
}

template <typename T, int V, int NW, int CP>
hipError_t run(const NormArgs& a, hipStream_t s) {
    const int64_t most = (int64_t)device_cu_count() * 64;
    block_norm<T, V, NW, CP><<<dim3((uint32_t)(a.rows < most ? a.rows : most)), dim3(64 * NW), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t run(bool vec, const NormArgs& a, hipStream_t s) {
    if (!vec) {
        if (a.width <= 1024) return run<T, 1, 4, 4>(a, s);
        if (a.width <= 8192) return run<T, 1, 16, 8>(a, s);
        return run<T, 1, 16, 32>(a, s);
    }
    if (a.width <= 512) return run<T, 8, 1, 1>(a, s);
    if (a.width <= 1024) return run<T, 8, 1, 2>(a, s);
    if (a.width <= 2048) return run<T, 8, 4, 1>(a, s);
    if (a.width <= 4096) return run<T, 8, 4, 2>(a, s);
    if (a.width <= 8192) return run<T, 8, 4, 4>(a, s);
    if (a.width <= 16384) return run<T, 8, 8, 4>(a, s);
    return run<T, 8, 16, 4>(a, s);
}

}  // namespace

hipError_t launch_block_norm(int32_t dtype, bool vec, const NormArgs& a, hipStream_t s) {
    return dtype == CONV_DTYPE_F32 ? run<float>(vec, a, s) : run<bf16>(vec, a, s);
}

}  // namespace conv2d
