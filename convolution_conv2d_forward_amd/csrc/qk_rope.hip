// Norms of queries and keys per head, position rotation, and the stores to
// the cache, in one pass over the projection's rows.
//
//   x' = gamma * x * rsqrt(mean x^2 + eps);  (a, b) -> (a c - b s, b c + a s)
//   with c, s = attn_factor * cos, sin(2 pi * frac(p * turns_i))
//
// Every element is read once and written once: the kernel is bound by memory
// traffic.  A position of 10^5 and more leaves an fp32 angle without its last
// digits, so the product p * turns_i and its reduction to a fraction of a
// turn are formed in fp64, and only the fraction goes on in fp32.
//
// A "unit" is 8 elements: four rotated pairs (two 4-element vectors
// rotary_dim/2 apart for the half layout, 8 consecutive elements for the
// interleaved one) or 8 consecutive elements that pass.  The lanes of a wave
// form groups of LPH lanes, one lane a unit, one group a head; a lane keeps
// its unit through all heads that its wave visits, so its four angles,
// and its gammas, are computed and read once per token.  The mean is
// summed over the lanes of a group by a butterfly.
#include "seq_common.h"

namespace conv2d {

namespace {

// sin and cos of the angle in turns, from its fp64 product.
__device__ __forceinline__ void turn_sincos(double t, float* s, float* c) {
    const float f = (float)(t - rint(t));
    sincospif(2.0f * f, s, c);
}

// The turns of P pairs as a kernel argument: half of a kilobyte less of them is
// half a microsecond less on the host.
template <int P>
struct RopeTurns {
    double t[P];
};

template <int P>
RopeTurns<P> turns_of(const RopeArgs& a) {
    RopeTurns<P> r;
    for (int i = 0; i < P; ++i) r.t[i] = a.turns[i];
    return r;
}

template <typename T>
__device__ __forceinline__ void load44(const T* p, int64_t off0, int64_t off1, f32x4& a, f32x4& b) {
    typedef typename Vec<T>::v4 V;
    a = to_f32(*(const V*)(p + off0));
    b = to_f32(*(const V*)(p + off1));
}

template <typename T>
__device__ __forceinline__ void store44(T* p, int64_t off0, int64_t off1, f32x4 a, f32x4 b) {
    typedef typename Vec<T>::v4 V;
    *(V*)(p + off0) = from_f32<T>(a);
    *(V*)(p + off1) = from_f32<T>(b);
}

// One wave: token blockIdx / parts, heads part, part + parts, ... in steps of
// the groups of a wave.
template <typename T, bool HALF, int LPH>
__global__ __launch_bounds__(256) void qk_rope_vec(RopeArgs a, RopeTurns<4 * LPH> turns, int parts, DivU32 dv_parts,
                                                   uint32_t waves) {
    constexpr int HPW = 64 / LPH;   // heads a wave visits at once
    const uint32_t wave = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (wave >= waves) return;
    const int lane = threadIdx.x & 63;
    const uint32_t t = divu(wave, dv_parts);
    const int part = (int)(wave - t * (uint32_t)parts);
    const int unit = lane & (LPH - 1);
    const bool live = unit * 8 < a.d;
    const bool rot = unit * 8 < a.r;
    // Offsets of the unit's two vectors within a head.
    int o0 = unit * 8, o1 = unit * 8 + 4;
    if (HALF && rot) {
        o0 = unit * 4;
        o1 = (a.r >> 1) + unit * 4;
    }
    if (!live) o0 = o1 = 0;
    f32x4 cs{1, 1, 1, 1}, sn{0, 0, 0, 0};
    if (rot) {
        const double pos = (double)a.positions[t];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s, c;
            turn_sincos(pos * turns.t[unit * 4 + i], &s, &c);
            cs[i] = c * a.attn_factor;
            sn[i] = s * a.attn_factor;
        }
    }
    f32x4 gq0{1, 1, 1, 1}, gq1 = gq0, gk0 = gq0, gk1 = gq0;
    const bool norm = a.q_gamma != nullptr;
    if (norm) {
        gq0 = *(const f32x4*)(a.q_gamma + o0);
        gq1 = *(const f32x4*)(a.q_gamma + o1);
        gk0 = *(const f32x4*)(a.k_gamma + o0);
        gk1 = *(const f32x4*)(a.k_gamma + o1);
    }
    const int64_t row = a.slots ? a.slots[t] : (int64_t)t;
    const bool keep = row >= 0 && row < a.cache_rows;
    const T* in = (const T*)a.qkv + (int64_t)t * a.qkv_s;
    T* qo = (T*)a.q + (int64_t)t * a.q_s;
    T* ko = (T*)a.k + row * a.k_s;
    T* vo = (T*)a.v + row * a.v_s;
    const int heads = a.heads_q + (a.v ? 2 : 1) * a.heads_kv;
    const float inv_d = 1.0f / (float)a.d;
    for (int h0 = part * HPW; h0 < heads; h0 += parts * HPW) {
        const int h = h0 + lane / LPH;
        const bool on = live && h < heads;
        f32x4 x0{0, 0, 0, 0}, x1{0, 0, 0, 0};
        if (on) load44(in + (int64_t)h * a.d, o0, o1, x0, x1);
        const bool is_q = h < a.heads_q, is_v = h >= a.heads_q + a.heads_kv;
        if (norm) {
            float ss = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
            for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor(ss, m, 64);
            const float r = is_v ? 1.0f : 1.0f / sqrtf(ss * inv_d + a.eps);
            if (!is_v) {
                x0 = x0 * r * (is_q ? gq0 : gk0);
                x1 = x1 * r * (is_q ? gq1 : gk1);
            }
        }
        if (rot && !is_v) {
            f32x4 y0, y1;
            if (HALF) {
                y0 = x0 * cs - x1 * sn;
                y1 = x1 * cs + x0 * sn;
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    y0[2 * i] = x0[2 * i] * cs[i] - x0[2 * i + 1] * sn[i];
                    y0[2 * i + 1] = x0[2 * i + 1] * cs[i] + x0[2 * i] * sn[i];
                    y1[2 * i] = x1[2 * i] * cs[2 + i] - x1[2 * i + 1] * sn[2 + i];
                    y1[2 * i + 1] = x1[2 * i + 1] * cs[2 + i] + x1[2 * i] * sn[2 + i];
                }
            }
            x0 = y0;
            x1 = y1;
        }
        if (!on) continue;
        if (is_q)
            store44(qo + (int64_t)h * a.d, o0, o1, x0, x1);
        else if (keep && !is_v)
            store44(ko + (int64_t)(h - a.heads_q) * a.d, o0, o1, x0, x1);
        else if (keep)
            store44(vo + (int64_t)(h - a.heads_q - a.heads_kv) * a.d, o0, o1, x0, x1);
    }
}

// Any head size, stride and alignment: one wave a (token, head), a lane a
// pair or a passing element at a time.  The sum of squares takes a first pass
// over the row; each thread then reads exactly what it overwrites, so the
// in-place form holds here too.
template <typename T, bool HALF>
__global__ __launch_bounds__(256) void qk_rope_any(RopeArgs a, RopeTurns<ROPE_MAX_PAIRS> turns, DivU32 dv_heads,
                                                   uint32_t waves) {
    const uint32_t wave = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (wave >= waves) return;
    const int lane = threadIdx.x & 63;
    const uint32_t t = divu(wave, dv_heads);
    const int h = (int)(wave - t * dv_heads.d);
    const bool is_q = h < a.heads_q, is_v = h >= a.heads_q + a.heads_kv;
    const T* in = (const T*)a.qkv + (int64_t)t * a.qkv_s + (int64_t)h * a.d;
    const int64_t row = a.slots ? a.slots[t] : (int64_t)t;
    if (!is_q && (row < 0 || row >= a.cache_rows)) return;
    T* out = is_q   ? (T*)a.q + (int64_t)t * a.q_s + (int64_t)h * a.d
             : is_v ? (T*)a.v + row * a.v_s + (int64_t)(h - a.heads_q - a.heads_kv) * a.d
                    : (T*)a.k + row * a.k_s + (int64_t)(h - a.heads_q) * a.d;
    if (is_v) {
        for (int e = lane; e < a.d; e += 64) out[e] = in[e];
        return;
    }
    const float* g = is_q ? a.q_gamma : a.k_gamma;
    float r = 1.0f;
    if (g) {
        float ss = 0;
        for (int e = lane; e < a.d; e += 64) {
            const float x = to_f32(in[e]);
            ss += x * x;
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) ss += __shfl_xor(ss, m, 64);
        r = 1.0f / sqrtf(ss / (float)a.d + a.eps);
    }
    const double pos = (double)a.positions[t];
    const int half = a.r >> 1;
    for (int i = lane; i < half; i += 64) {
        const int e0 = HALF ? i : 2 * i, e1 = HALF ? i + half : 2 * i + 1;
        float s, c;
        turn_sincos(pos * turns.t[i], &s, &c);
        s *= a.attn_factor;
        c *= a.attn_factor;
        float x0 = to_f32(in[e0]), x1 = to_f32(in[e1]);
        if (g) {
            x0 = x0 * r * g[e0];
            x1 = x1 * r * g[e1];
        }
        out[e0] = from_f32<T>(x0 * c - x1 * s);
        out[e1] = from_f32<T>(x1 * c + x0 * s);
    }
    for (int e = a.r + lane; e < a.d; e += 64) {
        const float x = to_f32(in[e]);
        out[e] = from_f32<T>(g ? x * r * g[e] : x);
    }
}

template <typename T, bool HALF, int LPH>
hipError_t run_vec(const RopeArgs& a, hipStream_t s) {
    constexpr int HPW = 64 / LPH;
    const int heads = a.heads_q + (a.v ? 2 : 1) * a.heads_kv;
    const int steps = (heads + HPW - 1) / HPW;
    // A wave takes all heads of its token where the tokens alone make enough
    // waves; few tokens (a step of single tokens) spread a token's heads over
    // up to `steps` waves.
    const int64_t want = (int64_t)device_cu_count() * 32;
    int64_t parts = (want + a.tokens - 1) / a.tokens;
    if (parts > steps) parts = steps;
    const int64_t waves = (int64_t)a.tokens * parts;
    qk_rope_vec<T, HALF, LPH><<<dim3((uint32_t)((waves + 3) / 4)), dim3(256), 0, s>>>(
        a, turns_of<4 * LPH>(a), (int)parts, make_divu32((uint32_t)parts), (uint32_t)waves);
    return hipGetLastError();
}

template <typename T, bool HALF>
hipError_t run(bool vec, const RopeArgs& a, hipStream_t s) {
    if (vec) {
        if (a.d <= 32) return run_vec<T, HALF, 4>(a, s);
        if (a.d <= 64) return run_vec<T, HALF, 8>(a, s);
        if (a.d <= 128) return run_vec<T, HALF, 16>(a, s);
        return run_vec<T, HALF, 32>(a, s);
    }
    const int heads = a.heads_q + (a.v ? 2 : 1) * a.heads_kv;
    const int64_t waves = (int64_t)a.tokens * heads;
    qk_rope_any<T, HALF><<<dim3((uint32_t)((waves + 3) / 4)), dim3(256), 0, s>>>(
        a, turns_of<ROPE_MAX_PAIRS>(a), make_divu32((uint32_t)heads), (uint32_t)waves);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_rope(int32_t dtype, int32_t layout, bool vec, const RopeArgs& a, hipStream_t s) {
    // So many tokens take a wave each, or one for each of their heads.
    const int heads = a.heads_q + (a.v ? 2 : 1) * a.heads_kv;
    const int64_t most = most_workgroups(256) * 4 / (vec ? 1 : heads);
    if (a.tokens > most) {
        const int64_t es = dtype == CONV_DTYPE_F32 ? 4 : 2;
        for (int64_t t = 0; t < a.tokens; t += most) {
            RopeArgs c = a;
            c.tokens = (int32_t)(a.tokens - t < most ? a.tokens - t : most);
            c.qkv = (const char*)a.qkv + t * a.qkv_s * es;
            c.q = (char*)a.q + t * a.q_s * es;
            c.positions = a.positions + t;
            if (a.slots) {
                c.slots = a.slots + t;
            } else {
                c.k = (char*)a.k + t * a.k_s * es;
                if (a.v) c.v = (char*)a.v + t * a.v_s * es;
                c.cache_rows = a.cache_rows - t;
            }
            const hipError_t e = launch_qk_rope(dtype, layout, vec, c, s);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const bool half = layout == ROPE_HALF;
    if (dtype == CONV_DTYPE_F32) return half ? run<float, true>(vec, a, s) : run<float, false>(vec, a, s);
    return half ? run<bf16, true>(vec, a, s) : run<bf16, false>(vec, a, s);
}

}  // namespace conv2d
