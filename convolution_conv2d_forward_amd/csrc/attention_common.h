// Device helpers of the attention kernels: row intervals, scores, the join of
// split results.
//
// Every mask of attention_forward leaves a query row one interval of keys:
// documents and lengths bound it on both sides, a window on both, causal
// order (with a prefix) above.  So a row carries [lo, hi) and nothing is read
// per key.
#pragma once

#include <cfloat>

#include "seq_common.h"

namespace conv2d {

struct SeqLens {
    int nq, nk;   // rows of this sequence that count
};

__device__ __forceinline__ SeqLens seq_lens(const AttnArgs& a, int b) {
    SeqLens s{a.q_len, a.kv_len};
    if (a.q_lens) s.nq = min(max(a.q_lens[b], 0), a.q_len);
    if (a.kv_lens) s.nk = min(max(a.kv_lens[b], 0), a.kv_len);
    return s;
}

// The keys that query i of sequence b sees; for all lanes of a wave at once
// (`live` false: none).  Empty: lo = hi = 0.
__device__ __forceinline__ void row_interval(const AttnArgs& a, SeqLens s, int b, int i, bool live, int& lo, int& hi) {
    const int p = s.nk - s.nq + i;
    lo = 0;
    hi = s.nk;
    if (!live || i >= s.nq) hi = 0;
    if (a.causal) {
        int end = p + 1;
        if (a.prefix_lens) end = max(end, a.prefix_lens[b]);
        hi = min(hi, end);
    }
    if (a.window) {
        lo = (int)max((int64_t)lo, (int64_t)p - a.window + 1);
        hi = (int)min((int64_t)hi, (int64_t)p + a.window);
    }
    if (a.doc_offsets) {
        // n: the number of borders <= p, so that document n - 1 holds p.
        // Offsets that do not ascend select some document; the interval stays
        // within the sequence.
        const int32_t* o = a.doc_offsets + (int64_t)b * (a.n_docs + 1);
        int n = 0, from = 0, to = 0;
        if (a.n_docs < 64) {
            // One load, a border a lane, and no chain of loads.
            const int lane = threadIdx.x & 63, mine = o[min(lane, a.n_docs)];
            for (int j = 0; j <= a.n_docs; ++j) n += __builtin_amdgcn_readlane(mine, j) <= p;
            from = __shfl(mine, max(n - 1, 0), 64);
            to = __shfl(mine, min(n, a.n_docs), 64);
        } else {
            int n1 = a.n_docs + 1;
            while (n < n1) {
                const int mid = (n + n1) >> 1;
                if (o[mid] <= p)
                    n = mid + 1;
                else
                    n1 = mid;
            }
            from = o[max(n - 1, 0)];
            to = o[min(n, a.n_docs)];
        }
        if (n == 0 || n > a.n_docs || p < 0) {
            hi = 0;
        } else {
            lo = max(lo, from);
            hi = min(hi, to);
        }
    }
    if (hi <= lo) lo = hi = 0;
}

// Forms of a score's cap.  kCapTurned, bf16 alone: cap (1 - 2 u) with
// u = 1 / (exp(2 t) + 1), off by some cap 2^-22, which up to the cap kMostTurned
// (2^-13) is small next to the weights' rounding.  kCapAny: a tanh whose error
// is relative to its value, so that a cap of any size may multiply it: fp32
// takes the library's; bf16 the same quotient from 1/4 on, and below it the
// series to x^7, whose next term is 62/2835 x^8 < 2^-21 of the sum.  (8192
// causal rows of 16 bf16 heads of 128 over 4: 357 us turned, 412 any.)
enum { kCapNone, kCapTurned, kCapAny };
constexpr float kMostTurned = 512.0f;

__device__ __forceinline__ float turned(float twice_log2e_t) {
    return __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(twice_log2e_t) + 1.0f);
}
template <typename T>
__device__ __forceinline__ float score_tanh(float x);
template <>
__device__ __forceinline__ float score_tanh<float>(float x) {
    return tanhf(x);
}
template <>
__device__ __forceinline__ float score_tanh<bf16>(float x) {
    const float q = x * x, near = x + x * q * (-1.0f / 3.0f + q * (2.0f / 15.0f - q * (17.0f / 315.0f)));
    return fabsf(x) < 0.25f ? near : 1.0f - 2.0f * turned(x * (2.0f * kLog2e));
}

// Factor that gives the tanh's argument, scale / cap: finite also for caps next
// to zero, so that a score of zero stays zero.
__device__ __forceinline__ float cap_scale(float scale, float cap) {
    return fminf(fmaxf(scale / cap, -FLT_MAX), FLT_MAX);
}

// Scores in units of log 2, so that exp2 gives the weights.
struct ScoreP {
    float scale;   // without a cap: scale log2(e); with one: scale / cap
    float cap;     // 0 without
};

__device__ __forceinline__ ScoreP score_params(const AttnArgs& a) {
    ScoreP p;
    p.cap = a.softcap;
    p.scale = a.softcap > 0.0f ? cap_scale(a.scale, a.softcap) : a.scale * kLog2e;
    return p;
}

// N products q.k become scores in these units.  (cap log2(e) alone may be
// beyond fp32.)  One decision for all: made for each, or the series for every
// cap, it costs 2 % of a token's time.
template <typename T, int N>
__device__ __forceinline__ void scores(const ScoreP& p, float (&s)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] *= p.scale;
    if (sizeof(T) == 2 && p.cap > 0.0f && p.cap <= kMostTurned) {
        const float cap = p.cap * kLog2e;
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = cap - 2.0f * cap * turned(s[i] * (2.0f * kLog2e));
    } else if (p.cap > 0.0f) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = p.cap * score_tanh<T>(s[i]) * kLog2e;
    }
}

// Whether a chunk holds elements whose exponent bits are all ones: one more in
// the exponent carries into the sign's place.
template <typename T>
__device__ __forceinline__ bool has_bad(u32x4 v) {
    constexpr uint32_t E = sizeof(T) == 2 ? 0x7f807f80u : 0x7f800000u, ONE = sizeof(T) == 2 ? 0x00800080u : 0x00800000u;
    return ((((v[0] & E) + ONE) | ((v[1] & E) + ONE) | ((v[2] & E) + ONE) | ((v[3] & E) + ONE)) & (~E & (E + ONE))) != 0;
}

// Elements whose exponent bits are all ones (infinities, NaN) become zero;
// says whether there were any.
template <typename T>
__device__ __forceinline__ bool clean_chunk(u32x4& v);
template <>
__device__ __forceinline__ bool clean_chunk<float>(u32x4& v) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if ((v[i] & 0x7f800000u) == 0x7f800000u) {
            v[i] = 0;
            bad = true;
        }
    return bad;
}
template <>
__device__ __forceinline__ bool clean_chunk<bf16>(u32x4& v) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((v[i] & 0x7f80u) == 0x7f80u) {
            v[i] &= 0xffff0000u;
            bad = true;
        }
        if ((v[i] & 0x7f800000u) == 0x7f800000u) {
            v[i] &= 0xffffu;
            bad = true;
        }
    }
    return bad;
}

// Partial results of a split: for each (sequence, key head, split, row)
// d unnormalised outputs, then for all rows the pair (running maximum, sum).
__device__ __forceinline__ int64_t ws_row(const AttnArgs& a, int bh, int split, int row) {
    return ((int64_t)bh * a.splits + split) * a.rows + row;
}
__device__ __forceinline__ float* ws_out(const AttnArgs& a, int64_t row) { return a.ws + row * a.d; }
__device__ __forceinline__ f32x2* ws_stat(const AttnArgs& a, int64_t row) {
    const int64_t all = (int64_t)a.batch * a.heads_kv * a.splits * a.rows;
    return (f32x2*)(a.ws + all * a.d) + row;
}

// Tiles of 128 or 64 rows (attention_tile.h).
template <typename T>
hipError_t launch_attention_tile(const AttnArgs& a, int rows, hipStream_t s);
template <>
hipError_t launch_attention_tile<float>(const AttnArgs& a, int rows, hipStream_t s);
template <>
hipError_t launch_attention_tile<bf16>(const AttnArgs& a, int rows, hipStream_t s);

// Joins the splits' results (attention_any.hip).
hipError_t launch_attention_join(int32_t dtype, const AttnArgs& a, hipStream_t s);

}  // namespace conv2d
