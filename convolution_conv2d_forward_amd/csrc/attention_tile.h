// Softmax attention of many rows.  Compiled once for each type
// (attention_f32.hip, attention_bf16.hip).
#pragma once

#include "attention_common.h"
#include "attention_layout.h"
#include "linear_common.h"

namespace conv2d {

namespace {

// A workgroup of four waves takes 128 of the rows (query i, head of the group)
// that share a key head, 32 rows a wave, and walks their keys in tiles of 64
// (fp32: 32), which are copied straight to LDS, one to three tiles ahead.  With KW = 2 it
// takes 64 rows, and two waves share a row group, each with half of a tile's
// keys; their results meet at the end.  That gives more workgroups, of less
// work, where there are few.
//
// Both products are formed transposed, S^T = K Q^T and O^T = V^T P^T, in 32x32
// steps: a lane holds scores of one row only (half of a tile's keys; lane ^ 32
// has the others), so a row's maximum takes one exchange, its weights
// (bf16: rounded in the registers that held the scores) are the second
// product's operand as they lie, and the running sums and the outputs are
// scaled by a factor of the lane's own.  V^T is read with transposing LDS
// loads, in the order of keys that the scores have.
//
// The reference of the running maximum is moved only when some row's scores
// rise past it by more than 8 (a factor of 256 in the weights, which fp32 sums
// and bf16 weights carry as well as 1): the outputs are then rarely rescaled.
//
// What bounds it: with capped scores the vector units (a score takes two
// exp2 and a reciprocal besides the products), else the matrix cores and the
// LDS reads that feed them; two workgroups on a CU fill each other's gaps.
//
// Keys that a row does not see get weight 0 by selection, in the tiles that
// the wave's rows do not all see whole.  An infinity or NaN in such a key's
// value would still spoil the row (0 * inf): tiles that some row of the
// workgroup does not see whole are searched for them, zeros take their place
// in LDS, and the rows that see them get them one by one.
template <typename T, int DP, int KW, int CAP, bool SLOPE>
__global__ __launch_bounds__(256, (TileAttn<T, DP, KW>::OCC)) void attention_tile(AttnArgs a) {
    typedef TileAttn<T, DP, KW> C;
    constexpr bool HALF = C::HALF;
    constexpr int BK = C::BK, TK = C::TK, CPR = C::CPR, KS = C::KS, DT = C::DT, CP = C::CP;
    // How a score x follows from what its register holds, u: x = u itself; or
    // PLAIN, x = scale u; or TURNED, x = cap (1 - 2 u).
    constexpr bool PLAIN = !CAP && !SLOPE, TURNED = CAP == kCapTurned && !SLOPE;
    __shared__ __align__(1024) u32x4 lds[C::S * C::STAGE];
    __shared__ int lrange[4][4];
    // The last even and odd tile that held infinities or NaN: a wave may reach
    // the next tile's search while another still asks for this one's outcome.
    __shared__ int lbad[2];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, g = lane >> 5, kpart = wave / C::RG;
    uint32_t blk = blockIdx.x;
    const int bh = (int)(blk % (uint32_t)(a.batch * a.heads_kv));
    blk /= (uint32_t)(a.batch * a.heads_kv);
    const int split = (int)(blk % (uint32_t)a.splits);
    const int tile_r = a.row_tiles - 1 - (int)(blk / (uint32_t)a.splits);   // causal: the longest rows first
    const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
    const SeqLens sl = seq_lens(a, b);

    // This lane's row, and the intervals of the wave and the workgroup.
    const int row = tile_r * (32 * C::RG) + wave % C::RG * 32 + n;
    const bool live = row < a.rows;
    const int qi = live ? row / a.group : 0, hq = hk * a.group + (live ? row - qi * a.group : 0);
    int lo = 0, hi = 0;
    row_interval(a, sl, b, qi, live, lo, hi);
    const bool empty = hi <= lo;
    int w_lo = empty ? INT32_MAX : lo, w_hi = hi;                                      // keys that some row sees
    int f_lo = live ? (empty ? INT32_MAX : lo) : 0, f_hi = live ? hi : INT32_MAX;      // keys that every row sees
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        w_lo = min(w_lo, __shfl_xor(w_lo, m, 64));
        w_hi = max(w_hi, __shfl_xor(w_hi, m, 64));
        f_lo = max(f_lo, __shfl_xor(f_lo, m, 64));
        f_hi = min(f_hi, __shfl_xor(f_hi, m, 64));
    }
    w_lo = __builtin_amdgcn_readfirstlane(w_lo);
    w_hi = __builtin_amdgcn_readfirstlane(w_hi);
    f_lo = __builtin_amdgcn_readfirstlane(f_lo);
    f_hi = __builtin_amdgcn_readfirstlane(f_hi);
    if (lane == 0) {
        lrange[wave][0] = w_lo;
        lrange[wave][1] = w_hi;
        lrange[wave][2] = f_lo;
        lrange[wave][3] = f_hi;
    }
    if (tid < 2) lbad[tid] = -1;
    const int chunks = a.d / C::C;
    if (a.d < DP)   // chunks past d stay zero: no copy touches them
        for (int i = tid; i < C::S * C::STAGE; i += 256) {
            const int r = i / CPR % BK;
            if (((i % CPR) ^ C::swizzle(r)) >= chunks) lds[i] = u32x4{0, 0, 0, 0};
        }
    __syncthreads();
    int g_lo = min(min(lrange[0][0], lrange[1][0]), min(lrange[2][0], lrange[3][0]));
    int g_hi = max(max(lrange[0][1], lrange[1][1]), max(lrange[2][1], lrange[3][1]));
    const int all_lo = __builtin_amdgcn_readfirstlane(max(max(lrange[0][2], lrange[1][2]), max(lrange[2][2], lrange[3][2])));
    const int all_hi = __builtin_amdgcn_readfirstlane(min(min(lrange[0][3], lrange[1][3]), min(lrange[2][3], lrange[3][3])));
    if (g_lo > g_hi) g_lo = g_hi;
    const int t0 = g_lo / BK, tn = (g_hi + BK - 1) / BK - t0;
    const int first = __builtin_amdgcn_readfirstlane(t0 + (int)((int64_t)tn * split / a.splits));
    const int last = __builtin_amdgcn_readfirstlane(t0 + (int)((int64_t)tn * (split + 1) / a.splits));

    // Q as the products' second operand; a negative scale goes into its signs,
    // and one of zero makes it zero: a masked score, -inf, is multiplied by the
    // scale later (PLAIN), which has to leave it -inf.
    const bool flat = a.scale == 0.0f;
    const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
    u32x4 fq[KS];
    {
        const T* qp = (const T*)a.q + b * a.q_s[0] + qi * a.q_s[1] + hq * a.q_s[2];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int e = (2 * s + g) * C::C;
            fq[s] = u32x4{0, 0, 0, 0};
            if (live && e < a.d && !flat) fq[s] = *(const u32x4*)(qp + e);
            if (a.scale < 0.0f) fq[s] ^= HALF ? 0x80008000u : 0x80000000u;
        }
    }
    const float scale = flat ? 1.0f : sign * a.scale * kLog2e;       // scores in units of log 2
    const float cap = CAP == kCapTurned ? a.softcap * kLog2e : a.softcap;
    const float tscale = CAP == kCapTurned ? fminf(fabsf(a.scale) / a.softcap * (2.0f * kLog2e), FLT_MAX)
                         : CAP             ? cap_scale(fabsf(a.scale), a.softcap)
                                           : 0.0f;
    const float slope = SLOPE && live ? a.slopes[hq] * kLog2e : 0.0f;
    const int pos = sl.nk - sl.nq + qi;

    // Copies: chunks of rows tid / CPR + i * (256 / CPR) of a tile.  Rows past
    // the last key repeat it; their weights are zero.
    const T* kp = (const T*)a.k + b * a.k_s[0] + hk * a.k_s[2];
    const T* vp = (const T*)a.v + b * a.v_s[0] + hk * a.v_s[2];
    const int ks = (int)a.k_s[1], vs = (int)a.v_s[1];
    const auto issue = [&](int tile, int stage) {
        u32x4* dst = lds + stage * C::STAGE + wave * 64;
        const T *kt = kp + (int64_t)tile * BK * a.k_s[1], *vt = vp + (int64_t)tile * BK * a.v_s[1];
        const int left = sl.nk - 1 - tile * BK;
        int r0 = tid / CPR;
        asm volatile("" : "+v"(r0));   // the offsets are formed anew for each tile: they would cost registers
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            const int r = r0 + i * (256 / CPR), c = (tid % CPR) ^ C::swizzle(r), rc = min(r, left);
            if (c < chunks) {
                copy16_to_lds(kt, (uint32_t)(rc * ks + c * C::C) * (uint32_t)sizeof(T), dst + i * 256);
                copy16_to_lds(vt, (uint32_t)(rc * vs + c * C::C) * (uint32_t)sizeof(T), dst + BK * CPR + i * 256);
            }
        }
    };

    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    f32x16 o[DT] = {};
    float m_run = -INFINITY, l_run = 0.0f;
#pragma unroll
    for (int i = 0; i < C::S - 1; ++i)
        if (first + i < last) issue(first + i, i);
    int stage = 0;
    for (int tile = first; tile < last; ++tile, stage = stage == C::S - 1 ? 0 : stage + 1) {
        const int k0 = tile * BK;
        // The wave's part of the tile.
        const int kw = k0 + kpart * 32 * TK;
        const uint32_t at0 = lds0 + (stage * C::STAGE + kpart * 32 * TK * CPR) * 16;
        uint32_t k_at = at0 + C::k_at(lane), v_at = at0 + C::v_at(lane);
        asm volatile("" : "+v"(k_at), "+v"(v_at));   // likewise
        // This tile's copies have landed; the next ones' may be in flight.
        if (C::S > 2 && tile + C::S - 2 < last)
            wait_vmem<2 * CP * (C::S - 2)>();
        else
            wait_vmem<0>();
        const bool mixed = k0 < all_lo || k0 + BK > all_hi;
        if (mixed) {
            // This thread's own chunks of V.
#pragma unroll
            for (int i = 0; i < CP; ++i) {
                const int r = tid / CPR + i * (256 / CPR);
                u32x4& chunk = lds[stage * C::STAGE + BK * CPR + i * 256 + tid];
                u32x4 v = chunk;
                if (((tid % CPR) ^ C::swizzle(r)) < chunks && has_bad<T>(v)) {
                    clean_chunk<T>(v);
                    chunk = v;
                    lbad[tile & 1] = tile;
                }
            }
        }
        __syncthreads();
        if (tile + C::S - 1 < last) issue(tile + C::S - 1, stage == 0 ? C::S - 1 : stage - 1);
        if (kw + 32 * TK <= w_lo || kw >= w_hi) continue;   // none of the wave's rows sees a key

        f32x16 s[TK] = {};
#pragma unroll
        for (int t = 0; t < TK; ++t)
#pragma unroll
            for (int i = 0; i < KS; ++i)
                s[t] = mfma32_step<T>(*lds_ptr<const lds_u32x4>((k_at ^ 32 * i) + t * 512 * CPR), fq[i], s[t]);
        const float a1 = PLAIN ? scale : TURNED ? -2.0f * cap : 1.0f, a0 = TURNED ? cap : 0.0f;
        const float far = (float)(pos - kw - 4 * g);
        if (CAP || SLOPE) {
#pragma unroll
            for (int t = 0; t < TK; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x = s[t][i];
                    if (CAP == kCapTurned) {
                        x = turned(x * tscale);
                        if (SLOPE) x = cap - 2.0f * cap * x;
                    } else if (CAP) {
                        x = cap * score_tanh<T>(x * tscale) * kLog2e;
                    } else {
                        x *= scale;
                    }
                    if (SLOPE) x -= slope * fabsf(far - (float)(32 * t + 8 * (i >> 2) + (i & 3)));
                    s[t][i] = x;
                }
        }
        // Keys before and past what a row sees, each where some row needs it.
        constexpr float NEVER = TURNED ? INFINITY : -INFINITY;
        if (kw < f_lo) {
            const int from = lo - kw - 4 * g;
#pragma unroll
            for (int i = 0; i < 16 * TK; ++i)
                if (32 * (i >> 4) + 8 * (i >> 2 & 3) + (i & 3) < from) s[i >> 4][i & 15] = NEVER;
        }
        if (kw + 32 * TK > f_hi) {
            const int to = hi - kw - 4 * g;
#pragma unroll
            for (int i = 0; i < 16 * TK; ++i)
                if (32 * (i >> 4) + 8 * (i >> 2 & 3) + (i & 3) >= to) s[i >> 4][i & 15] = NEVER;
        }
        float top = s[0][0];
#pragma unroll
        for (int i = 1; i < 16 * TK; ++i) {
            const float x = s[i >> 4][i & 15];
            top = TURNED ? fminf(top, x) : fmaxf(top, x);
        }
        {
            float u, v;
            both_halves(top, u, v);
            top = (TURNED ? fminf(u, v) : fmaxf(u, v)) * a1 + a0;
        }
        if (__ballot(top > m_run + 8.0f)) {
            const float m_new = fmaxf(m_run, top);
            const float fade = __builtin_amdgcn_exp2f(m_run - (m_new == -INFINITY ? 0.0f : m_new));
            m_run = m_new;
            l_run *= fade;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= fade;
        }
        const float base = a0 - (m_run == -INFINITY ? 0.0f : m_run);   // nothing seen yet: every weight is 0
        // The weights: bf16 ones are rounded before the product, as the values
        // are; their sum is of the unrounded ones.  Adding the product with what
        // the rounding leaves, as attention_rows does, takes the difference
        // from unrounded weights from 2.4e-3 (rms, of the outputs' rms) to 1e-4,
        // and from 64 bits, after the outputs' own rounding, from 2.2e-3 to
        // 1.7e-3, but 8192 causal capped rows of 16 heads of 128 over 4 from 354
        // to 450 us, uncapped ones from 289 to 395.
        bf16x8 p[2 * TK];
#pragma unroll
        for (int t = 0; t < 2 * TK; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = __builtin_amdgcn_exp2f(s[t >> 1][8 * (t & 1) + i] * a1 + base);
                s[t >> 1][8 * (t & 1) + i] = w;
                l_run += w;
                if (HALF) p[t][i] = (bf16)w;
            }
        if constexpr (HALF) {
#pragma unroll
            for (int t = 0; t < 2 * TK; ++t)
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(C::vt(v_at, 16 * t, 32 * d), p[t], o[d], 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(C::vt1(v_at, i, 32 * d), s[0][i], o[d], 0, 0, 0);
        }
        if (mixed && lbad[tile & 1] == tile) {
            for (int key = max(kw, w_lo); key < min(kw + 32 * TK, w_hi); ++key)
                for (int e0 = 0; e0 < a.d; e0 += 64) {
                    const float x = e0 + lane < a.d ? to_f32(vp[key * a.v_s[1] + e0 + lane]) : 0.0f;
                    for (uint64_t bad = __ballot(!(fabsf(x) < INFINITY)); bad; bad &= bad - 1) {
                        const int l = (int)__builtin_ctzll(bad);
                        const float v = __shfl(x, l, 64), add = key >= lo && key < hi ? v : 0.0f;
#pragma unroll
                        for (int d = 0; d < DT; ++d)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[d][i] += 32 * d + 8 * (i >> 2) + 4 * g + (i & 3) == e0 + l ? add : 0.0f;
                    }
                }
        }
    }
    {
        float u, v;
        both_halves(l_run, u, v);
        l_run = u + v;
    }
    if constexpr (KW == 2) {
        // The second half of the keys' results go to the first's waves.
        f32x4* part = (f32x4*)lds + wave % C::RG * (DT * 256);
        __shared__ f32x2 stat[C::RG][64];
        __syncthreads();
        if (kpart == 1) {
            stat[wave % C::RG][lane] = f32x2{m_run, l_run};
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    part[(4 * d + q) * 64 + lane] = f32x4{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
        }
        __syncthreads();
        if (kpart == 1) return;
        const f32x2 st = stat[wave][lane];
        const float m_new = fmaxf(m_run, st[0]), base = m_new == -INFINITY ? 0.0f : m_new;
        const float f0 = __builtin_amdgcn_exp2f(m_run - base), f1 = __builtin_amdgcn_exp2f(st[0] - base);
        m_run = m_new;
        l_run = l_run * f0 + st[1] * f1;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 v = part[(4 * d + q) * 64 + lane];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[d][4 * q + i] = o[d][4 * q + i] * f0 + v[i] * f1;
            }
    }
    if (!live) return;
    if (a.splits == 1) {
        const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
        T* op = (T*)a.out + b * a.o_s[0] + qi * a.o_s[1] + hq * a.o_s[2];
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int e = 32 * d + 8 * q + 4 * g;
                const f32x4 v = f32x4{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]} * inv;
                if (e < a.d) *(typename Vec<T>::v4*)(op + e) = from_f32<T>(v);
            }
        return;
    }
    const int64_t wr = ws_row(a, bh, split, row);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int e = 32 * d + 8 * q + 4 * g;
            const f32x4 v{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
            if (e < a.d) *(f32x4*)(ws_out(a, wr) + e) = v;
        }
    if (g == 0) *ws_stat(a, wr) = f32x2{m_run, l_run};
}

template <typename T, int DP, int KW>
hipError_t run(const AttnArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)((int64_t)a.batch * a.heads_kv * a.row_tiles * a.splits)), block(256);
    const auto launch = [&](auto cap) {
        if (a.slopes)
            attention_tile<T, DP, KW, cap(), true><<<grid, block, 0, s>>>(a);
        else
            attention_tile<T, DP, KW, cap(), false><<<grid, block, 0, s>>>(a);
    };
    if (a.softcap == 0.0f)
        launch(std::integral_constant<int, kCapNone>{});
    else if (sizeof(T) == 4 || a.softcap > kMostTurned)
        launch(std::integral_constant<int, kCapAny>{});
    else if constexpr (sizeof(T) == 2)
        launch(std::integral_constant<int, kCapTurned>{});
    return hipGetLastError();
}

template <typename T, int KW>
hipError_t run(const AttnArgs& a, hipStream_t s) {
    if (a.d <= 32) return run<T, 32, KW>(a, s);
    if (a.d <= 64) return run<T, 64, KW>(a, s);
    if (a.d <= 96) return run<T, 96, KW>(a, s);
    if (a.d <= 128) return run<T, 128, KW>(a, s);
    if constexpr (KW == 1 || sizeof(T) == 2) return run<T, 256, KW>(a, s);
    return hipErrorInvalidValue;   // two tiles of 64 fp32 keys do not fit in LDS: plan_attention takes 128 rows
}

}  // namespace

template <>
hipError_t launch_attention_tile<ATTENTION_T>(const AttnArgs& a, int rows, hipStream_t s) {
    return rows == 128 ? run<ATTENTION_T, 1>(a, s) : run<ATTENTION_T, 2>(a, s);
}

}  // namespace conv2d
