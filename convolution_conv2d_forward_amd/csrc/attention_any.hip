// Softmax attention for both types and every shape: dispatch, the general
// kernel, and the join of split results.
#include "attention_common.h"
#include "linear_common.h"

namespace conv2d {

namespace {

// A workgroup of four waves takes 64 of the rows (query i, head of the group)
// that share a key head, 16 rows a wave, and walks their keys in tiles of 32.
// The product is formed transposed, S^T = K Q^T, so a lane holds scores of
// one row only: maximum and sum need two exchanges between lanes, and the
// scores are already laid out as the second operand of O^T = V^T P^T.  That
// product's sum over keys takes them in the order in which the lanes hold them,
// and V^T is read accordingly.  K and V are staged in LDS with 16 bytes of
// padding a row; the next tile is in registers meanwhile.
//
// Keys that a row does not see get weight 0 by selection.  An infinity or NaN
// in such a key's value would still spoil the row (0 * inf), so tiles that
// some row of the workgroup does not see whole are staged with those elements
// set to zero, and the rows that do see them add them one by one.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attention_any(AttnArgs a) {
    constexpr int BK = 32, C = Vec<T>::chunk, DC = DP / C;     // DC: 16-byte chunks of a row
    constexpr int KS = DP * (int)sizeof(T) / 64;               // 64-byte product steps over a row
    constexpr int LROW = DP + C;                               // LDS row, elements
    constexpr int NCH = (BK * DC + 255) / 256;                 // chunks a thread stages per operand
    __shared__ __align__(16) T lk[BK * LROW];
    __shared__ __align__(16) T lv[BK * LROW];
    __shared__ float lp[4][BK * 16];   // weights, for the one-by-one addition alone
    __shared__ int lrange[4][4];
    __shared__ int lbad;               // the last tile that held infinities or NaN

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = lane & 15, g = lane >> 4;
    uint32_t blk = blockIdx.x;
    const int bh = (int)(blk % (uint32_t)(a.batch * a.heads_kv));
    blk /= (uint32_t)(a.batch * a.heads_kv);
    const int split = (int)(blk % (uint32_t)a.splits);
    const int tile_r = a.row_tiles - 1 - (int)(blk / (uint32_t)a.splits);   // causal: the longest rows first
    const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
    const SeqLens sl = seq_lens(a, b);

    // This lane's row, and the intervals of the wave and the workgroup.
    const int row = tile_r * 64 + wave * 16 + n;
    const bool live = row < a.rows;
    const int qi = live ? row / a.group : 0, hq = hk * a.group + (live ? row - qi * a.group : 0);
    int lo = 0, hi = 0;
    if (live) row_interval(a, sl, b, qi, lo, hi);
    const bool empty = hi <= lo;
    int min_lo = empty ? INT32_MAX : lo, max_hi = hi;
    // Rows past the end do not count against a tile being seen whole.
    int max_lo = live ? (empty ? INT32_MAX : lo) : 0, min_hi = live ? hi : INT32_MAX;
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {
        min_lo = min(min_lo, __shfl_xor(min_lo, m, 64));
        max_hi = max(max_hi, __shfl_xor(max_hi, m, 64));
        max_lo = max(max_lo, __shfl_xor(max_lo, m, 64));
        min_hi = min(min_hi, __shfl_xor(min_hi, m, 64));
    }
    if (lane == 0) {
        lrange[wave][0] = min_lo;
        lrange[wave][1] = max_hi;
        lrange[wave][2] = max_lo;
        lrange[wave][3] = min_hi;
    }
    if (tid == 0) lbad = -1;
    __syncthreads();
    int wlo = min(min(lrange[0][0], lrange[1][0]), min(lrange[2][0], lrange[3][0]));
    const int whi = max(max(lrange[0][1], lrange[1][1]), max(lrange[2][1], lrange[3][1]));
    const int full_lo = max(max(lrange[0][2], lrange[1][2]), max(lrange[2][2], lrange[3][2]));
    const int full_hi = min(min(lrange[0][3], lrange[1][3]), min(lrange[2][3], lrange[3][3]));
    if (wlo > whi) wlo = whi;

    // The tiles of this split.
    const int t0 = wlo / BK, tn = (whi + BK - 1) / BK - t0;
    const int first = t0 + (int)((int64_t)tn * split / a.splits), last = t0 + (int)((int64_t)tn * (split + 1) / a.splits);

    const T* kp = (const T*)a.k + b * a.k_s[0] + hk * a.k_s[2];
    const T* vp = (const T*)a.v + b * a.v_s[0] + hk * a.v_s[2];
    u32x4 fq[KS];
    {
        const T* qp = (const T*)a.q + b * a.q_s[0] + qi * a.q_s[1] + hq * a.q_s[2];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int e = (s * 4 + g) * C;
            fq[s] = u32x4{0, 0, 0, 0};
            if (live && e < a.d) fq[s] = *(const u32x4*)(qp + e);
        }
    }
    const ScoreP sp = score_params(a);
    const float slope = a.slopes && live ? a.slopes[hq] * kLog2e : 0.0f;
    const int pos = sl.nk - sl.nq + qi;

    u32x4 rk[NCH], rv[NCH];
    // Chunks of keys from kv_len on, and of elements from d on, are zero and not read.
    const auto fetch = [&](int tile) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = tid + i * 256, key = tile * BK + c / DC, e = (c % DC) * C;
            rk[i] = rv[i] = u32x4{0, 0, 0, 0};
            if (c < BK * DC && key < sl.nk && e < a.d) {
                rk[i] = *(const u32x4*)(kp + key * a.k_s[1] + e);
                rv[i] = *(const u32x4*)(vp + key * a.v_s[1] + e);
            }
        }
    };

    f32x4 o[DP / 16] = {};
    float m_run = -INFINITY, l_run = 0.0f;
    if (first < last) fetch(first);
    for (int tile = first; tile < last; ++tile) {
        const int k0 = tile * BK;
        const bool whole = k0 >= full_lo && k0 + BK <= full_hi;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = tid + i * 256;
            if (c < BK * DC) {
                const int at = (c / DC) * LROW + (c % DC) * C;
                if (!whole && clean_chunk<T>(rv[i])) lbad = tile;
                *(u32x4*)(lk + at) = rk[i];
                *(u32x4*)(lv + at) = rv[i];
            }
        }
        __syncthreads();
        if (tile + 1 < last) fetch(tile + 1);

        f32x4 s[2] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const u32x4 fk = *(const u32x4*)(lk + (16 * t + n) * LROW + (ks * 4 + g) * C);
                s[t] = mfma_step<T>(fk, fq[ks], s[t]);
            }
        float m_new = m_run;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = k0 + 16 * t + 4 * g + i;
                float x = s[t][i] * sp.scale;
                if (sp.cap > 0.0f) x = sp.cap * score_tanh<T>(x);
                if (a.slopes) x -= slope * fabsf((float)(pos - key));
                if (!whole) x = key >= lo && key < hi ? x : -INFINITY;
                s[t][i] = x;
                m_new = fmaxf(m_new, x);
            }
        m_new = fmaxf(m_new, __shfl_xor(m_new, 16, 64));
        m_new = fmaxf(m_new, __shfl_xor(m_new, 32, 64));
        const float base = m_new == -INFINITY ? 0.0f : m_new;   // nothing seen yet: every weight is 0
        const float fade = __builtin_amdgcn_exp2f(m_run - base);
        m_run = m_new;
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[t][i] = __builtin_amdgcn_exp2f(s[t][i] - base);
                sum += s[t][i];
            }
        l_run = l_run * fade + sum;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) o[d] *= fade;
        if constexpr (sizeof(T) == 2) {
            bf16x8 fp;
#pragma unroll
            for (int i = 0; i < 8; ++i) fp[i] = (bf16)s[i >> 2][i & 3];
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
                bf16x8 fv;
#pragma unroll
                for (int i = 0; i < 8; ++i) fv[i] = lv[(16 * (i >> 2) + 4 * g + (i & 3)) * LROW + 16 * d + n];
                o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, fp, o[d], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int d = 0; d < DP / 16; ++d)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float fv = lv[(16 * (i >> 2) + 4 * g + (i & 3)) * LROW + 16 * d + n];
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(fv, s[i >> 2][i & 3], o[d], 0, 0, 0);
                }
        }
        if (!whole && lbad == tile) {
            // The elements that were set to zero, for the rows that see them.
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) lp[wave][(16 * t + 4 * g + i) * 16 + n] = s[t][i];
            __builtin_amdgcn_wave_barrier();
            for (int j = 0; j < BK; ++j) {
                const int key = k0 + j;
                if (key < lo || key >= hi) continue;
                const float p = lp[wave][j * 16 + n];
                for (int d = 0; d < DP / 16; ++d)
                    for (int i = 0; i < 4; ++i) {
                        const int e = 16 * d + 4 * g + i;
                        if (e >= a.d) continue;
                        const float v = to_f32(vp[key * a.v_s[1] + e]);
                        if (!(fabsf(v) < INFINITY)) {
#pragma unroll
                            for (int dd = 0; dd < DP / 16; ++dd)
#pragma unroll
                                for (int ii = 0; ii < 4; ++ii)
                                    if (dd == d && ii == i) o[dd][ii] += p * v;
                        }
                    }
            }
        }
    }
    l_run += __shfl_xor(l_run, 16, 64);
    l_run += __shfl_xor(l_run, 32, 64);
    if (!live) return;
    if (a.splits == 1) {
        const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
        T* op = (T*)a.out + b * a.o_s[0] + qi * a.o_s[1] + hq * a.o_s[2];
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
            const int e = 16 * d + 4 * g;
            if (e < a.d) *(typename Vec<T>::v4*)(op + e) = from_f32<T>(o[d] * inv);
        }
        return;
    }
    const int64_t wr = ws_row(a, bh, split, row);
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) {
        const int e = 16 * d + 4 * g;
        if (e < a.d) *(f32x4*)(ws_out(a, wr) + e) = o[d];
    }
    if (g == 0) *ws_stat(a, wr) = f32x2{m_run, l_run};
}

// One wave per row: the splits' maxima and sums give each split's factor,
// then every lane adds up its elements over the splits.
template <typename T>
__global__ __launch_bounds__(256) void attention_join(AttnArgs a, uint32_t waves) {
    const uint32_t w = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (w >= waves) return;
    const int lane = threadIdx.x & 63;
    const int bh = (int)(w / (uint32_t)a.rows), row = (int)(w % (uint32_t)a.rows);
    const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
    const int qi = row / a.group, hq = hk * a.group + row % a.group;
    float top = -INFINITY;
    for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, (*ws_stat(a, ws_row(a, bh, s, row)))[0]);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    const float base = top == -INFINITY ? 0.0f : top;
    f32x4 sum{0, 0, 0, 0};
    float l = 0.0f;
    const int e = lane * 4;
    for (int s = 0; s < a.splits; ++s) {
        const int64_t wr = ws_row(a, bh, s, row);
        const f32x2 st = *ws_stat(a, wr);
        const float f = __builtin_amdgcn_exp2f(st[0] - base);
        l += f * st[1];
        if (e < a.d) sum += *(const f32x4*)(ws_out(a, wr) + e) * f;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T* op = (T*)a.out + b * a.o_s[0] + qi * a.o_s[1] + hq * a.o_s[2];
    if (e < a.d) *(typename Vec<T>::v4*)(op + e) = from_f32<T>(sum * inv);
}

template <typename T, int DP>
hipError_t run_any(const AttnArgs& a, hipStream_t s) {
    const int64_t blocks = (int64_t)a.batch * a.heads_kv * a.row_tiles * a.splits;
    attention_any<T, DP><<<dim3((uint32_t)blocks), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t run_any(const AttnArgs& a, hipStream_t s) {
    if (a.d <= 32) return run_any<T, 32>(a, s);
    if (a.d <= 64) return run_any<T, 64>(a, s);
    if (a.d <= 96) return run_any<T, 96>(a, s);
    if (a.d <= 128) return run_any<T, 128>(a, s);
    return run_any<T, 256>(a, s);
}

}  // namespace

hipError_t launch_attention_join(int32_t dtype, const AttnArgs& a, hipStream_t s) {
    const int64_t waves = (int64_t)a.batch * a.heads_kv * a.rows;
    if (waves > 0xfffffff0ll) return hipErrorInvalidValue;
    const dim3 grid((uint32_t)((waves + 3) / 4));
    if (dtype == CONV_DTYPE_F32)
        attention_join<float><<<grid, dim3(256), 0, s>>>(a, (uint32_t)waves);
    else
        attention_join<bf16><<<grid, dim3(256), 0, s>>>(a, (uint32_t)waves);
    return hipGetLastError();
}

AttnPlan plan_attention(int32_t dtype, const AttnArgs& a) {
    AttnPlan p{};
    // 64 keys within 32-bit byte offsets.
    const bool near = a.k_s[1] < 1 << 25 && a.v_s[1] < 1 << 25;
    p.kernel = dtype == CONV_DTYPE_BF16 && a.rows > 32 && near ? ATTN_TILE : ATTN_ANY;
    const int tile = p.kernel == ATTN_TILE ? 128 : 64;
    p.row_tiles = (a.rows + tile - 1) / tile;
    p.splits = 1;
    // Few row tiles leave compute units without work: the keys are then split
    // so that about two workgroups a unit run, each over 256 keys at least.
    const int64_t tiles = (int64_t)a.batch * a.heads_kv * p.row_tiles, want = 2 * (int64_t)device_cu_count();
    if (tiles < want) {
        int64_t s = (want + tiles - 1) / tiles;
        const int64_t most = ((int64_t)a.kv_len + 255) / 256;
        if (s > most) s = most;
        p.splits = s < 1 ? 1 : (int32_t)s;
    }
    if (p.splits > 1) p.ws_bytes = (int64_t)a.batch * a.heads_kv * p.splits * a.rows * (a.d + 2) * 4;
    return p;
}

hipError_t launch_attention(int32_t dtype, const AttnPlan& p, const AttnArgs& a, hipStream_t s) {
    const hipError_t e = p.kernel == ATTN_TILE           ? launch_attention_tile(a, s)
                         : dtype == CONV_DTYPE_F32 ? run_any<float>(a, s)
                                                   : run_any<bf16>(a, s);
    if (e != hipSuccess || p.splits == 1) return e;
    return launch_attention_join(dtype, a, s);
}

}  // namespace conv2d
