// Softmax attention of few rows: single tokens, and a few drafted ones, over
// long caches.
#include "attention_common.h"
#include "linear_common.h"

namespace conv2d {

namespace {

// 16 of the rows (query i, head of the group) that share a key head
// per workgroup.  It is bound by the bytes of K and V, so every wave reads
// tiles of 32 keys (or 16) of its own, straight from memory into the operands of the
// matrix cores, with the next tile's loads in flight, and no LDS or barrier
// stands between; the waves' results meet in LDS once, at the end, and the
// splits' in the workspace.
//
// S^T = K Q^T in 16x16 steps, lane l holding 16 bytes of key row l & 15.  In
// bf16 the key rows of a step are taken in the order that leaves lane group g
// with the scores of keys 8 g .. 8 g + 7, in order; in fp32 group g gets keys
// 4 g + i of each 16.  For O^T = V^T P^T a lane reads one 16-byte chunk of V's
// row for each of its group's keys, so that a load takes whole rows: in bf16
// eight rows' chunks become eight operands (chunk c's element j of all eight
// keys: output 8 c + j) by byte permutes, in fp32 they are operands as they
// are.
template <typename T, int DP>
struct RowsAttn {
    static constexpr int C = Vec<T>::chunk;
    static constexpr int KS = DP * (int)sizeof(T) / 64;               // 64-byte product steps over a row
    static constexpr int VC = (DP / C + 15) / 16;                     // 16-chunk groups of a row of V
    // Keys of a tile: rows of 1024 bytes spilled at 32 (8x4096 keys of 8 heads of
    // 256 fp32: 157 us, 128 at 16; one token over 25 keys: 18.4 and 12.5).
    static constexpr int BK = DP * (int)sizeof(T) > 512 ? 16 : 32, NT = BK / 16, NJ = BK / 4;
    static constexpr int OUT = VC * C;                                // 16x16 output blocks
    // A tile takes a quarter of the row's bytes in registers: rows to 256 bytes
    // leave room for two waves on a SIMD, each with two tiles.  Two tiles of
    // 256 bf16 leave no register (16x4096 keys: 128 us, 110 with one); of 128
    // fp32, without the permutes, they pay (115, 122 with one).
    static constexpr int RB = DP * (int)sizeof(T), NBUF = DP <= 128 ? 2 : 1, OCC = RB <= 256 ? 2 : 1, NW = 4;
    u32x4 k[NT][KS];
    u32x4 v[NJ][VC];

    // A tile's loads.  Keys from nk on repeat the last one.
    __device__ __forceinline__ void load(const T* kp, const T* vp, int64_t ks, int64_t vs, int k0, int nk, int d,
                                         int lane) {
        const int r = lane & 15, g = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int key = sizeof(T) == 2 ? 8 * (r >> 2) + 4 * t + (r & 3) : 16 * t + r;
            const T* p = kp + min(k0 + key, nk - 1) * ks;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int e = (4 * s + g) * C;
                k[t][s] = u32x4{0, 0, 0, 0};
                if (e < d) k[t][s] = *(const u32x4*)(p + e);
            }
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int key = sizeof(T) == 2 ? 8 * g + j : 16 * (j >> 2) + 4 * g + (j & 3);
            const T* p = vp + min(k0 + key, nk - 1) * vs;
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                const int e = (16 * c + r) * C;
                v[j][c] = u32x4{0, 0, 0, 0};
                if (e < d) v[j][c] = *(const u32x4*)(p + e);
            }
        }
    }
};

// The i-th longest sequence (of up to 64; else, and without lengths, i).
__device__ __forceinline__ int by_length(const AttnArgs& a, int i, int lane) {
    if (!a.kv_lens || a.batch > 64) return i;
    const int mine = lane < a.batch ? a.kv_lens[lane] : 0;
    int rank = 0;
    for (int j = 0; j < a.batch; ++j) {
        const int other = __builtin_amdgcn_readlane(mine, j);
        rank += other > mine || (other == mine && j < lane);
    }
    const uint64_t hit = __ballot(lane < a.batch && rank == i);
    return __builtin_amdgcn_readfirstlane((int)__builtin_ctzll(hit));
}

template <typename T, int DP>
__global__ __launch_bounds__((64 * RowsAttn<T, DP>::NW), (RowsAttn<T, DP>::OCC)) void attention_rows(AttnArgs a) {
    typedef RowsAttn<T, DP> R;
    constexpr int C = R::C, KS = R::KS, VC = R::VC, NW = R::NW, BK = R::BK, NT = R::NT, NJ = R::NJ, OUT = R::OUT;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    // Sequence, key head, split, row tile: with the longest sequences first,
    // whose workgroups take longest, the short ones fill the gaps at the end.
    uint32_t blk = blockIdx.x;
    const int hk = (int)(blk % (uint32_t)a.heads_kv);
    blk /= (uint32_t)a.heads_kv;
    const int split = (int)(blk % (uint32_t)a.splits);
    blk /= (uint32_t)a.splits;
    const int tile_r = (int)(blk % (uint32_t)a.row_tiles), b = by_length(a, (int)(blk / (uint32_t)a.row_tiles), lane);
    const int bh = b * a.heads_kv + hk;
    const SeqLens sl = seq_lens(a, b);
    const ScoreP sp = score_params(a);

    const int row = tile_r * 16 + r;
    const bool live = row < a.rows;
    const int qi = live ? row / a.group : 0, hq = hk * a.group + (live ? row - qi * a.group : 0);
    int lo = 0, hi = 0;
    row_interval(a, sl, b, qi, live, lo, hi);
    const bool empty = hi <= lo;
    int w_lo = empty ? INT32_MAX : lo, w_hi = hi;                                    // keys that some row sees
    int f_lo = live ? (empty ? INT32_MAX : lo) : 0, f_hi = live ? hi : INT32_MAX;    // keys that every row sees
    const int pos = sl.nk - sl.nq + qi;
    const float slope = a.slopes && live ? a.slopes[hq] * kLog2e : 0.0f;
    u32x4 fq[KS];
    const T* qp = (const T*)a.q + b * a.q_s[0] + qi * a.q_s[1] + hq * a.q_s[2];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const int e = (4 * s + g) * C;
        fq[s] = u32x4{0, 0, 0, 0};
        if (live && e < a.d) fq[s] = *(const u32x4*)(qp + e);
    }
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {
        w_lo = min(w_lo, __shfl_xor(w_lo, m, 64));
        w_hi = max(w_hi, __shfl_xor(w_hi, m, 64));
        f_lo = max(f_lo, __shfl_xor(f_lo, m, 64));
        f_hi = min(f_hi, __shfl_xor(f_hi, m, 64));
    }
    w_lo = __builtin_amdgcn_readfirstlane(min(w_lo, w_hi));
    w_hi = __builtin_amdgcn_readfirstlane(w_hi);
    f_lo = __builtin_amdgcn_readfirstlane(f_lo);
    f_hi = __builtin_amdgcn_readfirstlane(f_hi);

    // The tiles of this split, dealt to the waves.
    const int t0 = w_lo / BK, tn = (w_hi + BK - 1) / BK - t0;
    const int first = __builtin_amdgcn_readfirstlane(t0 + (int)((int64_t)tn * split / a.splits));
    const int last = __builtin_amdgcn_readfirstlane(t0 + (int)((int64_t)tn * (split + 1) / a.splits));
    const T* kp = (const T*)a.k + b * a.k_s[0] + hk * a.k_s[2];
    const T* vp = (const T*)a.v + b * a.v_s[0] + hk * a.v_s[2];

    f32x4 o[OUT] = {};
    float m_run = -INFINITY, l_run = 0.0f;
    const auto step = [&](R& f, int tile) {
        const int k0 = tile * BK;
        const bool whole = k0 >= f_lo && k0 + BK <= f_hi;
        // Infinities and NaN in values that some row does not see: zeros go
        // into the product, and the rows that see them get them one by one.
        bool bad = false;
        if (!whole) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int c = 0; c < VC; ++c) bad |= has_bad<T>(f.v[j][c]);
            bad = __ballot(bad) != 0;
        }
        if (bad) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int c = 0; c < VC; ++c) clean_chunk<T>(f.v[j][c]);
        }
        float p[NT][4];
        f32x4 s[NT] = {};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < KS; ++i) s[t] = mfma_step<T>(f.k[t][i], fq[i], s[t]);
        float top = -INFINITY, sc[4 * NT];
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) sc[i] = s[i >> 2][i & 3];
        scores<T>(sp, sc);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = k0 + (sizeof(T) == 2 ? 8 * g + 4 * t + i : 16 * t + 4 * g + i);
                float x = sc[4 * t + i];
                if (a.slopes) x -= slope * fabsf((float)(pos - key));
                if (!whole) x = key >= lo && key < hi ? x : -INFINITY;
                s[t][i] = x;
                top = fmaxf(top, x);
            }
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float m_new = fmaxf(m_run, top), base = m_new == -INFINITY ? 0.0f : m_new;
        const float fade = __builtin_amdgcn_exp2f(m_run - base);
        m_run = m_new;
        l_run *= fade;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[t][i] = __builtin_amdgcn_exp2f(s[t][i] - base);
                l_run += p[t][i];
            }
#pragma unroll
        for (int d = 0; d < OUT; ++d) o[d] *= fade;
        if constexpr (sizeof(T) == 2) {
            // The weights as a bf16 number and what it leaves, so 16 bits of
            // them: the products wait for memory, not the matrix cores for
            // them (16x4096 keys of 8 heads of 128: 62.1 us, 60.6 without;
            // 28x30 of 12 heads of 256: 19.4 and 18.9).  Both parts of a
            // weight are above zero (the first is cut off, the second gets
            // 2^-20 of the weight more), or a seen infinity would meet a zero
            // or both signs and become NaN.
            bf16x8 fp, fl;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = p[i >> 2][i & 3];
                const float cut = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, w) & 0xffff0000u);
                fp[i] = (bf16)cut;
                fl[i] = (bf16)__builtin_fmaf(w, 0x1p-20f, w - cut);
            }
#pragma unroll
            for (int c = 0; c < VC; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    u32x4 w;   // element e of this lane's chunk, for the group's eight keys
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = __builtin_amdgcn_perm(f.v[2 * j + 1][c][e >> 1], f.v[2 * j][c][e >> 1],
                                                     e & 1 ? 0x07060302u : 0x05040100u);
                    o[c * 8 + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), fp,
                                                                              o[c * 8 + e], 0, 0, 0);
                    o[c * 8 + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), fl,
                                                                              o[c * 8 + e], 0, 0, 0);
                }
        } else {
#pragma unroll
            for (int c = 0; c < VC; ++c)
#pragma unroll
                for (int e = 0; e < C; ++e)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        o[c * C + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            __builtin_bit_cast(f32x4, f.v[j][c])[e], p[j >> 2][j & 3], o[c * C + e], 0, 0, 0);
        }
        if (bad) {
            // Output block (c, e) of lane l has rows 16 c C + (4 (l / 16) + i) C + e of V^T.
            for (int j = 0; j < NJ; ++j)
#pragma unroll 1
                for (int gg = 0; gg < 4; ++gg) {
                    const int key = k0 + (sizeof(T) == 2 ? 8 * gg + j : 16 * (j >> 2) + 4 * gg + (j & 3));
                    if (key >= sl.nk) continue;
                    const T* v = vp + key * a.v_s[1];
#pragma unroll
                    for (int c = 0; c < VC; ++c)
#pragma unroll
                        for (int e = 0; e < C; ++e)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int at = (16 * c + 4 * g + i) * C + e;
                                const float x = at < a.d ? to_f32(v[at]) : 0.0f;
                                if (!(fabsf(x) < INFINITY))
                                    if (key >= lo && key < hi) o[c * C + e][i] += x;
                            }
                }
        }
    };
    const auto load = [&](R& f, int tile) {
        if (tile < last) f.load(kp, vp, a.k_s[1], a.v_s[1], tile * BK, sl.nk, a.d, lane);
    };
    if constexpr (R::NBUF == 2) {
        R f[2];
        load(f[0], first + wave);
        for (int tile = first + wave; tile < last; tile += 2 * NW) {
            load(f[1], tile + NW);
            step(f[0], tile);
            load(f[0], tile + 2 * NW);
            if (tile + NW < last) step(f[1], tile + NW);
        }
    } else {
        for (int tile = first + wave; tile < last; tile += NW) {
            R f;
            load(f, tile);
            step(f, tile);
        }
    }

    // The waves' results: the maxima and sums first, then the outputs at the
    // common maximum.  Wave w adds up output blocks w, w + NW ...
    __shared__ f32x2 stat[NW][16];
    __shared__ __align__(16) f32x4 part[NW][OUT][64];
    l_run += __shfl_xor(l_run, 16, 64);
    l_run += __shfl_xor(l_run, 32, 64);
    if (g == 0) stat[wave][r] = f32x2{m_run, l_run};
    __syncthreads();
    float top = -INFINITY, total = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, stat[w][r][0]);
    const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < NW; ++w) total += __builtin_amdgcn_exp2f(stat[w][r][0] - base) * stat[w][r][1];
    const float fade = __builtin_amdgcn_exp2f(m_run - base);
#pragma unroll
    for (int d = 0; d < OUT; ++d) part[wave][d][lane] = o[d] * fade;
    __syncthreads();
    if (!live) return;
    T* op = (T*)a.out + b * a.o_s[0] + qi * a.o_s[1] + hq * a.o_s[2];
    const int64_t wr = a.splits == 1 ? 0 : ws_row(a, bh, split, row);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    // A lane's chunk c of its row i: C consecutive outputs, one of each of C blocks.
    for (int ci = wave; ci < VC * 4; ci += NW) {
        const int c = ci >> 2, i = ci & 3, at = (16 * c + 4 * g + i) * C;
        if (at >= a.d) continue;
        float v[C];
#pragma unroll
        for (int e = 0; e < C; ++e) {
            v[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) v[e] += ((const float*)&part[w][c * C + e][lane])[i];
        }
        if (a.splits == 1) {
            T y[C];
#pragma unroll
            for (int e = 0; e < C; ++e) y[e] = from_f32<T>(v[e] * inv);
            __builtin_memcpy(op + at, y, 16);
        } else {
#pragma unroll
            for (int e = 0; e < C; ++e) ws_out(a, wr)[at + e] = v[e];
        }
    }
    if (a.splits > 1 && wave == 0 && g == 0) *ws_stat(a, wr) = f32x2{top, total};
}

template <typename T, int DP>
hipError_t run(const AttnArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)((int64_t)a.batch * a.heads_kv * a.row_tiles * a.splits)), block(256);
    attention_rows<T, DP><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t run(const AttnArgs& a, hipStream_t s) {
    if (a.d <= 32) return run<T, 32>(a, s);
    if (a.d <= 64) return run<T, 64>(a, s);
    if (a.d <= 96) return run<T, 96>(a, s);
    if (a.d <= 128) return run<T, 128>(a, s);
    return run<T, 256>(a, s);
}

}  // namespace

hipError_t launch_attention_rows(int32_t dtype, const AttnArgs& a, hipStream_t s) {
    return dtype == CONV_DTYPE_F32 ? run<float>(a, s) : run<bf16>(a, s);
}

}  // namespace conv2d
