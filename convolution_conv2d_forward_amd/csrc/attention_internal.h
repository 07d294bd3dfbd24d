// Internal declarations shared by the ABI layer of include/attention.h and its
// kernels.
#pragma once

#include "../../include/attention.h"
#include "conv2d_internal.h"

namespace conv2d {

// A launch counts its grid in work-items, in 32 bits: workgroups of `threads`
// threads that it may have.  Calls of more take several launches.
constexpr int64_t most_workgroups(int threads) { return 0xffffffffll / threads; }

// ------------------------------------------------------------- linear ----

struct LinearArgs {
    const void* x;
    const void* w;
    const float* bias;      // null when absent
    const void* residual;   // null when absent
    void* y;
    int64_t xs, ys, rs;     // row strides, elements
    int32_t m, k, n;
    int32_t act;
    float act_a, act_b;
    int32_t vec;            // 16 or 4: x and w rows start at boundaries of so many bytes, k fills whole pieces of them,
                            // and 256 rows lie within 32-bit byte offsets; 0: neither
    int32_t vec_out;        // 8 consecutive outputs of a row start at a 16-byte boundary in y and the residual
};

// Kernel of a call, by a rule on sizes alone.
const char* linear_kernel_name(int32_t dtype, const LinearArgs& a);
hipError_t launch_linear(int32_t dtype, const LinearArgs& a, hipStream_t s);

// ------------------------------------------------------------ qk_rope ----

constexpr int ROPE_MAX_PAIRS = 128;

struct RopeArgs {
    const void* qkv;
    const float* q_gamma;   // null without norm
    const float* k_gamma;
    const int32_t* positions;
    const int32_t* slots;   // null: row t
    void* q;
    void* k;
    void* v;                // null: not stored
    int64_t qkv_s, q_s, k_s, v_s;
    int64_t cache_rows;
    int32_t tokens, heads_q, heads_kv, d, r;
    float eps;
    float attn_factor;
    const double* turns;    // host: ROPE_MAX_PAIRS turns (angle / 2 pi) a position; the launch passes those in use by value
};

// vec: every row and head starts at a 16-byte boundary.
hipError_t launch_qk_rope(int32_t dtype, int32_t layout, bool vec, const RopeArgs& a, hipStream_t s);

// ---------------------------------------------------------- attention ----

struct AttnArgs {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    const int32_t* q_lens;
    const int32_t* kv_lens;
    const int32_t* prefix_lens;
    const int32_t* doc_offsets;
    const float* slopes;    // null without
    float* ws;              // partial results, null when splits == 1
    int64_t q_s[3], k_s[3], v_s[3], o_s[3];
    int32_t batch, q_len, kv_len, heads_q, heads_kv, group, d;
    int32_t causal, window, n_docs;
    int32_t rows;           // q_len * group: the rows that share one key head
    int32_t row_tiles, splits;
    float scale;            // on q.k
    float softcap;          // 0: none
};

// Kernels of attention_forward: any strides, few rows for each key head, or
// many.
enum attn_kernel_t { ATTN_ANY, ATTN_ROWS, ATTN_TILE_128, ATTN_TILE_64 };

constexpr int ATTN_MAX_SPLITS = 256;   // a join workgroup takes one a thread

// Workgroups and split of the keys that a call of these sizes runs with.
struct AttnPlan {
    attn_kernel_t kernel;
    int32_t row_tiles, splits;
    int64_t ws_bytes;
};

// Workgroups of each sequence.
inline int64_t sequence_workgroups(const AttnArgs& a, const AttnPlan& p) {
    return (int64_t)a.heads_kv * p.row_tiles * p.splits;
}

hipError_t launch_attention_rows(int32_t dtype, const AttnArgs& a, hipStream_t s);
AttnPlan plan_attention(int32_t dtype, const AttnArgs& a);
hipError_t launch_attention(int32_t dtype, const AttnPlan& p, const AttnArgs& a, hipStream_t s);

}  // namespace conv2d
