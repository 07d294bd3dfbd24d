/*
 * attention.h -- the operators of an attention layer in libconv2d.so, next to
 * the convolutions of conv2d.h, forward only, on one AMD Instinct MI355X:
 *
 *   linear_forward     matrix product with bias, activation and residual
 *   qk_rope_forward    norms of queries and keys for each head and the
 *                      position rotation in one pass, keys and values stored
 *                      to the rows of a cache
 *   attention_forward  softmax attention over contiguous or cached keys, with
 *                      capped scores, a distance bias, and length, causal,
 *                      window, prefix and document masks
 *
 * They follow conv2d.h: attributes are checked once, when a descriptor is
 * made; forward calls check their pointers and sizes, launch asynchronously on
 * the caller's HIP stream and allocate nothing; every call returns a
 * conv_status_t, never aborts, and conv2d_last_error() holds the detail of the
 * calling thread's last failure.  Descriptors own no device memory and are
 * not changed by forward calls, so one may be used from several streams and
 * threads at once.  Every call may be captured into a HIP graph.
 *
 * Element types are CONV_DTYPE_F32 and CONV_DTYPE_BF16 (I8 returns
 * UNSUPPORTED).  Sums, norms, angles and softmax statistics are held in fp32
 * or more for both; a bf16 result is rounded once, to nearest even.  In
 * attention_forward a bf16 call's softmax weights meet the values on the matrix
 * cores with 16 bits where at most 16 rows share a key head (q_len heads_q /
 * heads_kv: single tokens), rounded to bf16 beyond, and a capped score may be
 * off by softcap * 2^-21 up to a softcap of 512, by 2^-21 of itself beyond.
 * Strides count elements.
 */
#ifndef ATTENTION_MI355X_H
#define ATTENTION_MI355X_H

#include <stdint.h>

#include "conv2d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------- linear --- */

/* Activations of linear_forward besides conv_act_t's NONE, RELU, LEAKY_RELU
 * and CLIP (whose formulas and parameters are conv2d.h's; PRELU returns
 * UNSUPPORTED). */
typedef enum {
    LINEAR_ACT_SILU = 16,      /* v / (1 + exp(-v)) */
    LINEAR_ACT_GELU = 17,      /* v (1 + erf(v / sqrt 2)) / 2 */
    LINEAR_ACT_GELU_TANH = 18  /* v (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))) / 2 */
} linear_act_t;

typedef struct {
    int64_t x_stride, y_stride, residual_stride; /* row strides; 0 (default) means dense: k, n, n */
    int32_t k, n;              /* reduction length and output width, 1 .. 2^24 */
    int32_t has_bias;          /* 0/1, default 0 */
    int32_t has_residual;      /* 0/1, default 0 */
    int32_t act_type;          /* default CONV_ACT_NONE */
    float act_params[2];       /* as in conv2d_params_t (NaN selects the default) */
    int32_t dtype;             /* of x, w, residual and y; default CONV_DTYPE_F32 */
} linear_params_t;

typedef struct linear_desc* linear_desc_t;

CONV2D_API void linear_params_init(linear_params_t* p);

/* Errors: INVALID_ARG for a null pointer, a size outside its range, an unknown
 * activation or dtype, clip lo > hi or a non-finite leaky alpha;
 * INCOMPATIBLE_SHAPES for a row stride below the row's length; UNSUPPORTED for
 * PRELU and I8. */
CONV2D_API conv_status_t linear_desc_create(const linear_params_t* p, linear_desc_t* out);
CONV2D_API void linear_desc_destroy(linear_desc_t d);

/* Name of the kernel a call with `rows` rows of 16-byte aligned tensors runs
 * (static string; for logs). */
CONV2D_API const char* linear_desc_kernel_name(linear_desc_t d, int64_t rows);

/* y[i][o] = act(sum_c x[i][c] * w[o][c] + bias[o]) + residual[i][o] for
 * i < rows, o < n.
 *   x [rows][k], y and residual [rows][n] at their row strides; w [n][k]
 *   dense (the OIHW layout of a 1x1 convolution); bias float32[n], required
 *   iff has_bias; residual required iff has_residual.
 * Any alignment to the element size is accepted; rows that start at 16-byte
 * boundaries run faster.  y may be the residual itself (same pointer and
 * stride); any other overlap of y with an input returns ALIAS.  rows = 0
 * launches nothing.  INVALID_ARG for a null pointer, rows < 0 or > 2^31 - 1. */
CONV2D_API conv_status_t linear_forward(linear_desc_t d, int64_t rows, const void* x, const void* w,
                                        const float* bias, const void* residual, void* y, void* stream);

/* ------------------------------------------------------------ qk_rope --- */

typedef enum {
    ROPE_HALF = 0,        /* pair i is elements (i, i + rotary_dim/2) */
    ROPE_INTERLEAVED = 1  /* pair i is elements (2i, 2i + 1) */
} rope_layout_t;

/* Angle of pair i at position p: p * f_i, with f_i = theta^(-2i/rotary_dim)
 * scaled for contexts beyond the trained one:
 *   NONE    f_i
 *   LINEAR  f_i / factor
 *   YARN    f_i (1 - r_i) + f_i / factor * r_i, r_i = clamp((i - lo) /
 *           max(hi - lo, 0.001), 0, 1), where a pair that turns n times within
 *           original_len has the index t(n) = rotary_dim ln(original_len /
 *           (2 pi n)) / (2 ln theta), lo = max(floor t(beta_fast), 0) and
 *           hi = min(ceil t(beta_slow), rotary_dim - 1); the rotated elements
 *           are multiplied by attn_factor (Peng, Quesnelle, Fan and Shippole,
 *           "YaRN", 2023). */
typedef enum { ROPE_SCALING_NONE = 0, ROPE_SCALING_LINEAR = 1, ROPE_SCALING_YARN = 2 } rope_scaling_t;

typedef struct {
    int64_t qkv_stride;         /* token stride of qkv; 0 (default) means dense: (heads_q + 2 heads_kv) head_dim */
    int64_t q_stride;           /* token stride of q; 0 means heads_q * head_dim */
    int64_t k_stride, v_stride; /* row strides of k and v; 0 means heads_kv * head_dim */
    double theta;               /* > 1, default 10000 */
    double factor;              /* >= 1, default 1 */
    double beta_fast, beta_slow; /* > 0, defaults 32 and 1 */
    double attn_factor;         /* > 0; 0 (default) means 0.1 ln(factor) + 1 for YARN, else 1 */
    int32_t heads_q, heads_kv;  /* >= 1 */
    int32_t head_dim;           /* 1 .. 256 */
    int32_t rotary_dim;         /* even, <= head_dim; 0 (default) means head_dim */
    int32_t layout;             /* rope_layout_t, default ROPE_HALF */
    int32_t scaling;            /* rope_scaling_t, default NONE */
    int32_t original_len;       /* trained context of YARN, >= 1 there */
    int32_t has_norm;           /* 0/1, default 0 */
    float eps;                  /* >= 0, default 1e-6 */
    int32_t dtype;              /* of qkv, q, k and v; default CONV_DTYPE_F32 */
} qk_rope_params_t;

typedef struct qk_rope_desc* qk_rope_desc_t;

CONV2D_API void qk_rope_params_init(qk_rope_params_t* p);

/* Errors: INVALID_ARG for a null pointer or a value outside its range;
 * INCOMPATIBLE_SHAPES for rotary_dim > head_dim or a stride below its row's
 * length; UNSUPPORTED for I8 and head_dim > 256. */
CONV2D_API conv_status_t qk_rope_desc_create(const qk_rope_params_t* p, qk_rope_desc_t* out);
CONV2D_API void qk_rope_desc_destroy(qk_rope_desc_t d);

/* For each token t: qkv[t] holds heads_q query heads, then heads_kv key heads,
 * then heads_kv value heads of head_dim elements.  With has_norm a query or
 * key head x becomes gamma * x / sqrt(mean(x^2) + eps) (q_gamma, k_gamma
 * float32[head_dim], shared by the heads); its first rotary_dim elements are
 * then rotated, (a, b) -> (a cos - b sin, b cos + a sin), at positions[t]
 * (int32, any sign; the angle is reduced in fp64).  Queries go to q[t], keys
 * and values to rows slots[t] of k and v (t itself where slots is null).  A
 * slot outside [0, cache_rows) stores neither (a padding token); two tokens
 * must not share a slot.  v null: values are not stored.  attention_forward
 * reads a sequence's keys at one stride, so for it token i of sequence b goes to
 * a row first[b] + i (or first[b] + c i); rows of scattered pages are
 * paged_attention_forward's (decoder.h).
 * cache_rows is the number of rows of k and v (>= tokens where slots is null).
 * q may be qkv itself with q_stride == qkv_stride (in place); any other
 * overlap of an output with an input or another output returns ALIAS.
 * INVALID_ARG for a null pointer, tokens or cache_rows outside 0 .. 2^31 - 1;
 * INCOMPATIBLE_SHAPES for cache_rows < tokens without slots. */
CONV2D_API conv_status_t qk_rope_forward(qk_rope_desc_t d, int64_t tokens, const void* qkv, const float* q_gamma,
                                         const float* k_gamma, const int32_t* positions, const int32_t* slots,
                                         int64_t cache_rows, void* q, void* k, void* v, void* stream);

/* ---------------------------------------------------------- attention --- */

typedef struct {
    /* Strides of (batch, token, head) of each tensor; a head's head_dim
     * elements are contiguous.  Every stride is a multiple of 16 bytes, at
     * least 0 for the inputs (0 repeats one batch, token or head) and at
     * least head_dim for the output, each of whose strides reaches past what
     * the smaller ones span (any order of dimensions, any gaps). */
    int64_t q_strides[3], k_strides[3], v_strides[3], out_strides[3];
    int32_t heads_q, heads_kv;  /* heads_kv divides heads_q; query head h reads key head h / (heads_q / heads_kv) */
    int32_t head_dim;           /* <= 256, a multiple of 16 bytes */
    int32_t causal;             /* 0/1, default 0 */
    int32_t window;             /* > 0: keys at a distance below `window`; 0 (default): all */
    int32_t has_slopes;         /* 0/1, default 0 */
    float softcap;              /* > 0: scores become softcap * tanh(score / softcap); 0 (default): as they are */
    float scale;                /* factor on q.k; NaN (default) means 1 / sqrt(head_dim) */
    int32_t dtype;              /* of q, k, v and out; default CONV_DTYPE_F32 */
} attention_params_t;

typedef struct attention_desc* attention_desc_t;

CONV2D_API void attention_params_init(attention_params_t* p);

/* Errors: INVALID_ARG for a null pointer, a value outside its range or a
 * negative stride; INCOMPATIBLE_SHAPES for heads_kv not dividing heads_q or an
 * output stride below head_dim; UNSUPPORTED for I8, head_dim beyond 256 or not
 * a multiple of 16 bytes, and strides that are not multiples of 16 bytes. */
CONV2D_API conv_status_t attention_desc_create(const attention_params_t* p, attention_desc_t* out);
CONV2D_API void attention_desc_destroy(attention_desc_t d);

/* *bytes = the workspace a call of these sizes needs (0 where the keys are
 * not split over workgroups).  It depends on nothing else, and a larger
 * workspace serves too. */
CONV2D_API conv_status_t attention_workspace_bytes(attention_desc_t d, int64_t batch, int64_t q_len, int64_t kv_len,
                                                   int64_t* bytes);

/* Softmax attention of q [batch][q_len][heads_q][head_dim] over k, v
 * [batch][kv_len][heads_kv][head_dim] (prompts, or a cache filled up to each
 * sequence's length) into out [batch][q_len][heads_q][head_dim].
 *   q_lens, kv_lens  device int32[batch], or null for q_len, kv_len: the rows
 *                    of each sequence that count (clamped to [0, q_len] and
 *                    [0, kv_len])
 *   prefix_lens      device int32[batch] or null
 *   doc_offsets      device int32[batch][n_docs + 1], non-decreasing, or null:
 *                    document i of a sequence is keys [o[i], o[i+1])
 *   slopes           device float32[heads_q], required iff has_slopes
 * Query i of a sequence with Q queries and K keys is at position p = K - Q + i
 * (new tokens are the last ones of their cache).  It sees key j < K iff
 *   causal:       j <= p, or j < prefix_lens[b] where given;
 *   window:       |p - j| < window;
 *   doc_offsets:  p and j are in the same document (no document holds p: it
 *                 sees none).
 * Its score is s = scale * q.k, capped, minus slopes[h] * |p - j|.  Rows that
 * see no key, and rows from Q on, are zero.  Elements of k and v that a row
 * does not see do not reach it, whatever they hold; keys from K on are not
 * read at all.  An infinity that it sees makes that element of the row infinite
 * (NaN, as 0 * inf, where its weight is below fp32's range).
 *   workspace        at least attention_workspace_bytes, 16-byte aligned,
 *                    scratch of this call alone until it ends; may be null
 *                    where that is 0
 * Errors: INVALID_ARG for null or misaligned (16 bytes) pointers, negative
 * sizes, kv_len or q_len beyond 2^30 or a workspace that is too small;
 * UNSUPPORTED for a sequence of 2^24 workgroups and more (some 2^31 rows, all
 * heads together), and for more than 2^30 rows of a key head; ALIAS if rows of
 * out share memory, or if the bytes from out's first to its last element
 * overlap an input's or the workspace. */
CONV2D_API conv_status_t attention_forward(attention_desc_t d, int64_t batch, int64_t q_len, int64_t kv_len,
                                           const void* q, const void* k, const void* v, const int32_t* q_lens,
                                           const int32_t* kv_lens, const int32_t* prefix_lens,
                                           const int32_t* doc_offsets, int32_t n_docs, const float* slopes, void* out,
                                           void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTENTION_MI355X_H */
