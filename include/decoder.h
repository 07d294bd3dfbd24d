/*
 * decoder.h -- what a decoder layer needs beside the operators of attention.h
 * to be served from a paged cache, in libconv2d.so, forward only, on one AMD
 * Instinct MI355X:
 *
 *   kv_cache_store           keys and values of new tokens to pages, quantised
 *                            to 8 bits or as they are
 *   kv_cache_load            sequences read back from their pages
 *   paged_attention_forward  softmax attention of each sequence's new tokens
 *                            (single ones, chunks of prompts, both in a batch)
 *                            over its pages, with a sliding window and first
 *                            tokens that stay visible
 *   block_norm_forward       the norm behind a block, its gate and the scaled
 *                            residual, and the norm before the next block
 *
 * They follow attention.h: attributes are checked once, when a descriptor is
 * made; calls check their pointers and sizes, launch asynchronously on the
 * caller's HIP stream and allocate nothing; every call returns a
 * conv_status_t, never aborts, and conv2d_last_error() holds the detail of the
 * calling thread's last failure.  Descriptors own no device memory and are not
 * changed by calls.  Every call may be captured into a HIP graph.  Strides
 * count elements.
 *
 * A paged cache is `n_pages` pages of `page_size` tokens, heads_kv heads and
 * head_dim elements, for keys and for values, in any order of these
 * dimensions; a head's elements are contiguous.  Slot s is token s % page_size
 * of page s / page_size.  A sequence's page table lists its pages in order:
 * its token i lies in page table[i / page_size], at i % page_size.  Pages of
 * the call's own type that are dense ([page][token][head][element]) are also
 * the rows that qk_rope_forward stores to, row s being slot s.
 *
 * Cache types: the call's own dtype (CONV_DTYPE_F32 or CONV_DTYPE_BF16), or
 * KV_CACHE_E4M3: a code of 8 bits an element (1 sign, 4 exponent, 3 mantissa
 * bits; largest number 448, no infinities) and a scale byte a token and head,
 * so that an element is code * 2^(scale - 127).  Elements dequantised with the
 * scales that kv_cache_store writes (10 .. 246) are exact in either dtype; other
 * scales are not for these operators.  kv_cache_store and kv_cache_load take heads
 * of any width, paged_attention_forward those whose rows in the pages are multiples
 * of 16 bytes (16 codes).
 */
#ifndef DECODER_MI355X_H
#define DECODER_MI355X_H

#include <stdint.h>

#include "attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------- kv_cache --- */

/* Cache types besides the call's own conv_dtype_t. */
typedef enum { KV_CACHE_E4M3 = 16 } kv_cache_dtype_t;

typedef struct {
    int64_t k_stride, v_stride;             /* token strides of k and v; 0 (default): heads_kv * head_dim */
    int64_t k_batch_stride, v_batch_stride; /* kv_cache_load: sequence strides; 0 (default): kv_len tokens */
    int64_t k_page_strides[3];              /* (page, token, head) of the pages; all 0 (default): dense, */
    int64_t v_page_strides[3];              /*   [page][token][head][element] */
    int64_t scale_strides[3];               /* of both scales; all 0 (default): dense, [page][token][head] */
    int32_t heads_kv;                       /* 1 .. 2^16 */
    int32_t head_dim;                       /* 1 .. 256 */
    int32_t page_size;                      /* 1 .. 2^16 */
    int32_t dtype;                          /* of k and v; default CONV_DTYPE_F32 */
    int32_t cache_dtype;                    /* default CONV_DTYPE_F32 */
} kv_cache_params_t;

typedef struct kv_cache_desc* kv_cache_desc_t;

CONV2D_API void kv_cache_params_init(kv_cache_params_t* p);

/* Errors: INVALID_ARG for a null pointer or a value outside its range;
 * INCOMPATIBLE_SHAPES for a stride below what it has to span; UNSUPPORTED for
 * I8, head_dim > 256, and a cache_dtype that is neither dtype nor E4M3. */
CONV2D_API conv_status_t kv_cache_desc_create(const kv_cache_params_t* p, kv_cache_desc_t* out);
CONV2D_API void kv_cache_desc_destroy(kv_cache_desc_t d);

/* Stores k, v [tokens][heads_kv][head_dim] to slots[t] (device int32) of the
 * pages.  A slot outside [0, n_pages * page_size) stores nothing (a padding
 * token); two tokens must not share a slot.  To E4M3, for each token and head:
 * with a the largest of the finite |x_i|, e the least integer with
 * a <= 448 * 2^e, clamped to [-117, 119], code_i = x_i / 2^e rounded once, to
 * nearest even (at most 448: of rows beyond 448 * 2^119 = 2.98e38, so that no
 * finite element is read back as an infinity), and the scale byte is e + 127.
 * Infinities and NaN become NaN.  k_scales and v_scales are required iff the
 * cache is E4M3.
 * Errors: INVALID_ARG for a null or misaligned (element size) pointer, tokens
 * or n_pages * page_size outside 0 .. 2^31 - 1; UNSUPPORTED for a tensor beyond
 * 2^44 elements; ALIAS for pages or scales that overlap an input or each other,
 * or whose own elements share memory.  Keys, values and scales may lie in one
 * buffer, page by page, or in any order (beside each other for each token or head,
 * say) where their strides are the same in bytes; pages of different strides that
 * lie in each other's gaps otherwise count as overlapping. */
CONV2D_API conv_status_t kv_cache_store(kv_cache_desc_t d, int64_t tokens, const void* k, const void* v,
                                        const int32_t* slots, int64_t n_pages, void* k_pages, void* v_pages,
                                        uint8_t* k_scales, uint8_t* v_scales, void* stream);

/* Reads tokens 0 .. kv_lens[b] - 1 of sequence b from the pages that
 * page_table [batch][max_pages] (device int32) lists, into rows of k and v
 * [batch][kv_len][heads_kv][head_dim] (what attention_forward reads).  Lengths
 * are clamped to [0, min(kv_len, max_pages * page_size)]; kv_lens null: all of
 * that.  Rows from a sequence's length on, and rows of pages outside
 * [0, n_pages), are left as they were.
 * Errors: as kv_cache_store's, with kv_len and max_pages * page_size up to
 * 2^30; ALIAS also for rows of k or v that share memory; k and v may lie beside
 * each other row by row at the same strides. */
CONV2D_API conv_status_t kv_cache_load(kv_cache_desc_t d, int64_t batch, int64_t kv_len, int64_t max_pages,
                                       const int32_t* page_table, const int32_t* kv_lens, int64_t n_pages,
                                       const void* k_pages, const void* v_pages, const uint8_t* k_scales,
                                       const uint8_t* v_scales, void* k, void* v, void* stream);

/* ---------------------------------------------------- paged attention --- */

typedef struct {
    int64_t q_stride, out_stride;  /* token strides; 0 (default): heads_q * head_dim */
    int64_t k_page_strides[3];     /* (page, token, head); all 0 (default): dense; 0 repeats otherwise */
    int64_t v_page_strides[3];
    int64_t scale_strides[3];      /* of both scales; all 0 (default): dense */
    int32_t heads_q, heads_kv;     /* heads_kv divides heads_q; query head h reads key head h / (heads_q / heads_kv) */
    int32_t head_dim;              /* <= 256; a row of a head in q and in the pages is a multiple of 16 bytes */
    int32_t page_size;             /* 1 .. 2^16 */
    int32_t window;                /* > 0: keys at a distance below `window`; 0 (default): all */
    int32_t sinks;                 /* >= 0, default 0: keys 0 .. sinks - 1 are seen beyond the window too */
    float softcap;                 /* > 0: scores become softcap * tanh(score / softcap); 0 (default): as they are */
    float scale;                   /* factor on q.k; NaN (default) means 1 / sqrt(head_dim) */
    int32_t dtype;                 /* of q and out; default CONV_DTYPE_F32 */
    int32_t cache_dtype;           /* default CONV_DTYPE_F32 */
} paged_attention_params_t;

typedef struct paged_attention_desc* paged_attention_desc_t;

CONV2D_API void paged_attention_params_init(paged_attention_params_t* p);

/* Errors: INVALID_ARG for a null pointer, a value outside its range or a
 * negative stride; INCOMPATIBLE_SHAPES for heads_kv not dividing heads_q or a
 * token stride below its row; UNSUPPORTED for I8, head_dim beyond 256 or not
 * such a multiple, strides that are not multiples of 16 bytes (the scales' may
 * be any), and a cache_dtype that is neither dtype nor E4M3. */
CONV2D_API conv_status_t paged_attention_desc_create(const paged_attention_params_t* p, paged_attention_desc_t* out);
CONV2D_API void paged_attention_desc_destroy(paged_attention_desc_t d);

/* *bytes = the workspace a call of these sizes needs (0 where none).  It
 * depends on nothing else, and a larger workspace serves too. */
CONV2D_API conv_status_t paged_attention_workspace_bytes(paged_attention_desc_t d, int64_t tokens, int64_t batch,
                                                         int64_t max_pages, int64_t* bytes);

/* Softmax attention of the new tokens q [tokens][heads_q][head_dim] of `batch`
 * sequences over their pages, into out (of q's shape).
 *   q_offsets   device int32[batch + 1]: sequence b's new tokens are rows
 *               q_offsets[b] .. q_offsets[b + 1] - 1 of q (both clamped to
 *               [0, tokens]; none where they do not ascend)
 *   kv_lens     device int32[batch]: its tokens in the cache, the new ones
 *               among them (clamped to [0, max_pages * page_size])
 *   page_table  device int32[batch][max_pages]
 * New token i of a sequence with Q of them and K tokens is at position
 * p = K - Q + i and sees key j <= p iff there is no window, or p - j < window,
 * or j < sinks.  Keys on pages outside [0, n_pages) are seen by no row, and
 * are not read.  Scores are scale * q.k, capped.  Rows that see no key are
 * zero.  Rows of out that belong to no sequence are left as they were; two
 * sequences must not share rows.  Elements of k and v that a row does not see
 * do not reach it, whatever they and their scales hold.  An infinity that a row sees
 * makes that element of the row infinite (NaN, as 0 * inf, where its weight is
 * below fp32's range).
 *   workspace   at least paged_attention_workspace_bytes, 16-byte aligned,
 *               scratch of this call alone until it ends; may be null where
 *               that is 0
 * Sums and softmax statistics are held in fp32; in bf16 the weights meet the
 * values with 16 bits in sequences of at most 16 rows of a key head (new tokens *
 * heads_q / heads_kv: single tokens, above all), whatever else is in the batch,
 * and in all of them where tokens * heads_q / heads_kv <= 16 * min(batch,
 * tokens); rounded to bf16 elsewhere.  A capped score is off as
 * attention_forward's is.
 * Errors: INVALID_ARG for a null or misaligned pointer (16 bytes; lengths,
 * offsets and the table 4), a negative size, tokens or batch beyond 2^30,
 * max_pages * page_size beyond 2^30, or a workspace that is too small;
 * UNSUPPORTED for more than 2^30 rows of a key head and pages that reach beyond
 * 2^36 bytes (their scales: 2^32); ALIAS if out overlaps an input or the
 * workspace, or the workspace an input. */
CONV2D_API conv_status_t paged_attention_forward(paged_attention_desc_t d, int64_t tokens, int64_t batch,
                                                 int64_t max_pages, const void* q, const int32_t* q_offsets,
                                                 const int32_t* kv_lens, const int32_t* page_table, int64_t n_pages,
                                                 const void* k_pages, const void* v_pages, const uint8_t* k_scales,
                                                 const uint8_t* v_scales, void* out, void* workspace,
                                                 int64_t workspace_bytes, void* stream);

/* --------------------------------------------------------- block norm --- */

/* x is a row of n elements, m its mean:
 *   RMS    gamma * x / sqrt(mean(x^2) + eps) + beta
 *   LAYER  gamma * (x - m) / sqrt(mean((x - m)^2) + eps) + beta */
typedef enum { BLOCK_NORM_NONE = 0, BLOCK_NORM_RMS = 1, BLOCK_NORM_LAYER = 2 } block_norm_kind_t;

typedef struct {
    int64_t y_stride, x_stride, residual_stride, out_stride, gate_stride; /* row strides; 0 (default): width */
    int32_t width;                 /* elements of a row, 1 .. 32768 */
    int32_t post_norm, pre_norm;   /* block_norm_kind_t, default NONE */
    int32_t has_post_beta, has_pre_beta; /* 0/1, default 0 */
    int32_t has_gate;              /* 0/1, default 0 */
    int32_t gate_rows;             /* rows that share a row of the gate; 0 (default): all do */
    float residual_scale, block_scale; /* finite, default 1 */
    float eps;                     /* >= 0, default 1e-6 */
    int32_t dtype;                 /* of y, x, gate, residual and out; default CONV_DTYPE_F32 */
} block_norm_params_t;

typedef struct block_norm_desc* block_norm_desc_t;

CONV2D_API void block_norm_params_init(block_norm_params_t* p);

/* Errors: INVALID_ARG for a null pointer or a value outside its range (a beta
 * without its norm); INCOMPATIBLE_SHAPES for a row stride below width;
 * UNSUPPORTED for I8 and width beyond 32768. */
CONV2D_API conv_status_t block_norm_desc_create(const block_norm_params_t* p, block_norm_desc_t* out);
CONV2D_API void block_norm_desc_destroy(block_norm_desc_t d);

/* For each row i < rows of a block's output y and of the residual stream x:
 *   r = residual_scale * x[i] + block_scale * gate[i / gate_rows] * post(y[i])
 *   residual[i] = r,  out[i] = pre(r)
 * with the norms post and pre (NONE: as it is), r unrounded in pre.  post_gamma
 * and pre_gamma float32[width], required iff there is that norm; the betas
 * float32[width], required iff they are set; gate [ceil(rows / gate_rows)]
 * [width], required iff has_gate; out required iff there is a pre norm, and
 * unused otherwise.  Sums are fp32, LAYER's around the row's mean; where a row's
 * squares or their sum would leave fp32's range, the row is scaled for them by a
 * power of two.
 * residual may be x or y itself (same pointer and stride), out may be y itself;
 * any other overlap of residual or out with an input or with each other returns
 * ALIAS.  INVALID_ARG for a null or misaligned pointer, rows < 0 or > 2^31 - 1;
 * UNSUPPORTED for a tensor beyond 2^44 elements. */
CONV2D_API conv_status_t block_norm_forward(block_norm_desc_t d, int64_t rows, const void* y, const void* x,
                                            const void* gate, const float* post_gamma, const float* post_beta,
                                            const float* pre_gamma, const float* pre_beta, void* residual, void* out,
                                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DECODER_MI355X_H */
