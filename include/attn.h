/*
 * attn.h -- C ABI of softmax attention with grouped heads: over packed samples (forward
 * and backward), and of new tokens over a paged key/value cache (part of librope_qk.so).
 *
 * The operation.  For query row i and the keys j it sees, with G = n_q_heads /
 * n_kv_heads query heads sharing a key/value head:
 *
 *     s_ij = scale * q_i . k_j       lse_i = log sum_j exp(s_ij)
 *     o_i  = sum_j exp(s_ij - lse_i) v_j
 *
 * A row that sees no key has o = 0 and lse = -infinity.  The backward, with
 * p_ij = exp(s_ij - lse_i), D_i = do_i . o_i, and ds_ij = p_ij (do_i . v_j - D_i):
 *
 *     dq_i = scale sum_j ds_ij k_j     dk_j = scale sum_i ds_ij q_i     dv_j = sum_i p_ij do_i
 *
 * where dk and dv sum over the G query heads of their key head too.
 *
 * Arithmetic.  bf16 in, bf16 out, one rounding to nearest even at the end.  Products
 * accumulate in binary32; scores, maxima, sums, lse and D stay in binary32.  The weights p
 * (forward and dv) and the ds (dq, dk) are rounded to bf16 once where they enter a product:
 * relative error at most 2^-8 of each term, as the final rounding.  D is taken from out as it
 * was rounded, except where all keys of a row are in one tile of 128.  The backward has p from
 * lse, and lse is binary32: p is off by up to |lse| 2^-22 of itself, which stays below its
 * rounding to bf16 while |lse| does below 2^14.  Results do not depend on launch timing: no
 * atomics, the same bits each run.
 *
 * Values.  Rows of other samples, rows beyond seq_used or outside the pack, and slots of
 * the cache beyond a sequence's length may hold anything, NaN and infinities among it, and
 * reach no result.  Within a sample, a key that a causal row does not see has weight zero
 * in it, but its value row is a factor of the product: keys, values and output gradients
 * of a sample's own rows are expected to be finite, and queries in the backward.  A NaN or a
 * score above binary32's range, from a query or from a key that the row sees, makes the
 * row's out and lse NaN, however the keys are split; scores that are all -infinity weigh
 * nothing, as if the row saw no key.
 *
 * Layout.  q, k, v, out and the gradients are bf16 views [total_tokens, heads, head_dim],
 * head_dim contiguous, with token and head strides in elements (multiples of 8, pointers
 * 16-byte aligned, no two rows of a view sharing an element), e.g. the slices of one fused
 * QKV projection output.  head_dim is a multiple of 16 in [16, 128]; n_q_heads a multiple
 * of n_kv_heads, at most 128 query heads to a key head.  Outputs share no address range
 * with inputs (or interleave with them, as the slices of one buffer do).
 *
 * Ownership, streams, errors as in rope_qk.h: device pointers owned by the caller, no
 * allocation, asynchronous on `stream`, ROPE_OK or a negative rope_status, checked on the
 * host before anything is launched.  Values inside cu_seqlens, seq_used, kv_lens and the
 * page table are not read on the host; with invalid ones the kernels stay inside the
 * buffers.  Every wait inside a kernel is bounded: attn_fault reports one that ran out.
 */
#ifndef ATTN_H
#define ATTN_H

#include <stdint.h>

#include "paged_kv.h"
#include "rope_qk.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Attention within each sample of a pack.  cu_seqlens (device int32 [n_seqs + 1]) and the
 * optional seq_used (device int32 [n_seqs]) delimit the samples as for rope_qk_apply: row
 * r of sample s, r < seq_used[s], sees the keys of the same sample below seq_used[s], with
 * causal != 0 those at r or before.  Rows of no sample, and rows beyond seq_used, see no
 * key (out = 0) and are no key of any row (their dq, dk and dv are 0).
 */
typedef struct attn_varlen_desc {
    const void *q;                 /* [total_tokens, n_q_heads, head_dim]              */
    int64_t q_stride_token;
    int64_t q_stride_head;
    const void *k;                 /* [total_tokens, n_kv_heads, head_dim]             */
    int64_t k_stride_token;
    int64_t k_stride_head;
    const void *v;
    int64_t v_stride_token;
    int64_t v_stride_head;
    void *out;                     /* [total_tokens, n_q_heads, head_dim]: written by the
                                      forward, read by the backward                    */
    int64_t out_stride_token;
    int64_t out_stride_head;
    float *lse;                    /* float [n_q_heads, total_tokens], natural logarithm;
                                      forward: written, or NULL; backward: read        */
    const int32_t *cu_seqlens;
    const int32_t *seq_used;       /* or NULL                                          */
    int64_t total_tokens;          /* <= 2^24; times n_q_heads below 2^31              */
    int32_t n_seqs;                /* (total_tokens / 128 + n_seqs + 2) * n_q_heads is
                                      below 2^31 too, else ROPE_ERR_UNSUPPORTED        */
    int32_t n_q_heads;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t causal;
    float scale;                   /* finite and > 0, e.g. 1/sqrt(head_dim)            */
} attn_varlen_desc;

int attn_varlen_fwd(const attn_varlen_desc *desc, void *stream);

/* The gradients of attn_varlen_fwd: dout is read, dq, dk and dv are written whole. */
typedef struct attn_varlen_grads {
    const void *dout;              /* [total_tokens, n_q_heads, head_dim]              */
    int64_t dout_stride_token;
    int64_t dout_stride_head;
    void *dq;
    int64_t dq_stride_token;
    int64_t dq_stride_head;
    void *dk;                      /* [total_tokens, n_kv_heads, head_dim]             */
    int64_t dk_stride_token;
    int64_t dk_stride_head;
    void *dv;
    int64_t dv_stride_token;
    int64_t dv_stride_head;
} attn_varlen_grads;

/* Device bytes attn_varlen_bwd needs (16-byte aligned), or -1 for invalid counts. */
int64_t attn_varlen_bwd_workspace_bytes(int64_t total_tokens, int32_t n_q_heads);

/* desc as for the forward, with the out and lse that it wrote.  ROPE_ERR_WORKSPACE when
 * workspace_bytes is below attn_varlen_bwd_workspace_bytes. */
int attn_varlen_bwd(const attn_varlen_desc *desc, const attn_varlen_grads *grads, void *workspace,
                    int64_t workspace_bytes, void *stream);

/*
 * Attention of new tokens over a paged cache (paged_kv.h): new token i of sequence s, at
 * position kv_lens[s] - n + i, sees the cache's keys at positions up to its own (causal !=
 * 0), or all kv_lens[s] of them.  The new tokens' own keys and values are read from the
 * cache: append first.  A page id outside [0, n_pages) reads as keys and values of zero;
 * positions past max_pages * page_size are not read.  A row with a negative position, or
 * of no sequence, sees no key.
 *
 * One token per sequence up to whole prompts.  Where rows are few, a sequence's keys are
 * shared by the CTAs of a cluster, which join their results on the chip; only where that
 * leaves SMs idle are they split further, with partial results in the workspace and a second
 * launch that joins them.  All of it depends on the sizes on the host alone: max_kv_len, an
 * upper bound on kv_lens[s] (0: max_pages * page_size), tunes it and never cuts keys off.  A
 * page table much wider than the sequences, without that bound, is planned for as if they
 * were that long.
 */
typedef struct attn_paged_desc {
    const void *q;                 /* [total_tokens, n_q_heads, head_dim]              */
    int64_t q_stride_token;
    int64_t q_stride_head;
    void *out;
    int64_t out_stride_token;
    int64_t out_stride_head;
    rope_paged_kv cache;
    const int32_t *cu_seqlens;     /* device int32 [n_seqs + 1]                        */
    const int32_t *kv_lens;        /* device int32 [n_seqs]                            */
    const int32_t *page_table;     /* device int32 [n_seqs, max_pages]                 */
    int64_t page_table_stride;
    int64_t total_tokens;          /* new tokens, <= 2^24                              */
    int64_t max_kv_len;
    int32_t max_pages;
    int32_t n_seqs;                /* limits as for attn_varlen_desc                   */
    int32_t n_q_heads;
    int32_t causal;
    float scale;
    int32_t reserved;              /* 0 */
} attn_paged_desc;

/* Device bytes attn_paged needs for `desc` (16-byte aligned; 0: none), or a negative
 * rope_status for sizes that attn_paged would refuse.  Reads sizes only. */
int64_t attn_paged_workspace_bytes(const attn_paged_desc *desc);

int attn_paged(const attn_paged_desc *desc, void *workspace, int64_t workspace_bytes, void *stream);

/* 1 when a bounded wait inside an attention kernel has run out on the current device since
 * the library was loaded or this was last called (results since then are invalid), else 0;
 * ROPE_ERR_LAUNCH when the device cannot be read.  Waits for the work of every stream of the
 * device first: for tests and diagnosis, and not while a stream is captured. */
int attn_fault(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H */
