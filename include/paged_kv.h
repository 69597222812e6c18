/*
 * paged_kv.h -- C ABI of the paged key/value cache: its layout, and the append that
 * rotates new keys on their way into it (part of librope_qk.so).  attn.h reads the cache.
 *
 * Layout.  A cache holds keys and values in n_pages pages of page_size tokens.  Element
 * (page, slot, kv head, i) of the keys is k[page*k_stride_page + slot*k_stride_token +
 * head*k_stride_head + i], i contiguous, bf16; the values likewise.  Any strides (all
 * multiples of 8 elements) under which no two rows share an element: [pages, page_size,
 * heads, d], [pages, heads, page_size, d], or one pool [pages, 2, ...] holding both.
 *
 * Sequences.  Row s of the page table names the pages of sequence s: its token at
 * position p (0-based) sits in page page_table[s*page_table_stride + p / page_size],
 * slot p % page_size.  kv_lens[s] is the number of tokens of sequence s in the cache
 * WITH the new ones of this call; cu_seqlens [n_seqs + 1] delimits the new tokens in the
 * packed token stream as for rope_qk_fwd.  New token i of n has position
 * kv_lens[s] - n + i.  rope_kv_append and attn_paged take the same four arrays.
 * One step of a serving loop appends the step's tokens, then attends.
 *
 * Ownership, streams, errors as in rope_qk.h: device pointers owned by the caller, no
 * allocation, asynchronous on `stream`, ROPE_OK or a negative rope_status, checked on the
 * host before anything is launched.
 */
#ifndef PAGED_KV_H
#define PAGED_KV_H

#include <stdint.h>

#include "rope_qk.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct rope_paged_kv {
    void *k;                       /* bf16 [n_pages, page_size, n_kv_heads, head_dim]  */
    int64_t k_stride_page;         /* elements                                         */
    int64_t k_stride_token;
    int64_t k_stride_head;
    void *v;
    int64_t v_stride_page;
    int64_t v_stride_token;
    int64_t v_stride_head;
    int64_t n_pages;               /* >= 0, below 2^31                                 */
    int32_t page_size;             /* tokens a page, a multiple of 8, at most 65,536   */
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t reserved;              /* 0 */
} rope_paged_kv;

typedef struct rope_kv_append_desc {
    void *q;                       /* bf16 view [total_tokens, n_q_heads, head_dim]    */
    int64_t q_stride_token;
    int64_t q_stride_head;
    const void *k;                 /* bf16 view [total_tokens, n_kv_heads, head_dim]   */
    int64_t k_stride_token;
    int64_t k_stride_head;
    const void *v;
    int64_t v_stride_token;
    int64_t v_stride_head;
    void *q_out;                   /* NULL: q is rotated in place                      */
    int64_t q_out_stride_token;
    int64_t q_out_stride_head;
    rope_paged_kv cache;
    const int32_t *cu_seqlens;     /* device int32 [n_seqs + 1]                        */
    const int32_t *kv_lens;        /* device int32 [n_seqs], new tokens included       */
    const int32_t *page_table;     /* device int32 [n_seqs, max_pages]                 */
    int64_t page_table_stride;     /* elements between rows, >= max_pages              */
    int32_t max_pages;
    int32_t n_seqs;
    int32_t n_q_heads;
    int32_t reserved;              /* 0 */
    int64_t total_tokens;
    double theta;
    double position_scale;         /* 1.0 = plain rotation                             */
    const rope_cos_sin_cache *cos_sin_cache;   /* optional (NULL: none)                */
} rope_kv_append_desc;

/*
 * Rotate the new tokens' Q (in place or into q_out) and K by their positions in the
 * cache, write the rotated K and the V into their pages.  One pass, one launch; the
 * rotated values carry the bits rope_qk_apply gives at those positions (arithmetic of
 * rope_qk.h; head_dim a multiple of 16 in [16, 256]; cos/sin from the cache, or evaluated
 * in the kernel, with identical bits).  The k and v inputs are only read.
 *
 * Rows left out.  A row of no sequence, or whose position is negative or at least 2^24,
 * is not rotated (in place: untouched; out of place: q copied) and not appended.  A row
 * whose page lies beyond max_pages, or whose page id is outside [0, n_pages), is rotated
 * in q and not appended.  Two rows sent to the same slot of the same page race.
 *
 * q must share no element with k or v when rotated in place (the slices of one fused
 * QKV output qualify); the cache's keys and values share none with each other, nor their
 * address ranges with q, k, v or q_out (else ROPE_ERR_OVERLAP).
 */
int rope_kv_append(const rope_kv_append_desc *desc, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_KV_H */
