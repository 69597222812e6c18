/*
 * paged_step.h -- C ABI of a serving step's bookkeeping for the paged cache (paged_kv.h), on the
 * device: pages go back to and come from a stack of free ones, the page table grows, and the
 * arrays that rope_kv_append and attn_paged take are made from the sequences' lengths (part of
 * librope_qk.so).  Nothing is read on the host, so that a whole step fits one CUDA graph.
 *
 * The operation, in this order (s runs over the rows of the page table):
 *
 *   finished   row s with finished[s] != 0 gives back the pages of its past_lens[s] tokens, those
 *              ids of the row that are >= 0, onto the stack in the order of s and of the row; it
 *              is then an empty row, past 0 (new_lens[s] may admit another sequence into it).
 *   lengths    kv_lens[s] = past + new_lens[s]; cu_seqlens[0] = 0, cu_seqlens[s + 1] =
 *              cu_seqlens[s] + new_lens[s].  Negative lengths count as 0, sums stop at 2^31 - 1.
 *   pages      row s needs the pages ceil(past / page_size) .. ceil(kv_lens[s] / page_size) - 1;
 *              in the order of s and of the pages each takes the top of the stack.  Other entries
 *              of the table are left as they are.
 *   slots      slots[t] = id * page_size + place in the page of new token t, -1 for a token
 *              without a page and for t >= cu_seqlens[n_seqs].
 *
 * When the stack runs out the remaining pages get id -1, which the cache's readers treat as no
 * page (STEP_NO_PAGES); later steps do not fill it: finish the row, which gives back what it got.
 * Pages past the table's width are not taken (STEP_TABLE_FULL); what does not fit the stack is
 * dropped (STEP_STACK_FULL); tokens past the slots' end get none (STEP_TOKENS_PAST_END, where
 * slots are wanted).  The bits go to *status.
 *
 * Ownership, streams, errors as in rope_qk.h.  The order is that of the sequences, whatever the
 * timing: the same bits each run.
 */
#ifndef PAGED_STEP_H
#define PAGED_STEP_H

#include <stdint.h>

#include "rope_qk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define STEP_NO_PAGES         0x1
#define STEP_TABLE_FULL       0x2
#define STEP_STACK_FULL       0x4
#define STEP_TOKENS_PAST_END  0x8
#define STEP_NEGATIVE_LENGTH  0x10

typedef struct paged_kv_step_desc {
    int32_t *free_pages;           /* device int32 [n_free_max], the stack; its top is at the count */
    const int32_t *free_count;     /* device int32 [1], entries in use                    */
    int32_t *count_out;            /* device int32 [1], the count after the step; may be free_count */
    int32_t *page_table;           /* device int32 [n_seqs, max_pages]                    */
    int64_t page_table_stride;     /* elements between rows, >= max_pages                 */
    const int32_t *past_lens;      /* device int32 [n_seqs], tokens in the cache          */
    const int32_t *new_lens;       /* device int32 [n_seqs], tokens this step adds        */
    const int32_t *finished;       /* device int32 [n_seqs], or NULL: none                */
    int32_t *cu_seqlens;           /* device int32 [n_seqs + 1], written                  */
    int32_t *kv_lens;              /* device int32 [n_seqs], written                      */
    int64_t *slots;                /* device int64 [max_tokens], written; NULL: not wanted */
    int32_t *status;               /* device int32 [1], STEP_* bits, written; or NULL     */
    int64_t n_free_max;            /* below 2^31                                          */
    int64_t max_tokens;            /* below 2^31                                          */
    int32_t n_seqs;                /* at most 2^24                                        */
    int32_t max_pages;             /* at most 2^24, times page_size below 2^30             */
    int32_t page_size;             /* 1 .. 65,536                                         */
    int32_t reserved;              /* 0 */
} paged_kv_step_desc;

/* What is written shares no address with what else is read or written, but count_out with
 * free_count (else ROPE_ERR_OVERLAP). */
int paged_kv_step(const paged_kv_step_desc *desc, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_STEP_H */
