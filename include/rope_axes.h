/*
 * rope_axes.h -- C ABI of the rotation by several position axes, for images and video: a
 * token has a position on each axis (time, height, width), and every frequency turns by the
 * position on one of them (part of librope_qk.so).  Forward, backward, and on the way into a
 * paged cache.
 *
 * The operation.  As rope_qk.h, with the angle of frequency j at token t
 *
 *     phi = (float)position[axis(j)][t] * w_j          one binary32 multiply
 *
 * axis(j): `sections` counts the frequencies of each axis, head_dim/2 in all.  They are
 * consecutive (the first sections[0] frequencies turn by axis 0, the next by axis 1, ...), or,
 * with ROPE_AXES_INTERLEAVED, the axes take turns, one frequency each, and one that has had its
 * section is passed over.  w_j = (float)(theta^(-2j/d) / position_scale), as for one axis, or,
 * with ROPE_AXES_OWN_FREQUENCIES, theta^(-i/sections[a]) for the i-th frequency of axis a: each
 * axis has the whole range (an image's two axes alike).  A token whose positions are equal on
 * all axes (text) gets, with the shared frequencies, the bits of rope_qk_apply.
 *
 * Positions are exact in binary32: a token with a position outside [0, 2^24) on any axis is
 * left out (in place untouched, out of place copied, not appended); pad rows are given -1.
 *
 * Layouts, ownership, streams, errors as in rope_qk.h and paged_kv.h.
 */
#ifndef ROPE_AXES_H
#define ROPE_AXES_H

#include <stdint.h>

#include "paged_kv.h"
#include "rope_qk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ROPE_MAX_AXES 4

/* Bits of rope_axes.flags. */
#define ROPE_AXES_INTERLEAVED      0x1
#define ROPE_AXES_OWN_FREQUENCIES  0x2   /* no cos/sin cache: it holds the shared ones (ROPE_ERR_CACHE) */
#define ROPE_AXES_IDS_INT64        0x4   /* position_ids points to int64 values */

/* Host memory, read during the call. */
typedef struct rope_axes {
    const void *position_ids;      /* device int32 [n_axes, total_tokens], a token's positions
                                      contiguous along the tokens; aligned to its type      */
    int64_t position_stride;       /* elements from one axis to the next, >= 0 (0: all axes
                                      share their positions)                                */
    int32_t n_axes;                /* 1 .. ROPE_MAX_AXES                                    */
    int32_t flags;
    int32_t sections[ROPE_MAX_AXES];   /* each >= 1 (0 past n_axes), sum head_dim / 2       */
} rope_axes;

/*
 * Rotate q and k (forward, or with desc->backward the transpose) by their positions on the
 * axes.  desc as for rope_qk_apply, its own position sources unset: cu_seqlens, position_ids,
 * seq_used and segments NULL, n_seqs, n_segments, token_offset and flags 0 (else
 * ROPE_ERR_UNSUPPORTED).  A cos/sin cache serves the shared frequencies of every axis.
 */
int rope_axes_apply(const rope_qk_desc *desc, const rope_axes *axes, void *stream);

/*
 * rope_kv_append with the rotation by several axes.  The place of a token in the cache comes
 * from cu_seqlens, kv_lens and the page table as there; its angles from position_ids.  A row
 * that either leaves out is neither rotated nor appended; one whose page is not in the table or
 * the pool is rotated in q and not appended.
 */
int rope_kv_append_axes(const rope_kv_append_desc *desc, const rope_axes *axes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_AXES_H */
