// Host-side checks of a paged key/value cache, shared by the append and the attention.
#pragma once

#include "host_checks.h"
#include "paged_kv.h"

namespace pvr {

// The address pattern sum_i n_i * stride_i + [0, d) with every n_i below its extent names
// each element once: strides in increasing order, each at least the span of those below.
struct Axis {
    int64_t n, stride;
};

inline bool axes_injective(Axis *ax, int count, int64_t d)
{
    for (int i = 1; i < count; ++i)
        for (int j = i; j > 0 && ax[j].stride < ax[j - 1].stride; --j) std::swap(ax[j], ax[j - 1]);
    __int128 span = d;
    for (int i = 0; i < count; ++i) {
        if (ax[i].n <= 1) continue;
        if (ax[i].stride < span) return false;
        span += static_cast<__int128>(ax[i].n - 1) * ax[i].stride;
    }
    return span < (static_cast<__int128>(1) << 56);
}

// Elements a pool spans (after check_paged has bounded it).
inline int64_t pool_span(const rope_paged_kv &c, int64_t ps, int64_t ts, int64_t hs)
{
    return (c.n_pages - 1) * ps + (int64_t(c.page_size) - 1) * ts + (int64_t(c.n_kv_heads) - 1) * hs + c.head_dim;
}

inline int64_t k_span(const rope_paged_kv &c) { return pool_span(c, c.k_stride_page, c.k_stride_token, c.k_stride_head); }
inline int64_t v_span(const rope_paged_kv &c) { return pool_span(c, c.v_stride_page, c.v_stride_token, c.v_stride_head); }

// Sizes, strides, alignment and overlap of a cache.  With n_pages == 0 nothing is read.
inline int check_paged(const rope_paged_kv &c)
{
    if (c.n_pages < 0 || c.n_pages > INT32_MAX || c.n_kv_heads < 1 || c.n_kv_heads > (1 << 20)) return ROPE_ERR_SHAPE;
    if (c.page_size < 8 || c.page_size > 65536 || c.page_size % 8 != 0) return ROPE_ERR_SHAPE;
    if (c.reserved != 0) return ROPE_ERR_UNSUPPORTED;
    const int rc = check_head_dim(c.head_dim);
    if (rc != ROPE_OK || c.n_pages == 0) return rc;
    if (c.k == nullptr || c.v == nullptr) return ROPE_ERR_NULL;
    const int64_t st[6] = {c.k_stride_page, c.k_stride_token, c.k_stride_head,
                           c.v_stride_page, c.v_stride_token, c.v_stride_head};
    for (const int64_t s : st) {
        if (s < 0) return ROPE_ERR_SHAPE;
        if (s % 8 != 0) return ROPE_ERR_ALIGN;
    }
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return ROPE_ERR_ALIGN;
    Axis ka[4] = {{c.n_pages, st[0]}, {c.page_size, st[1]}, {c.n_kv_heads, st[2]}, {0, 0}};
    Axis va[3] = {{c.n_pages, st[3]}, {c.page_size, st[4]}, {c.n_kv_heads, st[5]}};
    if (!axes_injective(ka, 3, c.head_dim) || !axes_injective(va, 3, c.head_dim)) return ROPE_ERR_OVERLAP;
    if (!overlap(c.k, 2 * k_span(c), c.v, 2 * v_span(c))) return ROPE_OK;
    // keys and values of one pool: the same strides, and the distance between the two one
    // more axis of the pattern
    if (st[0] != st[3] || st[1] != st[4] || st[2] != st[5]) return ROPE_ERR_OVERLAP;
    const int64_t diff = static_cast<int64_t>(reinterpret_cast<uintptr_t>(c.v)) -
                         static_cast<int64_t>(reinterpret_cast<uintptr_t>(c.k));
    Axis both[4] = {{c.n_pages, st[0]}, {c.page_size, st[1]}, {c.n_kv_heads, st[2]}, {2, (diff < 0 ? -diff : diff) / 2}};
    return axes_injective(both, 4, c.head_dim) ? ROPE_OK : ROPE_ERR_OVERLAP;
}

// The arrays that place sequences in the cache.
inline int check_page_table(const int32_t *cu, const int32_t *kv_lens, const int32_t *table, int64_t table_stride,
                            int32_t max_pages, int32_t n_seqs)
{
    if (n_seqs < 0 || max_pages < 0 || (n_seqs > 1 && table_stride < max_pages)) return ROPE_ERR_SHAPE;
    if (cu == nullptr || (n_seqs > 0 && kv_lens == nullptr) || (n_seqs > 0 && max_pages > 0 && table == nullptr))
        return ROPE_ERR_NULL;
    return ROPE_OK;
}

}  // namespace pvr
