// What the attention entry points (attn.cu) pass to the kernels' launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pvr {

struct Rows {                       // a bf16 view [tokens, heads, d]
    __nv_bfloat16 *p;
    int64_t ts, hs;
};

// Keys and values in pages.
struct Pages {
    const __nv_bfloat16 *k, *v;
    int64_t k_ps, k_ts, k_hs, v_ps, v_ts, v_hs;
    const int32_t *table;
    int64_t table_stride;
    int32_t max_pages, page_size, n_pages;
};

struct AttnProblem {
    Rows q, k, v, out;
    Rows dout, dq, dk, dv;          // backward
    float *lse;                     // [hq, tokens] or NULL
    float *stats;                   // backward workspace, two floats per [hq, tokens]
    Pages pages;                    // read when paged is set, else k and v
    int32_t paged;
    const int32_t *cu;
    const int32_t *used;            // seq_used, or kv_lens of a paged problem
    int32_t n_tokens, n_seqs, hq, hkv, group, d, causal;
    float scale;
};

constexpr int kSMs = 152;

// Forward on the tensor cores; with splits > 1 the keys of every row are split over that
// many CTAs, and workspace holds attn_split_floats() floats.
cudaError_t launch_attn_fwd(const AttnProblem &p, int splits, float *workspace, cudaStream_t stream);
int attn_fwd_splits(const AttnProblem &p, int64_t max_kv);
inline int64_t attn_split_floats(int64_t n_tokens, int hq, int d, int splits)
{
    return splits > 1 ? n_tokens * hq * (static_cast<int64_t>(d) + 1) * splits : 0;
}
// The kernel for few new tokens a sequence: whether it serves the problem (sizes alone
// decide), and over how many CTAs of a cluster and further splits a sequence's keys go.
struct DecodePlan {
    bool use = false;
    int slots = 0, cluster = 1, splits = 1, warps = 4;
};
DecodePlan attn_decode_plan(const AttnProblem &p, int64_t max_kv);
cudaError_t launch_attn_decode(const AttnProblem &p, const DecodePlan &plan, float *workspace, cudaStream_t stream);
cudaError_t launch_attn_join(const float *part_o, const float *part_lse, const AttnProblem &p, int splits,
                             cudaStream_t stream);
// The kernels' counts of waits that ran out on the current device; 0 on success.  Nothing
// clears them, so that none is lost between two looks.
int attn_fault_word(int *word);
int attn_bwd_fault_word(int *word);
int attn_decode_fault_word(int *word);
// Backward: the rows' statistics, then dq, then dk and dv.  dq goes first: where all keys of a
// row are in one tile it rewrites the row's D, which the pass over the keys then reads.
cudaError_t launch_attn_bwd(const AttnProblem &p, cudaStream_t stream);

template <typename Symbol>
int read_fault_word(int *word, const Symbol &symbol)
{
    return cudaMemcpyFromSymbol(word, symbol, sizeof *word) == cudaSuccess ? 0 : -1;
}

}  // namespace pvr
