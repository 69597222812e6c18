// What the attention entry points (attn.cu) pass to the kernels' launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

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
    // rules on the scores (attn_score_rule)
    float cap;                      // 0: none
    const float *slopes;            // [hq] or NULL
    const int32_t *prefix;          // [n_seqs] or NULL

    // the instance that serves the rule (score_rule.cuh)
    int rule() const
    {
        const int shape = (cap > 0.0f ? 2 : 0) + (slopes != nullptr ? 4 : 0);
        return shape != 0 ? shape : prefix != nullptr ? 1 : 0;
    }
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
// Instances of the kernels by rule, each compiled on its own (attn_fwd.cu, attn_bwd.cu,
// attn_decode.cu with PVR_SCORE_RULE = RULE): their launch, and their count of waits that ran out.
template <int RULE> cudaError_t launch_attn_fwd_rule(const AttnProblem &p, int splits, float *workspace, cudaStream_t stream);
template <int RULE> cudaError_t launch_attn_bwd_rule(const AttnProblem &p, cudaStream_t stream);
template <int RULE> cudaError_t launch_attn_decode_rule(const AttnProblem &p, const DecodePlan &plan, float *workspace,
                                                        cudaStream_t stream);
template <int RULE> int attn_fwd_fault_of(int *word);
template <int RULE> int attn_bwd_fault_of(int *word);
template <int RULE> int attn_decode_fault_of(int *word);
#define PVR_DECLARE_RULE(R)                                                                                              \
    template <> cudaError_t launch_attn_fwd_rule<R>(const AttnProblem &, int, float *, cudaStream_t);                    \
    template <> cudaError_t launch_attn_bwd_rule<R>(const AttnProblem &, cudaStream_t);                                  \
    template <> cudaError_t launch_attn_decode_rule<R>(const AttnProblem &, const DecodePlan &, float *, cudaStream_t);  \
    template <> int attn_fwd_fault_of<R>(int *);                                                                         \
    template <> int attn_bwd_fault_of<R>(int *);                                                                         \
    template <> int attn_decode_fault_of<R>(int *);
PVR_DECLARE_RULE(0)
PVR_DECLARE_RULE(1)
PVR_DECLARE_RULE(2)
PVR_DECLARE_RULE(4)
PVR_DECLARE_RULE(6)
#undef PVR_DECLARE_RULE

// Calls fn(std::integral_constant<int, RULE>) with the instance that serves `rule`.
template <typename Fn>
auto for_rule(int rule, Fn fn)
{
    switch (rule) {
    case 1: return fn(std::integral_constant<int, 1>{});
    case 2: return fn(std::integral_constant<int, 2>{});
    case 4: return fn(std::integral_constant<int, 4>{});
    case 6: return fn(std::integral_constant<int, 6>{});
    default: return fn(std::integral_constant<int, 0>{});
    }
}

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

// The counts of all instances of a kernel together.
template <typename Read>
int sum_fault_words(int *word, Read read)
{
    *word = 0;
    for (const int rule : {0, 1, 2, 4, 6}) {
        int one = 0;
        if (for_rule(rule, [&](auto r) { return read(r, &one); }) != 0) return -1;
        *word += one;
    }
    return 0;
}

}  // namespace pvr
