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
    float *delta;                   // backward workspace, [hq, tokens]
    Pages pages;                    // read when paged is set, else k and v
    int32_t paged;
    const int32_t *cu;
    const int32_t *used;            // seq_used, or kv_lens of a paged problem
    int32_t n_tokens, n_seqs, hq, hkv, group, d, causal;
    float scale;
};

cudaError_t launch_attn_simple_fwd(const AttnProblem &p, cudaStream_t stream);
cudaError_t launch_attn_simple_bwd(const AttnProblem &p, cudaStream_t stream);

}  // namespace pvr
