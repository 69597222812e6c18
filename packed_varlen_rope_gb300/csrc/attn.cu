// Entry points of the attention operators: argument checks on the host, then the launch.

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "attn_internal.h"
#include "host_checks.h"
#include "paged_checks.h"

namespace {

using namespace pvr;

constexpr int kMaxAttnDim = 128;
constexpr int kMaxGroup = 128;

int check_heads(int64_t T, int32_t n_seqs, int32_t hq, int32_t hkv, int32_t d, float scale)
{
    if (T < 0 || n_seqs < 0 || hq < 1 || hkv < 1 || hq > (1 << 20) || hq % hkv != 0 || n_seqs > kMaxTokens) return ROPE_ERR_SHAPE;
    if (d < 16 || d > kMaxAttnDim || d % 16 != 0) return ROPE_ERR_HEAD_DIM;
    // (token, head) rows are counted in 32 bits
    if (hq / hkv > kMaxGroup || T > kMaxTokens || T * hq > INT32_MAX) return ROPE_ERR_UNSUPPORTED;
    // and so are a launch's CTAs: a head's tiles of 128 rows, and a slot more for every sequence
    if ((T / 128 + n_seqs + 2) * hq > INT32_MAX) return ROPE_ERR_UNSUPPORTED;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return ROPE_ERR_THETA;
    return ROPE_OK;
}

Rows rows_of(const View &v)
{
    return Rows{static_cast<__nv_bfloat16 *>(const_cast<void *>(v.base)), v.ts, v.hs};
}

int status_of(cudaError_t e) { return e == cudaSuccess ? ROPE_OK : ROPE_ERR_LAUNCH; }

// Checks shared by the forward and the backward; fills the problem.
int varlen_problem(const attn_varlen_desc &p, AttnProblem &a, View (&in)[3], View &out)
{
    int rc = check_heads(p.total_tokens, p.n_seqs, p.n_q_heads, p.n_kv_heads, p.head_dim, p.scale);
    if (rc != ROPE_OK || p.total_tokens == 0) return rc;
    if (p.cu_seqlens == nullptr) return ROPE_ERR_NULL;
    const int64_t T = p.total_tokens, d = p.head_dim;
    in[0] = View{p.q, T, p.n_q_heads, p.q_stride_token, p.q_stride_head, d};
    in[1] = View{p.k, T, p.n_kv_heads, p.k_stride_token, p.k_stride_head, d};
    in[2] = View{p.v, T, p.n_kv_heads, p.v_stride_token, p.v_stride_head, d};
    out = View{p.out, T, p.n_q_heads, p.out_stride_token, p.out_stride_head, d};
    for (const View *v : {&in[0], &in[1], &in[2], &out})
        if ((rc = check_view(*v)) != ROPE_OK) return rc;
    for (const View &v : in)
        if (!views_disjoint(v, out)) return ROPE_ERR_OVERLAP;
    a = AttnProblem{};
    a.q = rows_of(in[0]);
    a.k = rows_of(in[1]);
    a.v = rows_of(in[2]);
    a.out = rows_of(out);
    a.lse = p.lse;
    a.cu = p.cu_seqlens;
    a.used = p.seq_used;
    a.n_tokens = static_cast<int32_t>(T);
    a.n_seqs = p.n_seqs;
    a.hq = p.n_q_heads;
    a.hkv = p.n_kv_heads;
    a.group = p.n_q_heads / p.n_kv_heads;
    a.d = p.head_dim;
    a.causal = p.causal != 0;
    a.scale = p.scale;
    return ROPE_OK;
}

// Sizes of a paged call.
int check_paged_sizes(const attn_paged_desc &p)
{
    int rc = check_heads(p.total_tokens, p.n_seqs, p.n_q_heads, p.cache.n_kv_heads, p.cache.head_dim, p.scale);
    if (rc != ROPE_OK) return rc;
    if (p.reserved != 0) return ROPE_ERR_UNSUPPORTED;
    if (p.max_pages < 0 || p.max_kv_len < 0) return ROPE_ERR_SHAPE;
    if (p.cache.page_size < 8 || p.cache.page_size > 65536 || p.cache.page_size % 8 != 0) return ROPE_ERR_SHAPE;
    if (static_cast<int64_t>(p.max_pages) * p.cache.page_size > INT32_MAX / 2) return ROPE_ERR_UNSUPPORTED;
    return ROPE_OK;
}

// Which kernel serves a call and how it splits the keys: from the sizes on the host alone.
struct PagedPlan {
    DecodePlan decode;
    int splits = 1;
};

PagedPlan plan_of(const attn_paged_desc &p)
{
    PagedPlan plan;
    if (p.total_tokens == 0) return plan;
    AttnProblem a{};
    a.n_tokens = static_cast<int32_t>(p.total_tokens);
    a.n_seqs = p.n_seqs;
    a.hq = p.n_q_heads;
    a.hkv = p.cache.n_kv_heads;
    a.group = a.hq / a.hkv;
    a.d = p.cache.head_dim;
    int64_t keys = static_cast<int64_t>(p.max_pages) * p.cache.page_size;
    if (p.max_kv_len > 0 && p.max_kv_len < keys) keys = p.max_kv_len;
    plan.decode = attn_decode_plan(a, keys);
    plan.splits = plan.decode.use ? plan.decode.splits : attn_fwd_splits(a, keys);
    return plan;
}

}  // namespace

extern "C" {

int attn_varlen_fwd(const attn_varlen_desc *desc, void *stream)
{
    if (desc == nullptr) return ROPE_ERR_NULL;
    AttnProblem a;
    View in[3], out;
    const int rc = varlen_problem(*desc, a, in, out);
    if (rc != ROPE_OK || desc->total_tokens == 0) return rc;
    if (!aligned(a.lse, 4)) return ROPE_ERR_ALIGN;
    return status_of(launch_attn_fwd(a, 1, nullptr, static_cast<cudaStream_t>(stream)));
}

int64_t attn_varlen_bwd_workspace_bytes(int64_t total_tokens, int32_t n_q_heads)
{
    if (total_tokens < 0 || total_tokens > kMaxTokens || n_q_heads < 1 || n_q_heads > (1 << 20)) return -1;
    return total_tokens * n_q_heads * 2 * static_cast<int64_t>(sizeof(float));
}

int attn_varlen_bwd(const attn_varlen_desc *desc, const attn_varlen_grads *grads, void *workspace,
                    int64_t workspace_bytes, void *stream)
{
    if (desc == nullptr || grads == nullptr) return ROPE_ERR_NULL;
    AttnProblem a;
    View in[5], out;
    View qkv[3];
    int rc = varlen_problem(*desc, a, qkv, out);
    if (rc != ROPE_OK || desc->total_tokens == 0) return rc;
    const int64_t T = desc->total_tokens, d = desc->head_dim;
    const attn_varlen_grads &g = *grads;
    for (int i = 0; i < 3; ++i) in[i] = qkv[i];
    in[3] = out;
    in[4] = View{g.dout, T, a.hq, g.dout_stride_token, g.dout_stride_head, d};
    const View res[3] = {{g.dq, T, a.hq, g.dq_stride_token, g.dq_stride_head, d},
                         {g.dk, T, a.hkv, g.dk_stride_token, g.dk_stride_head, d},
                         {g.dv, T, a.hkv, g.dv_stride_token, g.dv_stride_head, d}};
    if ((rc = check_view(in[4])) != ROPE_OK) return rc;
    for (const View &v : res)
        if ((rc = check_view(v)) != ROPE_OK) return rc;
    for (int i = 0; i < 3; ++i) {
        for (const View &v : in)
            if (!views_disjoint(v, res[i])) return ROPE_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (!views_disjoint(res[j], res[i])) return ROPE_ERR_OVERLAP;
    }
    if (a.lse == nullptr || workspace == nullptr) return ROPE_ERR_NULL;
    if (!aligned(a.lse, 4) || !aligned(workspace, 16)) return ROPE_ERR_ALIGN;
    if (workspace_bytes < attn_varlen_bwd_workspace_bytes(T, a.hq)) return ROPE_ERR_WORKSPACE;
    a.stats = static_cast<float *>(workspace);
    a.dout = rows_of(in[4]);
    a.dq = rows_of(res[0]);
    a.dk = rows_of(res[1]);
    a.dv = rows_of(res[2]);
    return status_of(launch_attn_bwd(a, static_cast<cudaStream_t>(stream)));
}

int64_t attn_paged_workspace_bytes(const attn_paged_desc *desc)
{
    if (desc == nullptr) return ROPE_ERR_NULL;
    const int rc = check_paged_sizes(*desc);
    if (rc != ROPE_OK) return rc;
    return 4 * attn_split_floats(desc->total_tokens, desc->n_q_heads, desc->cache.head_dim, plan_of(*desc).splits);
}

int attn_paged(const attn_paged_desc *desc, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (desc == nullptr) return ROPE_ERR_NULL;
    const attn_paged_desc &p = *desc;
    const rope_paged_kv &c = p.cache;
    int rc;
    if ((rc = check_paged_sizes(p)) != ROPE_OK || (rc = check_paged(c)) != ROPE_OK) return rc;
    const int64_t T = p.total_tokens, d = c.head_dim;
    if (T == 0) return ROPE_OK;
    if ((rc = check_page_table(p.cu_seqlens, p.kv_lens, p.page_table, p.page_table_stride, p.max_pages,
                               p.n_seqs)) != ROPE_OK)
        return rc;
    const View q{p.q, T, p.n_q_heads, p.q_stride_token, p.q_stride_head, d};
    const View out{p.out, T, p.n_q_heads, p.out_stride_token, p.out_stride_head, d};
    for (const View *v : {&q, &out})
        if ((rc = check_view(*v)) != ROPE_OK) return rc;
    if (!views_disjoint(q, out)) return ROPE_ERR_OVERLAP;
    if (c.n_pages > 0 && (overlap(c.k, 2 * k_span(c), p.out, out.bytes()) ||
                          overlap(c.v, 2 * v_span(c), p.out, out.bytes())))
        return ROPE_ERR_OVERLAP;
    const PagedPlan plan = plan_of(p);
    const int64_t need = 4 * attn_split_floats(T, p.n_q_heads, c.head_dim, plan.splits);
    if (need > 0 && workspace == nullptr) return ROPE_ERR_NULL;
    if (need > 0 && !aligned(workspace, 16)) return ROPE_ERR_ALIGN;
    if (workspace_bytes < need) return ROPE_ERR_WORKSPACE;

    AttnProblem a{};
    a.q = rows_of(q);
    a.out = rows_of(out);
    a.paged = 1;
    a.pages = Pages{static_cast<const __nv_bfloat16 *>(c.k), static_cast<const __nv_bfloat16 *>(c.v),
                    c.k_stride_page, c.k_stride_token, c.k_stride_head,
                    c.v_stride_page, c.v_stride_token, c.v_stride_head,
                    p.page_table, p.page_table_stride,
                    c.n_pages > 0 ? p.max_pages : 0, c.page_size, static_cast<int32_t>(c.n_pages)};
    a.cu = p.cu_seqlens;
    a.used = p.kv_lens;
    a.n_tokens = static_cast<int32_t>(T);
    a.n_seqs = p.n_seqs;
    a.hq = p.n_q_heads;
    a.hkv = c.n_kv_heads;
    a.group = a.hq / a.hkv;
    a.d = c.head_dim;
    a.causal = p.causal != 0;
    a.scale = p.scale;
    float *ws = static_cast<float *>(workspace);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return status_of(plan.decode.use ? launch_attn_decode(a, plan.decode, ws, st)
                                     : launch_attn_fwd(a, plan.splits, ws, st));
}

int attn_fault(void)
{
    static std::atomic<int> reported[64][3];                 // of each device's counts
    int dev = 0, now[3] = {0, 0, 0};
    // the copies below wait for the default stream alone, and kernels run on any
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return ROPE_ERR_LAUNCH;
    if (attn_fault_word(&now[0]) != 0 || attn_bwd_fault_word(&now[1]) != 0 || attn_decode_fault_word(&now[2]) != 0)
        return ROPE_ERR_LAUNCH;
    int raised = 0;
    for (int i = 0; i < 3; ++i) {
        std::atomic<int> &known = reported[dev & 63][i];
        int before = known.load();
        while (before < now[i] && !known.compare_exchange_weak(before, now[i])) {}
        if (before < now[i]) raised = 1;
    }
    return raised;
}

}  // extern "C"
