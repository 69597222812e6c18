// Appending new keys and values to a paged cache, rotated on the way (GB300, sm_103a).
//
// One CTA owns a tile of consecutive new tokens and moves every Q, K and V head of them:
// Q and K rows are rotated by the token's position in its sequence with the arithmetic of
// the rotation kernel (y = x*cos + rotate_half(x)*sin, identical bits), V rows are copied;
// Q goes back to where it was or to q_out, K and V to their page.  Every element is read
// once and written once, about half a flop a byte: the bound is HBM for prompts (16,384 tokens
// of 64/8 heads of 128: 111 us, 6.05 TB/s, 104 us with a cos/sin cache; of 32/8 heads 68 and
// 63 us), the evaluation of cos and sin where heads are few (8/2 heads: 3.7 TB/s), and the
// chain of dependent loads (sequence, cache length, page) for a decoding step.  Against
// that chain cu_seqlens and kv_lens are staged in one round of loads, the page lookup
// overlaps the evaluation of cos and sin, and the first rows are loaded before any of it.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fastdiv.cuh"
#include "host_checks.h"
#include "paged_checks.h"
#include "paged_kv.h"
#include "rope_core.cuh"

namespace {

using namespace pvr;

constexpr int kThreads = 128;
// 16-byte pair units in flight per thread.  16,384 tokens of 48 and of 80 heads of 128: 68 and
// 111 us; with 2 71 and 110 us, with 5 84 and 110 us (fewer resident CTAs).
constexpr int kUnits = 3;
constexpr int kMaxTile = 16;            // tokens per tile
constexpr int kMaxStaged = 256;         // sequences whose cu_seqlens and kv_lens are staged

struct AppendArgs {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_pages, *v_pages;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs;
    int64_t kp_ps, kp_ts, kp_hs, vp_ps, vp_ts, vp_hs;
    const int32_t *cu, *kv_lens, *table;
    int64_t table_stride;
    const float4 *cache;                // cos/sin rows, or NULL
    int32_t cache_rows;
    int32_t max_pages, n_pages, page_size;
    int32_t n_seqs, n_tokens, staged;
    int32_t hq, hkv, h_tot, cph, tile;
    int32_t in_place;
    FastDiv div_htot, div_cph;
    float w[kMaxHalf];
};

// Last sequence s in [0, n) with cu[s] <= t, when t lies in [cu[0], cu[n]); else -1.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int n, int t)
{
    if (n <= 0 || t < cu[0] || t >= cu[n]) return -1;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = lo + ((hi - lo) >> 1);
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) rope_kv_append_kernel(const __grid_constant__ AppendArgs a)
{
    extern __shared__ __align__(16) float4 s_cs[];
    __shared__ int s_pos[kMaxTile];
    __shared__ int64_t s_slot_k[kMaxTile], s_slot_v[kMaxTile];

    const int cph = a.cph;
    const int h = 8 * cph;
    const int row4 = 4 * cph;
    const int t0 = blockIdx.x * a.tile;
    const int tt = min(a.tile, a.n_tokens - t0);
    const uint32_t units = static_cast<uint32_t>(tt) * static_cast<uint32_t>(a.h_tot * cph);

    // Unit u: 8 elements from each half of one head of one token.
    struct Where {
        uint32_t tok, head, chunk;
    };
    auto where = [&](uint32_t u) {
        const uint32_t hr = fast_div(u, a.div_cph);
        const uint32_t i = fast_div(hr, a.div_htot);
        return Where{i, hr - i * static_cast<uint32_t>(a.h_tot), u - hr * static_cast<uint32_t>(cph)};
    };
    auto source = [&](const Where &w) {
        const int64_t t = t0 + static_cast<int64_t>(w.tok);
        const int head = static_cast<int>(w.head);
        const __nv_bfloat16 *p = head < a.hq ? a.q + (t * a.q_ts + head * a.q_hs)
                                 : head < a.hq + a.hkv ? a.k + (t * a.k_ts + (head - a.hq) * a.k_hs)
                                                       : a.v + (t * a.v_ts + (head - a.hq - a.hkv) * a.v_hs);
        return p + 8 * w.chunk;
    };
    // where the unit goes; NULL: nowhere
    auto target = [&](const Where &w) -> __nv_bfloat16 * {
        const int64_t t = t0 + static_cast<int64_t>(w.tok);
        const int head = static_cast<int>(w.head);
        if (head < a.hq) {
            if (a.in_place && s_pos[w.tok] < 0) return nullptr;
            return a.q_out + (t * a.qo_ts + head * a.qo_hs) + 8 * w.chunk;
        }
        const bool key = head < a.hq + a.hkv;
        const int64_t slot = key ? s_slot_k[w.tok] : s_slot_v[w.tok];
        if (slot < 0) return nullptr;
        return (key ? a.k_pages + (slot + (head - a.hq) * a.kp_hs)
                    : a.v_pages + (slot + (head - a.hq - a.hkv) * a.vp_hs)) + 8 * w.chunk;
    };

    // the grid may be scheduled while the kernel before it drains: nothing is read earlier
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    Where at[kUnits];
    uint4 lo[kUnits], hi[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const uint32_t u = threadIdx.x + k * kThreads;
        if (u >= units) continue;
        at[k] = where(u);
        const __nv_bfloat16 *src = source(at[k]);
        lo[k] = load_stream(src);
        hi[k] = load_stream(src + h);
    }

    // positions and pages, one thread per token
    int32_t *s_cu = reinterpret_cast<int32_t *>(s_cs + a.tile * row4);
    int32_t *s_kv = s_cu + a.n_seqs + 1;
    if (a.staged) {
        for (int i = threadIdx.x; i < 2 * a.n_seqs + 1; i += kThreads)
            s_cu[i] = i <= a.n_seqs ? __ldg(a.cu + i) : __ldg(a.kv_lens + (i - a.n_seqs - 1));
        __syncthreads();
    }
    if (static_cast<int>(threadIdx.x) < tt) {
        const int t = t0 + static_cast<int>(threadIdx.x);
        const int32_t *cu = a.staged ? s_cu : a.cu;
        const int s = sequence_of(cu, a.n_seqs, t);
        int pos = -1;
        int64_t slot_k = -1, slot_v = -1;
        if (s >= 0) {
            const int64_t p = static_cast<int64_t>(a.staged ? s_kv[s] : __ldg(a.kv_lens + s)) -
                              (static_cast<int64_t>(cu[s + 1]) - t);
            if (p >= 0 && p < kMaxTokens && cu[s] >= 0) pos = static_cast<int>(p);
        }
        s_pos[threadIdx.x] = pos;
        if (pos >= 0) {
            const int index = pos / a.page_size;
            const int in_page = pos - index * a.page_size;
            const int page = index < a.max_pages ? __ldg(a.table + s * a.table_stride + index) : -1;
            if (page >= 0 && page < a.n_pages) {
                slot_k = page * a.kp_ps + in_page * a.kp_ts;
                slot_v = page * a.vp_ps + in_page * a.vp_ts;
            }
        }
        s_slot_k[threadIdx.x] = slot_k;
        s_slot_v[threadIdx.x] = slot_v;
    }
    __syncthreads();

    // (cos, sin) rows of the tile, in the cache's [quad][chunk] order
    float2 *s_cs2 = reinterpret_cast<float2 *>(s_cs);
    for (int p2 = threadIdx.x; p2 < 2 * tt * row4; p2 += kThreads) {
        const int idx = p2 >> 1;
        const int i = idx / row4;
        const int r = idx - i * row4;
        const int pos = s_pos[i];
        float2 cs = make_float2(1.0f, 0.0f);
        if (pos >= 0) {
            if (pos < a.cache_rows) {
                cs = __ldg(reinterpret_cast<const float2 *>(a.cache + static_cast<int64_t>(pos) * row4 + r) + (p2 & 1));
            } else {
                const int quad = r / cph;
                cs = cos_sin_at(pos, a.w[8 * (r - quad * cph) + 2 * quad + (p2 & 1)]);
            }
        }
        s_cs2[p2] = cs;
    }
    __syncthreads();

    auto finish = [&](const Where &w, uint4 x, uint4 y) {
        __nv_bfloat16 *dst = target(w);
        if (dst == nullptr) return;
        if (static_cast<int>(w.head) < a.hq + a.hkv && s_pos[w.tok] >= 0) {
            const float4 *cs = s_cs + w.tok * row4 + w.chunk;
            rotate2(x.x, y.x, cs[0]);
            rotate2(x.y, y.y, cs[cph]);
            rotate2(x.z, y.z, cs[2 * cph]);
            rotate2(x.w, y.w, cs[3 * cph]);
        }
        *reinterpret_cast<uint4 *>(dst) = x;
        *reinterpret_cast<uint4 *>(dst + h) = y;
    };
    for (uint32_t base = 0;;) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
            if (base + threadIdx.x + k * kThreads < units) finish(at[k], lo[k], hi[k]);
        base += kUnits * kThreads;
        if (base >= units) break;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const uint32_t u = base + threadIdx.x + k * kThreads;
            if (u >= units) continue;
            at[k] = where(u);
            const __nv_bfloat16 *src = source(at[k]);
            lo[k] = load_stream(src);
            hi[k] = load_stream(src + h);
        }
    }
}

}  // namespace

extern "C" int rope_kv_append(const rope_kv_append_desc *dp, void *stream)
{
    if (dp == nullptr) return ROPE_ERR_NULL;
    const rope_kv_append_desc &p = *dp;
    const rope_paged_kv &c = p.cache;
    const int64_t T = p.total_tokens;
    AppendViews w;
    const int rc = check_append(p, w);
    if (rc != ROPE_OK || T == 0) return rc;
    const int64_t d = c.head_dim;
    const View &q = w.q, &k = w.k, &v = w.v, &qo = w.q_out;
    const bool in_place = p.q_out == nullptr;

    AppendArgs a{};
    a.q = static_cast<const __nv_bfloat16 *>(p.q);
    a.k = static_cast<const __nv_bfloat16 *>(p.k);
    a.v = static_cast<const __nv_bfloat16 *>(p.v);
    a.q_out = static_cast<__nv_bfloat16 *>(const_cast<void *>(qo.base));
    a.k_pages = static_cast<__nv_bfloat16 *>(c.k);
    a.v_pages = static_cast<__nv_bfloat16 *>(c.v);
    a.q_ts = q.ts; a.q_hs = q.hs; a.k_ts = k.ts; a.k_hs = k.hs; a.v_ts = v.ts; a.v_hs = v.hs;
    a.qo_ts = qo.ts; a.qo_hs = qo.hs;
    a.kp_ps = c.k_stride_page; a.kp_ts = c.k_stride_token; a.kp_hs = c.k_stride_head;
    a.vp_ps = c.v_stride_page; a.vp_ts = c.v_stride_token; a.vp_hs = c.v_stride_head;
    a.cu = p.cu_seqlens; a.kv_lens = p.kv_lens; a.table = p.page_table;
    a.table_stride = p.page_table_stride;
    const rope_cos_sin_cache *cs = p.cos_sin_cache;
    a.cache = cs != nullptr && cs->rows > 0 ? reinterpret_cast<const float4 *>(cs->data) : nullptr;
    a.cache_rows = a.cache != nullptr ? static_cast<int32_t>(cs->rows) : 0;
    a.max_pages = p.max_pages;
    a.n_pages = static_cast<int32_t>(c.n_pages);
    a.page_size = c.page_size;
    a.n_seqs = p.n_seqs;
    a.n_tokens = static_cast<int32_t>(T);
    a.staged = p.n_seqs < kMaxStaged ? 1 : 0;
    a.hq = p.n_q_heads;
    a.hkv = c.n_kv_heads;
    a.h_tot = a.hq + 2 * a.hkv;
    a.cph = static_cast<int32_t>(d / 16);
    a.in_place = in_place ? 1 : 0;
    a.div_htot = make_fastdiv(static_cast<uint32_t>(a.h_tot));
    a.div_cph = make_fastdiv(static_cast<uint32_t>(a.cph));
    host_inv_freq(p.theta, c.head_dim, p.position_scale, a.w);
    // as many tokens as one batch of units covers
    const int64_t per_token = static_cast<int64_t>(a.h_tot) * a.cph;
    const int64_t fit = (kUnits * kThreads) / per_token;
    a.tile = static_cast<int32_t>(fit < 1 ? 1 : fit > kMaxTile ? kMaxTile : fit);
    const size_t smem = static_cast<size_t>(a.tile) * 4 * a.cph * sizeof(float4) +
                        (a.staged ? (2 * static_cast<size_t>(a.n_seqs) + 1) * sizeof(int32_t) : 0);

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((T + a.tile - 1) / a.tile));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kv_append_kernel, a) == cudaSuccess ? ROPE_OK : ROPE_ERR_LAUNCH;
}
