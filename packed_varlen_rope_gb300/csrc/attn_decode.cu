// Attention of few new tokens over a paged cache (GB300, sm_103a): a decoding step, or a
// handful of drafted tokens.
//
// Mathematics.  As in the forward (running maximum m, sum l, output o per row), over key
// subsets that are joined at the end: with M = max m_w, o = sum_w 2^(m_w - M) o_w / sum_w
// 2^(m_w - M) l_w.
//
// Layout.  Up to 16 rows, (token, query head) pairs of one key head, fill one m16 tile of
// the warp-level tensor product, so all heads of a group read the cache once.  Every warp
// walks its own chunks of 16 keys (chunk w, w + W, ... of the sequence, W warps in all)
// through its own ring of asynchronous copies, and meets no other warp until the end.  The
// warps of a CTA join through shared memory, the CTAs of a cluster (up to 8 share a
// sequence's keys) through distributed shared memory; only where that leaves SMs idle do
// further splits join through the workspace in a second launch.
//
// Bound by HBM: 4 G operations a byte of cache.  The 128-row tiles of the prompt kernel
// would do for it too, but their tensor memory, barriers and tile maps cost a decoding
// step more than its loads.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "fastdiv.cuh"
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace pvr {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 16;               // keys of a chunk
constexpr int kRows = 16;
constexpr int kStages = 3;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 30.0f;          // log2 growth of the maximum that triggers a rescale

struct DecodeArgs {
    const __nv_bfloat16 *q;
    int64_t q_ts, q_hs;
    __nv_bfloat16 *out;
    int64_t out_ts, out_hs;
    Pages pages;
    const int32_t *cu, *kv_lens;
    float *part_o, *part_lse;           // of each outer split, or NULL
    int32_t n_tokens, n_seqs, hq, hkv, group, d, causal, tile_tokens, splits;
    FastDiv div_page;
    float scale;
};

template <int DP>
struct Shared {
    static constexpr int kRowBytes = DP * 2;
    static constexpr int kChunkBytes = 2 * kKeys * kRowBytes;          // keys, then values
    static constexpr int kWarpBytes = kStages * kChunkBytes;
    static constexpr int kBytes = kWarps * kWarpBytes;
    // after the loop the same memory holds each warp's o (binary32)
    static_assert(kWarpBytes >= kRows * DP * 4, "o of a warp fits its ring");
};

// 16 bytes global to shared, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What CTA `rank` of the cluster holds at this CTA's shared address `addr`.
__device__ __forceinline__ float cluster_load(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("{\n .reg .u32 p;\n mapa.shared::cluster.u32 p, %1, %2;\n ld.shared::cluster.f32 %0, [p];\n}"
                 : "=f"(v) : "r"(addr), "r"(rank) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr, uint32_t rank)
{
    float4 v;
    asm volatile("{\n .reg .u32 p;\n mapa.shared::cluster.u32 p, %4, %5;\n"
                 " ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [p];\n}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr), "r"(rank) : "memory");
    return v;
}

template <int DP>
__global__ void __launch_bounds__(kThreads) attn_decode_kernel(const __grid_constant__ DecodeArgs a)
{
    using Sh = Shared<DP>;
    constexpr int kCols = DP / 8;                            // 16-byte columns of a row
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ float s_cm[kRows], s_cl[kRows];               // the CTA's
    __shared__ __align__(16) float s_o[kRows][DP];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int unit = blockIdx.x / ranks, split = unit % a.splits;
    const int kvh = unit / a.splits % a.hkv, slot = unit / a.splits / a.hkv;
    const TileSlot f = find_slot(a.cu, a.kv_lens, a.n_seqs, a.n_tokens, a.tile_tokens, slot);
    const int first = f.tile * a.tile_tokens, len = f.end - f.start;
    if (f.tile < 0 || first >= len) return;                  // the whole cluster
    const bool inside = f.sample >= 0 && f.sample < a.n_seqs;
    const int kv = inside ? max(f.used, -1) : 0;
    const int keys = inside ? static_cast<int>(min(static_cast<int64_t>(max(kv, 0)),
                                                   static_cast<int64_t>(a.pages.max_pages) * a.pages.page_size)) : 0;
    const int offset = kv - len;
    auto limit = [&](int i) {                                // keys that row i of the sample sees
        if (!inside || i >= len || i + offset < 0) return 0;
        return a.causal ? min(keys, i + offset + 1) : keys;
    };
    const int n_tok = min(a.tile_tokens, len - first);
    const int n_rows = n_tok * a.group;
    const int n_keys = limit(first + n_tok - 1);             // the most any row sees
    const int n_chunks = (n_keys + kKeys - 1) / kKeys;

    // this lane's rows of the m16 tile: lane / 4 and that + 8
    int lim[2];
    const __nv_bfloat16 *q_row[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = (lane >> 2) + 8 * r;
        const bool in = row < n_rows;
        const int tok = in ? row / a.group : 0, head = kvh * a.group + (in ? row - tok * a.group : 0);
        lim[r] = in ? limit(first + tok) : 0;
        q_row[r] = a.q + (f.start + first + tok) * a.q_ts + head * a.q_hs;
    }

    const uint32_t ring = smem_addr(smem) + warp * Sh::kWarpBytes;
    const int step = static_cast<int>(ranks) * a.splits * kWarps;
    int chunk = (split * static_cast<int>(ranks) + static_cast<int>(rank)) * kWarps + warp;
    const int32_t *table = a.pages.table + f.sample * a.pages.table_stride;
    // a chunk's copies: lane l takes 16-byte column l % kCols of rows l / kCols, + 32 / kCols, ...
    const int col = lane % kCols, row0 = lane / kCols;
    constexpr int kRowStep = 32 / kCols;
    const __nv_bfloat16 *k_base = a.pages.k + kvh * a.pages.k_hs + 8 * col;
    const __nv_bfloat16 *v_base = a.pages.v + kvh * a.pages.v_hs + 8 * col;
    const bool col_in = 8 * col < a.d;
    // page ids of the chunk's two groups of 8 keys (a page holds whole groups)
    auto pages_of = [&](int c, int (&id)[2], int (&at)[2]) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int key = c * kKeys + 8 * g;
            id[g] = -1;
            at[g] = 0;
            if (key < n_keys) {
                const int index = static_cast<int>(fast_div(static_cast<uint32_t>(key), a.div_page));
                at[g] = key - index * a.pages.page_size;
                id[g] = __ldg(table + index);
            }
        }
    };
    auto fetch = [&](int c, int stage, const int (&id)[2], const int (&at)[2]) {
        const uint32_t dst = ring + stage * Sh::kChunkBytes;
#pragma unroll
        for (int j = 0; j < kKeys / kRowStep; ++j) {
            const int r = row0 + j * kRowStep;
            const int g = r >> 3;
            const int page = g == 0 ? id[0] : id[1];
            const bool valid = col_in && page >= 0 && page < a.pages.n_pages && c * kKeys + r < n_keys;
            const int64_t slot_in = (g == 0 ? at[0] : at[1]) + (r & 7);
            const uint32_t to = dst + r * Sh::kRowBytes + ((col ^ (r & 7)) << 4);
            copy16(to, valid ? k_base + (page * a.pages.k_ps + slot_in * a.pages.k_ts) : a.q, valid);
            copy16(to + kKeys * Sh::kRowBytes, valid ? v_base + (page * a.pages.v_ps + slot_in * a.pages.v_ts) : a.q, valid);
        }
    };

    // the page ids of all chunks of the first round, then their copies
    int id[2], at[2];
    {
        int ids[kStages - 1][2], ats[kStages - 1][2];
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) pages_of(chunk + s * step, ids[s], ats[s]);
        pages_of(chunk + (kStages - 1) * step, id, at);
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            if (chunk + s * step < n_chunks) fetch(chunk + s * step, s, ids[s], ats[s]);
            copy_commit();
        }
    }

    // queries as the A operand: 16 x 16 per k step
    uint32_t qf[DP / 16][4];
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = 16 * s + 2 * (lane & 3) + 8 * (e >> 1);
            const bool in = c < a.d && (lane >> 2) + 8 * (e & 1) < n_rows;
            qf[s][e] = in ? __ldg(reinterpret_cast<const unsigned int *>(q_row[e & 1] + c)) : 0u;
        }
    }
    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const float c = a.scale * kLog2e;

    // ldmatrix addresses: matrix lane / 8, row lane % 8
    const int mi = lane >> 3, mr = lane & 7;
    int stage = 0;
    for (; chunk < n_chunks; chunk += step) {
        copy_wait<kStages - 2>();
        __syncwarp();
        {   // the stage read one turn ago is free: the next chunk goes there
            const int next = chunk + (kStages - 1) * step;
            const int to = stage == 0 ? kStages - 1 : stage - 1;
            if (next < n_chunks) {
                fetch(next, to, id, at);
                if (next + step < n_chunks) pages_of(next + step, id, at);
            }
            copy_commit();
        }
        const uint32_t kt = ring + stage * Sh::kChunkBytes, vt = kt + kKeys * Sh::kRowBytes;
        // S = Q K^T: two n8 tiles of 8 keys
        float s[2][4] = {};
#pragma unroll
        for (int k = 0; k < DP / 32; ++k) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t b[4];                               // 32 of d for 8 keys
                ldmatrix4(b, kt + (8 * n + mr) * Sh::kRowBytes + (((4 * k + mi) ^ mr) << 4));
                mma16816(s[n], qf[2 * k], b[0], b[1]);
                mma16816(s[n], qf[2 * k + 1], b[2], b[3]);
            }
        }
        bool grew = false;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = chunk * kKeys + 8 * n + 2 * (lane & 3) + (e & 1);
                if (key >= lim[e >> 1]) s[n][e] = -INFINITY;
                grew = grew || (s[n][e] - m[e >> 1]) * c > kGrow;
            }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float high = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, 1));
                high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, 2));
                const float grown = fmaxf(m[r], high);
                const float shrink = m[r] == grown ? 1.0f : ex2((m[r] - grown) * c);
                m[r] = grown;
                l[r] *= shrink;
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                    o[n][2 * r] *= shrink;
                    o[n][2 * r + 1] *= shrink;
                }
            }
        }
        uint32_t p[4];
        {
            float w[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float top = m[e >> 1];
                    w[n][e] = ex2((s[n][e] - (top == -INFINITY ? 0.0f : top)) * c);
                    l[e >> 1] += w[n][e];
                }
            p[0] = pack_bf16(w[0][0], w[0][1]);
            p[1] = pack_bf16(w[0][2], w[0][3]);
            p[2] = pack_bf16(w[1][0], w[1][1]);
            p[3] = pack_bf16(w[1][2], w[1][3]);
        }
        // O += P V: 16 keys, n8 tiles of d, two at a time
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
            uint32_t b[4];
            ldmatrix4_t(b, vt + (8 * (mi & 1) + mr) * Sh::kRowBytes + (((2 * n + (mi >> 1)) ^ mr) << 4));
            mma16816(o[2 * n], p, b[0], b[1]);
            mma16816(o[2 * n + 1], p, b[2], b[3]);
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copy_wait<0>();
    __syncwarp();

    // ---- join: the warps of the CTA
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if ((lane & 3) == 0) {
            s_m[warp][(lane >> 2) + 8 * r] = m[r];
            s_l[warp][(lane >> 2) + 8 * r] = l[r];
        }
    }
    float *mine = reinterpret_cast<float *>(smem + warp * Sh::kWarpBytes);
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2 *>(mine + ((lane >> 2) + 8 * r) * DP + 8 * n + 2 * (lane & 3)) =
                make_float2(o[n][2 * r], o[n][2 * r + 1]);
    __syncthreads();
    for (int i = threadIdx.x; i < n_rows * (DP / 4); i += kThreads) {
        const int row = i / (DP / 4), e = 4 * (i - row * (DP / 4));
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][row]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = s_m[w][row] == -INFINITY ? 0.0f : ex2((s_m[w][row] - top) * c);
            const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + w * Sh::kWarpBytes) +
                                                               row * DP + e);
            acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
            sum += f * s_l[w][row];
        }
        *reinterpret_cast<float4 *>(&s_o[row][e]) = acc;
        if (e == 0) {
            s_cm[row] = top;
            s_cl[row] = sum;
        }
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();

    // ---- join: the CTAs of the cluster; CTA r takes every ranks-th group of four elements
    const uint32_t a_o = smem_addr(s_o), a_m = smem_addr(s_cm), a_l = smem_addr(s_cl);
    for (int i = threadIdx.x * ranks + rank; i < n_rows * (DP / 4); i += kThreads * ranks) {
        const int row = i / (DP / 4), e = 4 * (i - row * (DP / 4));
        if (e >= a.d) continue;
        float top = -INFINITY, sum = 0.0f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ranks == 1) {
            top = s_cm[row];
            x = *reinterpret_cast<const float4 *>(&s_o[row][e]);
            sum = s_cl[row];
        } else {
            // all loads are independent (a CTA that saw no key holds zeros); past the cluster's
            // size they repeat its own
            float ms[kMaxCluster], ls[kMaxCluster];
            float4 os[kMaxCluster];
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                const uint32_t from = r < static_cast<int>(ranks) ? r : rank;
                ms[r] = cluster_load(a_m + 4 * row, from);
                ls[r] = cluster_load(a_l + 4 * row, from);
                os[r] = cluster_load4(a_o + 4 * (row * DP + e), from);
                if (r >= static_cast<int>(ranks)) ms[r] = -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) top = fmaxf(top, ms[r]);
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                const float f = ms[r] == -INFINITY ? 0.0f : ex2((ms[r] - top) * c);
                x.x += f * os[r].x; x.y += f * os[r].y; x.z += f * os[r].z; x.w += f * os[r].w;
                sum += f * ls[r];
            }
        }
        const int tok_in = row / a.group;
        const int head = kvh * a.group + row - tok_in * a.group;
        const int tok = f.start + first + tok_in;
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        x.x *= inv; x.y *= inv; x.z *= inv; x.w *= inv;
        if (a.splits == 1) {
            *reinterpret_cast<uint2 *>(a.out + tok * a.out_ts + head * a.out_hs + e) =
                make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
        } else {
            const int64_t to = static_cast<int64_t>(split) * a.n_tokens * a.hq + static_cast<int64_t>(tok) * a.hq + head;
            *reinterpret_cast<float4 *>(a.part_o + to * a.d + e) = x;
            if (e == 0) a.part_lse[to] = sum > 0.0f ? top * c + log2f(sum) : -INFINITY;
        }
    }
    if (ranks > 1) cluster_sync();      // no CTA leaves while its memory is read
}

template <int DP>
cudaError_t launch(const DecodeArgs &a, int cluster, int slots, cudaStream_t stream)
{
    static std::atomic<uint64_t> sized{0};
    const cudaError_t err = allow_smem(attn_decode_kernel<DP>, Shared<DP>::kBytes, sized);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster) * static_cast<unsigned>(a.splits) * static_cast<unsigned>(slots) *
                       static_cast<unsigned>(a.hkv));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shared<DP>::kBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, attn_decode_kernel<DP>, a);
}

}  // namespace

DecodePlan attn_decode_plan(const AttnProblem &p, int64_t max_kv)
{
    DecodePlan plan;
    // few rows a sequence, on average; longer stretches still come out right, a tile at a time
    plan.use = p.group <= kRows && static_cast<int64_t>(p.n_tokens) * p.group <= 2 * kRows * static_cast<int64_t>(p.n_seqs);
    if (!plan.use) return plan;
    plan.slots = slot_count(p.n_tokens, p.n_seqs, kRows / p.group);
    // live CTAs of one rank: a sequence with new tokens fills at least one slot
    const int64_t ctas = static_cast<int64_t>(p.n_seqs < p.n_tokens ? p.n_seqs : p.n_tokens) * p.hkv;
    const int64_t chunks = (max_kv + kKeys - 1) / kKeys;
    plan.cluster = 1;
    while (plan.cluster < kMaxCluster && ctas * plan.cluster < 8 * kSMs && chunks > 2 * plan.cluster * 2 * kWarps)
        plan.cluster *= 2;
    plan.splits = 1;
    while (ctas * plan.cluster * plan.splits * 2 <= kSMs && chunks > 32 * plan.cluster * plan.splits * kWarps &&
           plan.splits < 64)
        plan.splits *= 2;
    plan.use = static_cast<int64_t>(plan.slots) * p.hkv * plan.cluster * plan.splits <= INT32_MAX;
    return plan;
}

cudaError_t launch_attn_decode(const AttnProblem &p, const DecodePlan &plan, float *workspace, cudaStream_t stream)
{
    DecodeArgs a{};
    a.q = p.q.p;
    a.q_ts = p.q.ts;
    a.q_hs = p.q.hs;
    a.out = p.out.p;
    a.out_ts = p.out.ts;
    a.out_hs = p.out.hs;
    a.pages = p.pages;
    a.cu = p.cu;
    a.kv_lens = p.used;
    a.n_tokens = p.n_tokens;
    a.n_seqs = p.n_seqs;
    a.hq = p.hq;
    a.hkv = p.hkv;
    a.group = p.group;
    a.d = p.d;
    a.causal = p.causal;
    a.tile_tokens = kRows / p.group;
    a.splits = plan.splits;
    a.div_page = make_fastdiv(static_cast<uint32_t>(p.pages.page_size));
    a.scale = p.scale;
    const int64_t rows = static_cast<int64_t>(p.n_tokens) * p.hq;
    a.part_o = workspace;
    a.part_lse = plan.splits > 1 ? workspace + plan.splits * rows * p.d : nullptr;
    const cudaError_t err = p.d <= 64 ? launch<64>(a, plan.cluster, plan.slots, stream)
                                      : launch<128>(a, plan.cluster, plan.slots, stream);
    if (err != cudaSuccess || plan.splits == 1) return err;
    return launch_attn_join(a.part_o, a.part_lse, p, plan.splits, stream);
}

}  // namespace pvr
