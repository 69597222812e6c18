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
// through its own ring of TMA loads, and meets no other warp until the end.  The
// warps of a CTA join through shared memory, the CTAs of a cluster (up to 8 share a
// sequence's keys) through distributed shared memory; only where that leaves SMs idle do
// further splits join through the workspace in a second launch.
//
// Rules on the scores (score_rule.cuh), an instance each: a few operations a score more, hidden by the
// loads (the batch below, capped: 327-333 us; another draw of it, 1.42 GB: plain 226.5, prefixes 226.7,
// capped 226.8, slopes of a geometric series from 2^-0.25 to 2^-8 231.1, both 239.0 us).  Keys go upwards, so that
// with steep slopes a row's maximum moves at nearly every chunk; 2 % is what that costs.
//
// Bound by HBM: G operations a byte of cache (64 sequences of 500-16,000 tokens, 32/8 heads
// of 128: 325-330 us for 2.2 GB, 6.7-6.8 TB/s, a copy's rate); a short sequence by the chain of
// its dependent steps (one of 4,098 tokens 10.7 us, of which 2.5 us of loads).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "fastdiv.cuh"
#include "score_rule.cuh"
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace pvr {
namespace {

constexpr int kKeys = 16;               // keys of a chunk
constexpr int kRows = 16;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 30.0f;          // log2 growth of the maximum that triggers a rescale

__device__ int g_attn_decode_fault;     // bounded waits that ran out

struct DecodeArgs {
    CUtensorMap q, k, v;
    __nv_bfloat16 *out;
    int64_t out_ts, out_hs;
    const int32_t *table;
    int64_t table_stride;
    int32_t max_pages, page_size, n_pages, box_rows;
    const int32_t *cu, *kv_lens;
    float *part_o, *part_lse;           // of each outer split, or NULL
    int32_t n_tokens, n_seqs, hq, hkv, group, d, causal, tile_tokens, splits;
    FastDiv div_page, div_tile, div_group;
    float scale;
    ScoreRule rule;
};

template <int DP, int WARPS>
struct Shared {
    static constexpr int kRowBytes = DP * 2, kHalves = DP / 64;
    static constexpr int kChunkBytes = 2 * kKeys * kRowBytes;          // keys, then values, 64 of d at a time
    // more chunks in flight against fewer resident CTAs: head_dim 64 with 3, 4, 5 stages, 64 x
    // 500-16,000 keys 211, 201, 242 us, 16 x 1,024 keys 13.0, 12.1, 11.6
    static constexpr int kStages = DP == 128 ? 3 : 4;
    static constexpr int kWarpBytes = kStages * kChunkBytes;
    static constexpr int kOffQ = WARPS * kWarpBytes;
    static constexpr int kBytes = kOffQ + kRows * kRowBytes + 1024;    // + alignment slack
    static_assert(kStages <= 5, "the first round of loads is four chunks of eight lanes");
    // after the loop the same memory holds each warp's o (binary32)
    static_assert(kWarpBytes >= kRows * DP * 4, "o of a warp fits its ring");
};

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

template <int DP, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) attn_decode_kernel(const __grid_constant__ DecodeArgs a)
{
    using Sh = Shared<DP, WARPS>;
    constexpr int kThreads = 32 * WARPS, kStages = Sh::kStages;
    constexpr int kItems = kRows * DP / 4;                   // groups of four elements of o
    constexpr uint32_t kHalfBytes = kKeys * 128;             // 64 of d of a chunk's keys
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t s_full[WARPS][kStages], s_qfull;
    __shared__ float s_m[WARPS][kRows], s_l[WARPS][kRows];
    // what the cluster's CTAs send: m and l of every row, and of o this CTA's share
    __shared__ float s_pm[kMaxCluster][kRows], s_pl[kMaxCluster][kRows];
    __shared__ float4 s_po[kItems];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full = smem_addr(&s_full[warp][0]), q_full = smem_addr(&s_qfull);
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(full + 8 * i, 1);
        if (warp == 0) mbar_init(q_full, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int unit = blockIdx.x / ranks, split = unit % a.splits;
    const int kvh = unit / a.splits % a.hkv, slot = unit / a.splits / a.hkv;
    const TileSlot f = find_slot(a.cu, a.kv_lens, a.n_seqs, a.n_tokens, a.div_tile, slot);
    const int first = f.tile * a.tile_tokens, len = f.end - f.start;
    if (f.tile < 0 || first >= len) return;                  // the whole cluster
    if (ranks > 1) cluster_arrive();                         // this CTA runs: its memory may be written
    const bool inside = f.sample >= 0 && f.sample < a.n_seqs;
    const int kv = inside ? max(f.used, -1) : 0;
    const int keys = inside ? min(max(kv, 0), a.max_pages * a.page_size) : 0;
    const int offset = kv - len;
    const int prefix = prefix_of(a.rule, f.sample, a.n_seqs, keys);
    auto limit = [&](int i) {                                // keys that row i of the sample sees
        if (!inside || i >= len || i + offset < 0) return 0;
        const int own = a.causal ? min(keys, i + offset + 1) : keys;
        return kRuled ? max(own, prefix) : own;
    };
    const int n_tok = min(a.tile_tokens, len - first);
    const int n_rows = n_tok * a.group;
    const int n_keys = limit(first + n_tok - 1);             // the most any row sees
    const int n_chunks = (n_keys + kKeys - 1) / kKeys;

    // loads: a chunk is up to 8 boxes (keys or values, 64 of d, 16 or 8 keys), a lane each
    const uint32_t ring = smem_addr(smem) + warp * Sh::kWarpBytes;
    const int step = static_cast<int>(ranks) * a.splits * WARPS;
    int chunk = (split * static_cast<int>(ranks) + static_cast<int>(rank)) * WARPS + warp;
    const int box = lane & 7;
    const int box_half = Sh::kHalves == 2 ? (box >> 1) & 1 : 0, box_key = (box >> Sh::kHalves) * a.box_rows;
    const bool box_in = box_key < kKeys;
    const uint32_t box_to = ((box & 1) * Sh::kHalves + box_half) * kHalfBytes + box_key * 128;
    const CUtensorMap *map = (box & 1) == 0 ? &a.k : &a.v;
    int page = a.n_pages, in_page = 0;                       // of this lane's box in the next chunk
    // past the keys, and for a page id outside the pool, a coordinate past the pool's end: zeros
    auto find_page = [&](int c) {
        const int key = c * kKeys + box_key;
        page = a.n_pages;
        in_page = 0;
        if (box_in && key < n_keys) {
            const int index = static_cast<int>(fast_div(static_cast<uint32_t>(key), a.div_page));
            in_page = key - index * a.page_size;
            page = __ldg(a.table + f.sample * a.table_stride + index);
            if (page < 0 || page >= a.n_pages) page = a.n_pages;
        }
    };
    auto fetch = [&](int stage) {
        if (box == 0) mbar_expect_tx(full + 8 * stage, Sh::kChunkBytes);
        if (box_in)
            tma_load_4d(ring + stage * Sh::kChunkBytes + box_to, map, 64 * box_half, in_page, kvh, page, full + 8 * stage);
    };
    // the first round: the ring but one stage at once, eight lanes a chunk
    if (warp == 0 && lane == 31) {
        mbar_expect_tx(q_full, static_cast<uint32_t>(a.group * a.tile_tokens) * Sh::kRowBytes);
        for (int h = 0; h < Sh::kHalves; ++h)
            tma_load_3d(smem_addr(smem) + Sh::kOffQ + h * kRows * 128, &a.q, 64 * h, kvh * a.group, f.start + first, q_full);
    }
    {
        const int s = lane >> 3;
        find_page(chunk + s * step);
        if (s < kStages - 1 && chunk + s * step < n_chunks) fetch(s);
    }
    find_page(chunk + (kStages - 1) * step);

    // this lane's rows of the m16 tile: lane / 4 and that + 8
    int lim[2], own_key[2];
    float slope2[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = (lane >> 2) + 8 * r, tok_in = static_cast<int>(fast_div(row, a.div_group));
        lim[r] = row < n_rows ? limit(first + tok_in) : 0;
        own_key[r] = first + tok_in + offset;
        slope2[r] = kBias && row < n_rows ? a.rule.slopes[kvh * a.group + row - tok_in * a.group] * kLog2e : 0.0f;
    }
    // ldmatrix addresses: matrix lane / 8, row lane % 8
    const int mi = lane >> 3, mr = lane & 7;
    bool ok = true;
    auto wait = [&](uint32_t bar, int phase) {
        return warp_wait(bar, phase & 1, nullptr, &g_attn_decode_fault);
    };
    // queries as the A operand: 16 x 16 per k step (rows past the tile's hold anything: they
    // see no key)
    uint32_t qf[DP / 16][4];
    ok = wait(q_full, 0);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        const int r = 8 * (mi & 1) + mr, col = 2 * s + (mi >> 1);
        ldmatrix4(qf[s], smem_addr(smem) + Sh::kOffQ + (col >> 3) * kRows * 128 + r * 128 + (((col & 7) ^ mr) << 4));
    }
    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const float c = kShaped ? 1.0f : a.scale * kLog2e;       // shaped scores are exponents of 2

    int stage = 0, turn = 0;
    for (; ok && chunk < n_chunks; chunk += step) {
        if (!(ok = wait(full + 8 * stage, turn))) break;
        {   // the stage read one turn ago is free: the next chunk goes there
            const int next = chunk + (kStages - 1) * step;
            if (next < n_chunks) {
                if (lane < 8) fetch(stage == 0 ? kStages - 1 : stage - 1);
                find_page(next + step);
            }
        }
        const uint32_t kt = ring + stage * Sh::kChunkBytes, vt = kt + Sh::kHalves * kHalfBytes;
        // value rows past the last key may hold anything: their weights are zero, but zero
        // times NaN is not
        const int valid = n_keys - chunk * kKeys;
        if (valid < kKeys) {
            for (int r = valid + (lane >> 3); r < kKeys; r += 4)
                for (int h = 0; h < Sh::kHalves; ++h)
                    *reinterpret_cast<uint4 *>(smem + warp * Sh::kWarpBytes + stage * Sh::kChunkBytes +
                                               (Sh::kHalves + h) * kHalfBytes + r * 128 + (lane & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        // S = Q K^T: two n8 tiles of 8 keys
        float s[2][4] = {};
#pragma unroll
        for (int k = 0; k < DP / 32; ++k) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t b[4];                               // 32 of d for 8 keys
                const int col = 4 * k + mi;
                ldmatrix4(b, kt + (col >> 3) * kHalfBytes + (8 * n + mr) * 128 + (((col & 7) ^ mr) << 4));
                mma16816(s[n], qf[2 * k], b[0], b[1]);
                mma16816(s[n], qf[2 * k + 1], b[2], b[3]);
            }
        }
        bool grew = false;
        auto shape_chunk = [&](auto form) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {                // two neighbouring keys of a row
                    uint32_t x[2] = {__float_as_uint(s[n][2 * r]), __float_as_uint(s[n][2 * r + 1])};
                    shape<decltype(form)::value>(
                        a.rule, x, slope2[r], static_cast<float>(chunk * kKeys + 8 * n + 2 * (lane & 3) - own_key[r]), 0.0f);
                    s[n][2 * r] = __uint_as_float(x[0]);
                    s[n][2 * r + 1] = __uint_as_float(x[1]);
                }
        };
        if (kShaped) {
            if (kCap && a.rule.large) shape_chunk(FormTag<kLarge>{});
            else shape_chunk(FormTag<kAny>{});
        }
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
            const int col = 2 * n + (mi >> 1);
            ldmatrix4_t(b, vt + (col >> 3) * kHalfBytes + (8 * (mi & 1) + mr) * 128 + (((col & 7) ^ mr) << 4));
            mma16816(o[2 * n], p, b[0], b[1]);
            mma16816(o[2 * n + 1], p, b[2], b[3]);
        }
        if (++stage == kStages) {
            stage = 0;
            ++turn;
        }
    }
    if (!ok) {                          // copies in flight land before the memory is used again
        for (int s = 0; s < kStages; ++s) mbar_drain(full + 8 * s, (turn + (s < stage ? 1 : 0)) & 1);
    }
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

    // ---- and the CTAs of the cluster: item i of o goes to CTA i % ranks
    if (ranks > 1) cluster_wait();
    const int share = kItems / static_cast<int>(ranks);
    for (int i = threadIdx.x; i < n_rows * (DP / 4); i += kThreads) {
        const int row = i / (DP / 4), e = 4 * (i - row * (DP / 4));
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_m[w][row]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = s_m[w][row] == -INFINITY ? 0.0f : ex2((s_m[w][row] - top) * c);
            const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + w * Sh::kWarpBytes) +
                                                               row * DP + e);
            acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
            sum += f * s_l[w][row];
        }
        const uint32_t to = i % ranks;
        cluster_store4(smem_addr(&s_po[rank * share + i / ranks]), to, acc);
        if (e < 4 * static_cast<int>(ranks)) {               // the row's first `ranks` items, one to each CTA
            cluster_store(smem_addr(&s_pm[rank][row]), e >> 2, top);
            cluster_store(smem_addr(&s_pl[rank][row]), e >> 2, sum);
        }
    }
    if (ranks > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    for (int j = threadIdx.x; j * ranks + rank < n_rows * (DP / 4); j += kThreads) {
        const int i = j * ranks + rank, row = i / (DP / 4), e = 4 * (i - row * (DP / 4));
        if (e >= a.d) continue;
        float top = -INFINITY, sum = 0.0f;
        for (uint32_t r = 0; r < ranks; ++r) top = fmaxf(top, s_pm[r][row]);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t r = 0; r < ranks; ++r) {
            const float f = s_pm[r][row] == -INFINITY ? 0.0f : ex2((s_pm[r][row] - top) * c);
            const float4 y = s_po[r * share + j];
            x.x += f * y.x; x.y += f * y.y; x.z += f * y.z; x.w += f * y.w;
            sum += f * s_pl[r][row];
        }
        const int tok_in = static_cast<int>(fast_div(row, a.div_group));
        const int head = kvh * a.group + row - tok_in * a.group;
        const int tok = f.start + first + tok_in;
        // no weight is sum == 0, not !(sum > 0): a NaN score makes the sum NaN, and that must come out
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        x.x *= inv; x.y *= inv; x.z *= inv; x.w *= inv;
        if (a.splits == 1) {
            *reinterpret_cast<uint2 *>(a.out + tok * a.out_ts + head * a.out_hs + e) =
                make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
        } else {
            const int64_t to = static_cast<int64_t>(split) * a.n_tokens * a.hq + static_cast<int64_t>(tok) * a.hq + head;
            *reinterpret_cast<float4 *>(a.part_o + to * a.d + e) = x;
            if (e == 0) a.part_lse[to] = sum == 0.0f ? -INFINITY : top * c + log2f(sum);
        }
    }
}

template <int DP, int WARPS>
cudaError_t launch(const DecodeArgs &a, int cluster, int slots, cudaStream_t stream)
{
    static std::atomic<uint64_t> sized{0};
    const cudaError_t err = allow_smem(attn_decode_kernel<DP, WARPS>, Shared<DP, WARPS>::kBytes, sized);
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
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = Shared<DP, WARPS>::kBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, attn_decode_kernel<DP, WARPS>, a);
}

}  // namespace

#if PVR_SCORE_RULE == 0
DecodePlan attn_decode_plan(const AttnProblem &p, int64_t max_kv)
{
    DecodePlan plan;
    // at most one tile of rows a sequence, on average (longer stretches still come out right, a
    // tile at a time).  16 sequences, 4,096 tokens cached, 32/8 heads of 128, this kernel and the
    // 128-row one: 4 rows 50 and 55 us, 16 rows 53 and 56 us, 32 rows 87 and 55 us.
    plan.use = p.group <= kRows && static_cast<int64_t>(p.n_tokens) * p.group <= kRows * static_cast<int64_t>(p.n_seqs);
    if (!plan.use) return plan;
    plan.slots = slot_count(p.n_tokens, p.n_seqs, kRows / p.group);
    // live CTAs of one rank: a sequence with new tokens fills at least one slot
    const int64_t ctas = static_cast<int64_t>(p.n_seqs < p.n_tokens ? p.n_seqs : p.n_tokens) * p.hkv;
    const int64_t chunks = (max_kv + kKeys - 1) / kKeys;
    // CTAs of a cluster share a sequence's keys: while the SMs hold all CTAs at once (a CTA an
    // SM; two of half the size with head_dim up to 64), and so that none has more than about
    // 5,000 keys, as lengths are uneven.  32/8 heads of 128, one token each, by 1, 2, 4, 8 CTAs:
    // 1 x 4,096 keys 17, 17, 15, 11 us; 16 x 1,024 14, 14, 19, 29; 64 x 4,096 156, 173, 178, 210;
    // 64 x 500-16,000 389, 343, 321, -.
    const int64_t room = p.d <= 64 ? 2 * kSMs : kSMs;
    const int most = chunks > 512 ? 4 : kMaxCluster;      // clusters of 8 leave SMs of a GPC idle
    plan.cluster = 1;
    while (plan.cluster < most && chunks > 16 * plan.cluster &&
           (ctas * plan.cluster * 2 <= room || chunks > 320 * plan.cluster))
        plan.cluster *= 2;
    // and a second launch joins further splits of few long sequences (1 x 32,768 keys: 33 us as
    // 4 splits of 4, 50 us as 2 of 8)
    plan.splits = 1;
    while (ctas * plan.cluster * plan.splits * 2 <= kSMs && chunks > 128 * plan.cluster * plan.splits && plan.splits < 64)
        plan.splits *= 2;
    // with a CTA an SM at most, eight warps each keep more loads in flight (1 x 4,096 keys:
    // 10.7 us, 12.7 with four)
    plan.warps = ctas * plan.cluster * plan.splits <= kSMs ? 8 : 4;
    plan.use = static_cast<int64_t>(plan.slots) * p.hkv * plan.cluster * plan.splits <= INT32_MAX;
    return plan;
}

cudaError_t launch_attn_decode(const AttnProblem &p, const DecodePlan &plan, float *workspace, cudaStream_t stream)
{
    return for_rule(p.rule(), [&](auto rule) { return launch_attn_decode_rule<decltype(rule)::value>(p, plan, workspace, stream); });
}

int attn_decode_fault_word(int *word)
{
    return sum_fault_words(word, [](auto rule, int *w) { return attn_decode_fault_of<decltype(rule)::value>(w); });
}
#endif

template <>
cudaError_t launch_attn_decode_rule<kRule>(const AttnProblem &p, const DecodePlan &plan, float *workspace, cudaStream_t stream)
{
    DecodeArgs a;
    const int tile = kRows / p.group;
    a.box_rows = p.pages.page_size % kKeys == 0 ? kKeys : 8;
    if (!make_q_map(&a.q, p, tile) || !make_page_maps(&a.k, &a.v, p, a.box_rows)) return cudaErrorInvalidValue;
    a.out = p.out.p;
    a.out_ts = p.out.ts;
    a.out_hs = p.out.hs;
    a.table = p.pages.table;
    a.table_stride = p.pages.table_stride;
    a.max_pages = p.pages.max_pages;
    a.page_size = p.pages.page_size;
    a.n_pages = p.pages.n_pages;
    a.cu = p.cu;
    a.kv_lens = p.used;
    a.n_tokens = p.n_tokens;
    a.n_seqs = p.n_seqs;
    a.hq = p.hq;
    a.hkv = p.hkv;
    a.group = p.group;
    a.d = p.d;
    a.causal = p.causal;
    a.tile_tokens = tile;
    a.splits = plan.splits;
    a.div_tile = make_fastdiv(static_cast<uint32_t>(a.tile_tokens));
    a.div_group = make_fastdiv(static_cast<uint32_t>(p.group));
    a.div_page = make_fastdiv(static_cast<uint32_t>(p.pages.page_size));
    a.scale = p.scale;
    a.rule = rule_of(p);
    const int64_t rows = static_cast<int64_t>(p.n_tokens) * p.hq;
    a.part_o = workspace;
    a.part_lse = plan.splits > 1 ? workspace + plan.splits * rows * p.d : nullptr;
    const cudaError_t err = plan.warps == 8
                                ? (p.d <= 64 ? launch<64, 8>(a, plan.cluster, plan.slots, stream)
                                             : launch<128, 8>(a, plan.cluster, plan.slots, stream))
                                : (p.d <= 64 ? launch<64, 4>(a, plan.cluster, plan.slots, stream)
                                             : launch<128, 4>(a, plan.cluster, plan.slots, stream));
    if (err != cudaSuccess || plan.splits == 1) return err;
    return launch_attn_join(a.part_o, a.part_lse, p, plan.splits, stream);
}

template <>
int attn_decode_fault_of<kRule>(int *word)
{
    return read_fault_word(word, g_attn_decode_fault);
}

}  // namespace pvr
