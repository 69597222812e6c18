// Attention backward on the tensor cores (GB300, sm_103a), deterministic.
//
// Mathematics, per query row i and key j of its sample (lse, out from the forward):
//   D_i = do_i . o_i;  p_ij = exp(scale q_i.k_j - lse_i);  ds_ij = p_ij (do_i.v_j - D_i)
//   dq_i = scale sum_j ds_ij k_j;  dk_j = scale sum_i ds_ij q_i;  dv_j = sum_i p_ij do_i
//
// Two passes over the pairs, neither with an atomic: one CTA per 128 keys of a key head
// runs through the query rows of all G heads that share it and keeps dk and dv in tensor
// memory; one CTA per 128 rows of a query head runs through its keys and keeps dq.  The
// scores are computed in both (7 products instead of 5), which buys the same bits on every
// run and no binary32 gradients in HBM.
//
// One kernel serves both.  X1, X2 stay in shared memory (keys and values, or queries and
// output gradients: 128 rows); Y1, Y2 stream through TMA stages of 64 rows (queries and
// output gradients, or keys and values):
//   S  = X1 Y1^T, dP = X2 Y2^T     128x64 each, double-buffered in tensor memory
//   P  = exp2(c S - lse), dS = P (dP - D)  by one of two warpgroups (tiles alternate), written as
//                                  bf16 over S and dP
//   acc1 += dS Y1;  acc2 += P Y2 (keys only)   128xd in tensor memory
// S and dP of the next tile are issued before the products that wait for this tile's P and
// dS, so the tensor core works while a warpgroup computes.  Bound by the tensor core:
// 1280 cycles a tile for dk and dv (768 of them S and dP, whose 64-wide tiles are limited
// by reading X from shared memory), 1024 for dq.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace pvr {
namespace {

constexpr int kThreads = 384;              // two softmax warpgroups, one for products and loads
constexpr int kX = 128, kY = 64;           // rows of the resident and the streamed tiles
constexpr float kLog2e = 1.4426950408889634f;

__device__ int g_attn_bwd_fault;           // a bounded wait ran out

struct BwdArgs {
    CUtensorMap x1, x2, y1, y2;
    __nv_bfloat16 *out1, *out2;            // dk, dv, or dq
    int64_t o1_ts, o1_hs, o2_ts, o2_hs;
    const float2 *stats;                   // [hq, T]: (-lse log2(e), -D); -infinity first for rows not in use
    const int32_t *cu, *used;
    int32_t n_tokens, n_seqs, hq, hkv, group, d, causal, n_slots;
    FastDiv div_x;                         // by kX
    float scale;
};

template <int DP>
struct Shared {
    static constexpr int kBoxes = DP / 64;
    static constexpr int kXBytes = kX * DP * 2, kYBytes = kY * DP * 2;
    static constexpr int kStageBytes = 2 * kYBytes + 1024;            // + the rows' statistics
    static constexpr int kStages = DP == 128 ? 4 : 6;
    static constexpr int kOffY = 2 * kXBytes;
    static constexpr int kOffBars = kOffY + kStages * kStageBytes;
    static constexpr int kBytes = kOffBars + 256 + 1024;              // + alignment slack
};

// KEYS: dk and dv (X = keys and values); else dq (X = queries and output gradients).
template <int DP, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1) attn_bwd_kernel(const __grid_constant__ BwdArgs a)
{
    using Sh = Shared<DP>;
    constexpr int kStages = Sh::kStages;
    constexpr uint32_t kXBox = kX * 128, kYBox = kY * 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_addr(smem);
    const uint32_t bars = base + Sh::kOffBars;
    const uint32_t x_full = bars, s_full = bars + 16, p_full = bars + 32, done = bars + 48, drain = bars + 56,
                   acc_done = bars + 72, x_ready = bars + 88, y_full = bars + 96,
                   y_empty = y_full + 8 * kStages;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ TileSlot s_slot;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(x_full, 1);
        mbar_init(x_ready, 8);
        mbar_init(done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(drain + 8 * i, 1);
            mbar_init(acc_done + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(y_full + 8 * i, KEYS ? 2 : 1);
            mbar_init(y_empty + 8 * i, 1);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == 8) tmem_alloc(smem_addr(&s_tmem), 512);
    if (warp == 9 && lane == 0) {
        tma_prefetch_map(&a.x1);
        tma_prefetch_map(&a.x2);
        tma_prefetch_map(&a.y1);
        tma_prefetch_map(&a.y2);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int heads = KEYS ? a.hkv : a.hq;
    const int xhead = blockIdx.x % heads;
    // with a causal mask early keys and late queries have the most work: they go first
    const int order = static_cast<int>(blockIdx.x) / heads;
    const int slot = KEYS ? order : a.n_slots - 1 - order;
    if (warp == 0) {
        const TileSlot f = find_slot(a.cu, a.used, a.n_seqs, a.n_tokens, a.div_x, slot);
        if (lane == 0) s_slot = f;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const TileSlot where = s_slot;
    const int first = where.tile * kX;                       // of the sample
    const int len = where.end - where.start;
    const bool live = where.tile >= 0 && first < len;
    const int rows = min(len, max(where.used, 0));               // rows (and keys) in use
    // streamed tiles [y_lo, y_hi) of each pass, `passes` of them (the heads of the group)
    int y_lo = 0, y_hi = 0;
    if (live && first < rows) {
        if (KEYS) {
            y_lo = a.causal ? first / kY : 0;
            y_hi = (rows + kY - 1) / kY;
        } else {
            const int keys = a.causal ? min(rows, first + kX) : rows;
            y_hi = (keys + kY - 1) / kY;
        }
    }
    const int per_pass = y_hi - y_lo;
    const int n_tiles = per_pass * (KEYS ? a.group : 1);
    // tensor memory: S and dP twice, the accumulators, and, where there is room, X as bf16: an
    // operand read from there leaves shared memory to the other one, and 64-wide products run
    // at the tensor core's rate (32 cycles a k step) instead of shared memory's (48)
    constexpr uint32_t kColS = 0, kColP = 128, kCol1 = 256, kCol2 = 256 + DP;
    constexpr bool kXInTmem = !KEYS || DP == 64;
    constexpr uint32_t kColX = KEYS ? 256 + 2 * DP : 256 + DP;

    if (warp >= 8) {
        if (warp == 9) {
            // -------------------------------------------------------- loads
            int issued = 0;
            if (lane == 0 && n_tiles > 0) {
                mbar_expect_tx(x_full, 2 * Sh::kXBytes);
                for (int b = 0; b < Sh::kBoxes; ++b) {
                    tma_load_3d(base + b * kXBox, &a.x1, 64 * b, where.start + first, xhead, x_full);
                    tma_load_3d(base + Sh::kXBytes + b * kXBox, &a.x2, 64 * b, where.start + first, xhead, x_full);
                }
                int g = 0, y = y_lo;
                for (int t = 0; t < n_tiles; ++t) {
                    const int stage = t % kStages;
                    if (t >= kStages &&
                        !mbar_wait(y_empty + 8 * stage, (t / kStages - 1) & 1, &s_abort, &g_attn_bwd_fault))
                        break;
                    const uint32_t bar = y_full + 8 * stage, dst = base + Sh::kOffY + stage * Sh::kStageBytes;
                    mbar_expect_tx(bar, 2 * Sh::kYBytes);
                    const int yhead = KEYS ? xhead * a.group + g : xhead / a.group;
                    for (int b = 0; b < Sh::kBoxes; ++b) {
                        tma_load_3d(dst + b * kYBox, &a.y1, 64 * b, where.start + y * kY, yhead, bar);
                        tma_load_3d(dst + Sh::kYBytes + b * kYBox, &a.y2, 64 * b, where.start + y * kY, yhead, bar);
                    }
                    ++issued;
                    if (++y == y_hi) {
                        y = y_lo;
                        ++g;
                    }
                }
                if (s_abort != 0) {     // copies in flight land before the memory is given back
                    for (int t = max(0, issued - kStages); t < issued; ++t) {
                        if (KEYS) mbar_arrive(y_full + 8 * (t % kStages));   // for the statistics that may not come
                        mbar_drain(y_full + 8 * (t % kStages), (t / kStages) & 1);
                    }
                    mbar_drain(x_full, 0);
                }
            }
            __syncwarp();
        } else if (warp == 8 || warp == 11) {
            // ------- products: S and dP by warp 8, those with P and dS by warp 11
            bool ok = true;
            auto wait = [&](uint32_t bar, int phase) {
                if (ok) ok = warp_wait(bar, phase & 1, &s_abort, &g_attn_bwd_fault);
            };
            const uint32_t ubase = uniform(base), utmem = uniform(tmem);
            if (warp == 8) {
                constexpr uint32_t kDescS = mma_desc(kX, kY, false);
                const uint32_t d_x = desc_lo(ubase, 0), d_y = desc_lo(ubase + Sh::kOffY, 0);
                if (n_tiles > 0) wait(kXInTmem ? x_ready : x_full, 0);
                tc_fence_after();
                for (int t = 0; ok && t < n_tiles; ++t) {
                    const int stage = t % kStages, b = t & 1;
                    wait(y_full + 8 * stage, t / kStages);
                    // streamed rows past the sample's end (another sample's, or anything) are
                    // cleared: their weights are zero, but zero times NaN is not
                    const int valid = rows - (y_lo + t % per_pass) * kY;
                    if (ok && valid < kY) {
                        uint8_t *y = smem + Sh::kOffY + stage * Sh::kStageBytes;
                        for (int r = valid + (lane >> 3); r < kY; r += 4)
                            for (int i = 0; i < 2 * Sh::kBoxes; ++i)
                                *reinterpret_cast<uint4 *>(y + i * kYBox + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                        __syncwarp();
                    }
                    // the buffer's P and dS have been used
                    if (t >= 2) wait(acc_done + 8 * b, (t >> 1) - 1);
                    tc_fence_after();
                    if (ok && elect_one()) {
                        const uint32_t yd = d_y + stage * (Sh::kStageBytes >> 4);
#pragma unroll
                        for (int s = 0; s < DP / 16; ++s) {
                            const uint32_t ax = ((s / 4) * kXBox + (s % 4) * 32) >> 4, ay = ((s / 4) * kYBox + (s % 4) * 32) >> 4;
                            if (kXInTmem) mma_ts(utmem + kColS + b * kY, utmem + kColX + 8 * s, yd + ay, kDescS, s > 0);
                            else mma_ss(utmem + kColS + b * kY, d_x + ax, yd + ay, kDescS, s > 0);
                        }
#pragma unroll
                        for (int s = 0; s < DP / 16; ++s) {
                            const uint32_t ax = ((s / 4) * kXBox + (s % 4) * 32) >> 4, ay = ((s / 4) * kYBox + (s % 4) * 32) >> 4;
                            if (kXInTmem)
                                mma_ts(utmem + kColP + b * kY, utmem + kColX + DP / 2 + 8 * s, yd + (Sh::kYBytes >> 4) + ay,
                                       kDescS, s > 0);
                            else
                                mma_ss(utmem + kColP + b * kY, d_x + (Sh::kXBytes >> 4) + ax, yd + (Sh::kYBytes >> 4) + ay,
                                       kDescS, s > 0);
                        }
                        tc_commit(s_full + 8 * b);
                    }
                    __syncwarp();
                }
            } else {
                constexpr uint32_t kDescA = mma_desc(kX, DP, true);
                const uint32_t d_y = desc_lo(ubase + Sh::kOffY, kYBox);
                for (int t = 0; ok && t < n_tiles; ++t) {
                    const int stage = t % kStages, b = t & 1;
                    const uint32_t y = d_y + stage * (Sh::kStageBytes >> 4);
                    wait(p_full + 8 * b, t >> 1);
                    tc_fence_after();
                    if (ok && elect_one()) {
                        if (KEYS) {
#pragma unroll
                            for (int s = 0; s < kY / 16; ++s)
                                mma_ts(utmem + kCol2, utmem + kColS + b * kY + s * 8,
                                       y + (Sh::kYBytes >> 4) + s * (2048 >> 4), kDescA, t > 0 || s > 0);
                        }
#pragma unroll
                        for (int s = 0; s < kY / 16; ++s)
                            mma_ts(utmem + kCol1, utmem + kColP + b * kY + s * 8, y + s * (2048 >> 4), kDescA, t > 0 || s > 0);
                        tc_commit(acc_done + 8 * b);
                        tc_commit(y_empty + 8 * stage);
                        if (t + 1 == n_tiles) tc_commit(done);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {                  // products in flight finish before tensor memory is freed
                const uint32_t mine = drain + (warp == 8 ? 0 : 8);
                if (lane == 0) tc_commit(mine);
                mbar_drain(mine, 0);
            }
            __syncwarp();
        } else if (KEYS && warp == 10) {
            // --------------------- statistics of the streamed rows, per stage
            int g = 0, y = y_lo;
            for (int t = 0; t < n_tiles; ++t) {
                const int stage = t % kStages;
                const float2 *src = a.stats + static_cast<int64_t>(xhead * a.group + g) * a.n_tokens + where.start;
                float2 v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = y * kY + lane + 32 * i;
                    v[i] = r < rows ? __ldg(src + r) : make_float2(-INFINITY, 0.0f);
                }
                if (t >= kStages && !warp_wait(y_empty + 8 * stage, (t / kStages - 1) & 1, &s_abort, &g_attn_bwd_fault))
                    break;
                float *dst = reinterpret_cast<float *>(smem + Sh::kOffY + stage * Sh::kStageBytes + 2 * Sh::kYBytes);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    dst[lane + 32 * i] = v[i].x;
                    dst[kY + lane + 32 * i] = v[i].y;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(y_full + 8 * stage);
                if (++y == y_hi) {
                    y = y_lo;
                    ++g;
                }
            }
        }
    } else {
        // ---------------------------------------------------------- softmax
        const int w = warp >> 2;
        const int row = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + kColS + w * kY, t_p = tmem + lanes + kColP + w * kY;
        const int xi = first + row;                                    // key or query of the sample
        const float c = a.scale * kLog2e;
        float2 mine = make_float2(-INFINITY, 0.0f);
        if (!KEYS && live && xi < rows)
            mine = __ldg(a.stats + static_cast<int64_t>(xhead) * a.n_tokens + where.start + xi);
        const float2 c2 = make_float2(c, c);
        bool ok = true;
        if (kXInTmem && n_tiles > 0) {          // X1 by one group, X2 by the other, a row a thread
            ok = warp_wait(x_full, 0, &s_abort, &g_attn_bwd_fault);
            const uint32_t src = base + w * Sh::kXBytes + row * 128;
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) {              // 32 of d: four 16-byte columns, swizzled
                uint32_t r[16];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = 4 * j + e;
                    const float4 v = smem_load4(src + (col >> 3) * kXBox + (((col & 7) ^ (row & 7)) << 4));
                    r[4 * e] = __float_as_uint(v.x);
                    r[4 * e + 1] = __float_as_uint(v.y);
                    r[4 * e + 2] = __float_as_uint(v.z);
                    r[4 * e + 3] = __float_as_uint(v.w);
                }
                tmem_st16(tmem + lanes + kColX + w * (DP / 2) + 16 * j, r);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(x_ready);
        }
        for (int t = w; ok && t < n_tiles; t += 2) {
            const int y0 = (y_lo + t % per_pass) * kY;
            const int stage = t % kStages;
            ok = warp_wait(s_full + 8 * w, (t >> 1) & 1, &s_abort, &g_attn_bwd_fault);
            if (KEYS && ok) ok = warp_wait(y_full + 8 * stage, (t / kStages) & 1, &s_abort, &g_attn_bwd_fault);
            if (!ok) break;
            tc_fence_after();
            const uint32_t st = base + Sh::kOffY + stage * Sh::kStageBytes + 2 * Sh::kYBytes;
            // columns [from, to) are visible: keys of a query row, or queries of a key row
            int from = 0, to = kY;
            if (KEYS) {
                if (a.causal) from = max(0, xi - y0);
            } else {
                to = min(rows, a.causal ? xi + 1 : rows) - y0;
            }
            const bool masked = KEYS ? a.causal && y0 < first + kX : y0 + kY > (a.causal ? min(rows, first + 1) : rows);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t s[32], p[32], sp[16], sd[16];
                tmem_ld32(t_s + 32 * half, s);
                tmem_ld32(t_p + 32 * half, p);
                tc_wait_ld(s);
                tmem_loaded(p);
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float4 nl, nd;
                    if (KEYS) {
                        nl = smem_load4(st + 4 * (32 * half + j));
                        nd = smem_load4(st + 4 * (kY + 32 * half + j));
                    } else {
                        nl = make_float4(mine.x, mine.x, mine.x, mine.x);
                        nd = make_float4(mine.y, mine.y, mine.y, mine.y);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int e = j + 2 * h, col = 32 * half + e;
                        float2 pr = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2,
                                         h == 0 ? make_float2(nl.x, nl.y) : make_float2(nl.z, nl.w));
                        pr.x = ex2(pr.x);
                        pr.y = ex2(pr.y);
                        if (masked) {
                            if (col < from || col >= to) pr.x = 0.0f;
                            if (col + 1 < from || col + 1 >= to) pr.y = 0.0f;
                        }
                        const float2 ds = mul2(pr, add2(make_float2(__uint_as_float(p[e]), __uint_as_float(p[e + 1])),
                                                        h == 0 ? make_float2(nd.x, nd.y) : make_float2(nd.z, nd.w)));
                        sp[e / 2] = pack_bf16(pr.x, pr.y);
                        sd[e / 2] = pack_bf16(ds.x, ds.y);
                    }
                }
                // P and dS take half the columns: what they overwrite has been read
                if (KEYS) tmem_st16(t_s + 16 * half, sp);
                tmem_st16(t_p + 16 * half, sd);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 8 * w);
        }
        if (ok && n_tiles > 0) {
            ok = warp_wait(done, 0, &s_abort, &g_attn_bwd_fault);
            tc_fence_after();
        }
        // epilogue: dk by one group and dv by the other, or half of dq's columns each
        const bool mine_row = live && xi < len;
        const bool in_use = xi < rows && n_tiles > 0;
        const bool second = KEYS && w == 1;
        const float mult = second ? 1.0f : a.scale;
        __nv_bfloat16 *dst = (second ? a.out2 : a.out1) + (where.start + xi) * (second ? a.o2_ts : a.o1_ts) +
                             xhead * (second ? a.o2_hs : a.o1_hs);
        constexpr int kCols = KEYS ? DP : DP / 2;
        const int col0 = KEYS ? 0 : w * kCols;
        const uint32_t acc = tmem + lanes + (second ? kCol2 : kCol1) + col0;
#pragma unroll
        for (int j = 0; j < kCols / 32; ++j) {
            uint32_t o[32];
            __syncwarp();
            if (ok && n_tiles > 0) {
                tmem_ld32(acc + 32 * j, o);
                tc_wait_ld(o);
            }
            if (!ok || !mine_row) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = col0 + 32 * j + 8 * e;
                if (col >= a.d) continue;
                uint32_t q[4];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    q[f] = in_use ? pack_bf16(__uint_as_float(o[8 * e + 2 * f]) * mult,
                                              __uint_as_float(o[8 * e + 2 * f + 1]) * mult) : 0u;
                *reinterpret_cast<uint4 *>(dst + col) = make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// (-lse log2(e), -D) of every (head, token) row, D = dout . out.  Eight lanes a row, 16
// elements each (head_dim <= 128); HBM-bound.
__global__ void __launch_bounds__(256) attn_stats_kernel(const __nv_bfloat16 *__restrict__ dout, int64_t g_ts, int64_t g_hs,
                                                         const __nv_bfloat16 *__restrict__ out, int64_t o_ts, int64_t o_hs,
                                                         const float *__restrict__ lse, float2 *__restrict__ stats,
                                                         int n_tokens, int hq, int d)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t r = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
    const int part = threadIdx.x & 7;
    const bool in = r < static_cast<int64_t>(n_tokens) * hq;
    const int tok = in ? static_cast<int>(r / hq) : 0, head = in ? static_cast<int>(r % hq) : 0;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = 8 * (part + 8 * i);
        if (!in || col >= d) continue;
        const uint4 g = __ldg(reinterpret_cast<const uint4 *>(dout + tok * g_ts + head * g_hs + col));
        const uint4 o = __ldg(reinterpret_cast<const uint4 *>(out + tok * o_ts + head * o_hs + col));
        const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&gw[e]));
            const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&ow[e]));
            sum += x.x * y.x + x.y * y.y;
        }
    }
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (in && part == 0) {
        const int64_t at = static_cast<int64_t>(head) * n_tokens + tok;
        const float x = lse[at];
        // a row that sees no key has no weights
        stats[at] = x == -INFINITY ? make_float2(-INFINITY, 0.0f) : make_float2(-x * kLog2e, -sum);
    }
}

void plain_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute &attr, unsigned grid, unsigned threads, size_t smem,
                  cudaStream_t stream)
{
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
}

template <int DP, bool KEYS>
cudaError_t launch_pass(const AttnProblem &p, cudaStream_t stream)
{
    static std::atomic<uint64_t> sized{0};
    const cudaError_t err = allow_smem(attn_bwd_kernel<DP, KEYS>, Shared<DP>::kBytes, sized);
    if (err != cudaSuccess) return err;
    BwdArgs a;
    const Rows &x1 = KEYS ? p.k : p.q, &x2 = KEYS ? p.v : p.dout, &y1 = KEYS ? p.q : p.k, &y2 = KEYS ? p.dout : p.v;
    const int xh = KEYS ? p.hkv : p.hq, yh = KEYS ? p.hq : p.hkv;
    auto map = [&](CUtensorMap *m, const Rows &r, int heads, int rows) {
        const int64_t ext[3] = {p.d, p.n_tokens, heads}, st[3] = {1, r.ts, r.hs};
        const int box[3] = {64, rows, 1};
        return make_map(m, r.p, 3, ext, st, box);
    };
    if (!map(&a.x1, x1, xh, kX) || !map(&a.x2, x2, xh, kX) || !map(&a.y1, y1, yh, kY) || !map(&a.y2, y2, yh, kY))
        return cudaErrorInvalidValue;
    const Rows &o1 = KEYS ? p.dk : p.dq;
    a.out1 = o1.p;
    a.o1_ts = o1.ts;
    a.o1_hs = o1.hs;
    a.out2 = p.dv.p;
    a.o2_ts = p.dv.ts;
    a.o2_hs = p.dv.hs;
    a.stats = reinterpret_cast<const float2 *>(p.stats);
    a.cu = p.cu;
    a.used = p.used;
    a.n_tokens = p.n_tokens;
    a.n_seqs = p.n_seqs;
    a.hq = p.hq;
    a.hkv = p.hkv;
    a.group = p.group;
    a.d = p.d;
    a.causal = p.causal;
    a.n_slots = slot_count(p.n_tokens, p.n_seqs, kX);
    a.scale = p.scale;
    a.div_x = make_fastdiv(kX);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    plain_config(cfg, attr, static_cast<unsigned>(a.n_slots) * static_cast<unsigned>(xh), kThreads, Shared<DP>::kBytes,
                 stream);
    return cudaLaunchKernelEx(&cfg, attn_bwd_kernel<DP, KEYS>, a);
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnProblem &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    const int64_t threads = static_cast<int64_t>(p.n_tokens) * p.hq * 8;
    plain_config(cfg, attr, static_cast<unsigned>((threads + 255) / 256), 256, 0, stream);
    cudaError_t err = cudaLaunchKernelEx(&cfg, attn_stats_kernel, static_cast<const __nv_bfloat16 *>(p.dout.p), p.dout.ts,
                                         p.dout.hs, static_cast<const __nv_bfloat16 *>(p.out.p), p.out.ts, p.out.hs,
                                         static_cast<const float *>(p.lse), reinterpret_cast<float2 *>(p.stats),
                                         static_cast<int>(p.n_tokens), static_cast<int>(p.hq), static_cast<int>(p.d));
    if (err != cudaSuccess) return err;
    err = p.d <= 64 ? launch_pass<64, true>(p, stream) : launch_pass<128, true>(p, stream);
    if (err != cudaSuccess) return err;
    return p.d <= 64 ? launch_pass<64, false>(p, stream) : launch_pass<128, false>(p, stream);
}

int attn_bwd_fault_word(int *word)
{
    return cudaMemcpyFromSymbol(word, g_attn_bwd_fault, sizeof *word) == cudaSuccess ? 0 : -1;
}

}  // namespace pvr
