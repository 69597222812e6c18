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
// output gradients: 128 rows); Y1, Y2 stream through TMA in tiles of 128 rows (queries and
// output gradients, or keys and values):
//   S  = X1 Y1^T, dP = X2 Y2^T     128x128 in tensor memory
//   P  = exp2(c S - lse), dS = P (dP - D)    four warpgroups, 32 columns of a row a thread,
//                                  written as bf16 over S and dP
//   acc1 += dS Y1;  acc2 += P Y2 (keys only)   128xd in tensor memory
// The products are issued in an order that keeps the tensor core busy while the warpgroups
// compute, although tensor memory holds S and dP only once: for keys dP(t), dV(t), S(t+1),
// dK(t), so that P(t) has the time of dK(t-1) and dP(t), and dS(t) that of dV(t) and S(t+1);
// for queries, with two dP and no P to keep, S(t+1), dP(t+1), dQ(t).  Products of one issuer
// run in the order of issue: one that overwrites an operand of an earlier one follows it.
// The issuing warp waits twice a tile: the arrival of Y is folded into the barrier of P by a
// warp that watches it, as a wait costs some 200 cycles while the tensor core reads shared
// memory.
//
// Bound by the tensor core: 2048 cycles a 128x128 tile for dk and dv, 1536 for dq.  32/8 heads
// of 128, causal: one sample of 32,768 tokens 19.7-19.9 ms, 1,108-1,118 TFLOP/s by the five
// products it needs, 1,551-1,565 by the seven it runs, and 20.0 ms over 0.8 s under the power
// limit (the library's sustain 1,705); 8,192 tokens 1.30 and 1.35 ms.

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

constexpr int kThreads = 640;              // four softmax warpgroups, one for products and loads
constexpr int kMmaWarp = 16, kWatchWarp = 17;
constexpr int kLoadWarp = 18;              // loads: one warp for X, Y1 and its statistics, one for Y2
constexpr int kTile = 128;                 // rows of the resident and of the streamed tiles
constexpr float kLog2e = 1.4426950408889634f;

__device__ int g_attn_bwd_fault;           // bounded waits that ran out

struct BwdArgs {
    CUtensorMap x1, x2, y1, y2;
    __nv_bfloat16 *out1, *out2;            // dk, dv, or dq
    int64_t o1_ts, o1_hs, o2_ts, o2_hs;
    float2 *stats;                         // [hq, T]: (-lse log2(e), -D); -infinity first for rows not in use
    const int32_t *cu, *used;
    int32_t n_tokens, n_seqs, hq, hkv, group, d, causal, n_slots;
    FastDiv div_tile;                      // by kTile
    float scale;
};

template <int DP>
struct Shared {
    static constexpr int kBoxes = DP / 64;
    static constexpr int kTileBytes = kTile * DP * 2;
    // Y1 stays from S(t) to the accumulation of tile t, past S(t + 1): three tiles of it are
    // held, so that the next one loads meanwhile; of Y2 two
    static constexpr int kY1 = 3, kY2 = 2;
    static constexpr int kOffY = 2 * kTileBytes;                      // Y1 tiles, then Y2 tiles
    static constexpr int kOffStats = kOffY + (kY1 + kY2) * kTileBytes;   // of even and odd tiles: -lse, then -D
    static constexpr int kOffBars = kOffStats + 2 * 2 * kTile * 4;
    static constexpr int kOffRest = kOffBars + 192;
    static constexpr int kBytes = kOffRest + 64;
};

// What a CTA shares besides tiles and barriers.
struct Rest {
    uint32_t tmem;
    int abort;
    TileSlot slot;
};

// KEYS: dk and dv (X = keys and values); else dq (X = queries and output gradients).
template <int DP, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1) attn_bwd_kernel(const __grid_constant__ BwdArgs a)
{
    using Sh = Shared<DP>;
    constexpr uint32_t kBox = kTile * 128;
    // all of the shared memory there is: tiles on 1024-byte boundaries with no slack
    extern __shared__ __align__(1024) uint8_t smem[];
    static_assert(sizeof(Rest) <= 64 && Sh::kBytes <= 227 * 1024, "shared memory");
    const uint32_t base = smem_addr(smem);
    const uint32_t bars = base + Sh::kOffBars;
    const uint32_t x_full = bars, s_full = bars + 8, p_full = bars + 16, ds_full = bars + 24, done = bars + 32,
                   drain = bars + 40, dp_full = bars + 48, st_full = bars + 64, st_empty = bars + 80, first_full = bars + 96,
                   y_full = bars + 104,
                   y_empty = y_full + 8 * (Sh::kY1 + Sh::kY2);
    Rest &rest = *reinterpret_cast<Rest *>(smem + Sh::kOffRest);
    volatile int &s_abort = rest.abort;
    // where tile t of Y1 (0) or Y2 (1) is, and how often that place was used before
    auto place = [](int t, int which) { return which == 0 ? t % Sh::kY1 : Sh::kY1 + t % Sh::kY2; };
    auto turn = [](int t, int which) { return which == 0 ? t / Sh::kY1 : t / Sh::kY2; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(x_full, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, 17);
        mbar_init(ds_full, 16);
        mbar_init(done, 1);
        mbar_init(drain, 1);
        mbar_init(first_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(dp_full + 8 * i, 1);
            mbar_init(st_full + 8 * i, 1);
            mbar_init(st_empty + 8 * i, 1);
        }
        for (int i = 0; i < Sh::kY1 + Sh::kY2; ++i) {
            mbar_init(y_full + 8 * i, 1);
            mbar_init(y_empty + 8 * i, 1);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&rest.tmem), 512);
    if (warp == kLoadWarp && lane == 0) {
        tma_prefetch_map(&a.x1);
        tma_prefetch_map(&a.x2);
        tma_prefetch_map(&a.y1);
        tma_prefetch_map(&a.y2);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // the CTAs of a cluster share the streamed tiles of one tile of keys
    const int ranks = KEYS ? static_cast<int>(cluster_size()) : 1, rank = KEYS ? static_cast<int>(cluster_rank()) : 0;
    const int unit = static_cast<int>(blockIdx.x) / ranks;
    const int heads = KEYS ? a.hkv : a.hq;
    const int xhead = unit % heads;
    // with a causal mask early keys and late queries have the most work: they go first
    const int order = unit / heads;
    const int slot = KEYS ? order : a.n_slots - 1 - order;
    if (warp == 0) {
        const TileSlot f = find_slot(a.cu, a.used, a.n_seqs, a.n_tokens, a.div_tile, slot);
        if (lane == 0) rest.slot = f;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = rest.tmem;
    const TileSlot where = rest.slot;
    const int first = where.tile * kTile;                    // of the sample
    const int len = where.end - where.start;
    const bool live = where.tile >= 0 && first < len;
    const int rows = min(len, max(where.used, 0));           // rows (and keys) in use
    // streamed tiles [y_lo, y_hi) of each pass; a pass for every head of the group
    int y_lo = 0, y_hi = 0;
    if (live && first < rows) {
        if (KEYS && a.causal) y_lo = where.tile;
        y_hi = ((!KEYS && a.causal ? min(rows, first + kTile) : rows) + kTile - 1) / kTile;
    }
    const int per_pass = y_hi - y_lo;
    const int n_all = per_pass * (KEYS ? a.group : 1);       // the cluster's
    int n_tiles = n_all, head0 = 0, y0_first = y_lo;
    if (KEYS && ranks > 1 && n_all > 0) {
        const int from = static_cast<int>(static_cast<int64_t>(n_all) * rank / ranks);
        n_tiles = static_cast<int>(static_cast<int64_t>(n_all) * (rank + 1) / ranks) - from;
        head0 = from / per_pass;
        y0_first = y_lo + from - head0 * per_pass;
    }
    // tensor memory; for queries dP is there twice
    constexpr uint32_t kColS = 0, kColP = 128, kCol1 = KEYS ? 256 : 384, kCol2 = 256 + DP;
    constexpr uint32_t kNextP = KEYS ? 0 : 128;

    bool ok_softmax = true;
    if (n_all == 0) {
        // rows outside the pack or not in use: zeros, without any of the rest
        const int n_rows = live && rank == 0 ? min(kTile, len - first) : 0;
        for (int i = threadIdx.x; i < n_rows * (DP / 8); i += kThreads) {
            const int64_t tok = where.start + first + i / (DP / 8);
            const int col = 8 * (i % (DP / 8));
            if (col >= a.d) continue;
            *reinterpret_cast<uint4 *>(a.out1 + tok * a.o1_ts + xhead * a.o1_hs + col) = make_uint4(0, 0, 0, 0);
            if (KEYS) *reinterpret_cast<uint4 *>(a.out2 + tok * a.o2_ts + xhead * a.o2_hs + col) = make_uint4(0, 0, 0, 0);
        }
    } else if (warp >= kLoadWarp) {
        // ------------------------------------------------------------ loads
        const int which = warp - kLoadWarp;
        if (which == 0 && lane == 0 && n_tiles > 0) {
            mbar_expect_tx(x_full, 2 * Sh::kTileBytes);
            for (int b = 0; b < Sh::kBoxes; ++b) {
                tma_load_3d(base + b * kBox, &a.x1, 64 * b, where.start + first, xhead, x_full);
                tma_load_3d(base + Sh::kTileBytes + b * kBox, &a.x2, 64 * b, where.start + first, xhead, x_full);
            }
        }
        const CUtensorMap *map = which == 0 ? &a.y1 : &a.y2;
        const int places = which == 0 ? Sh::kY1 : Sh::kY2, place0 = which == 0 ? 0 : Sh::kY1;
        int g = head0, y = y0_first, at = 0, before = 0, issued = 0;
        for (int t = 0; t < n_tiles; ++t) {
            const uint32_t bar = y_full + 8 * (place0 + at);
            const int yhead = KEYS ? xhead * a.group + g : xhead / a.group;
            float2 v[4];
            if (KEYS && which == 0) {
                const float2 *src = a.stats + static_cast<int64_t>(yhead) * a.n_tokens + where.start;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = y * kTile + lane + 32 * i;
                    v[i] = r < rows ? src[r] : make_float2(-INFINITY, 0.0f);
                }
            }
            if (before > 0 && !warp_wait(y_empty + 8 * (place0 + at), (before - 1) & 1, &s_abort, &g_attn_bwd_fault)) break;
            if (lane == 0) {
                const uint32_t dst = base + Sh::kOffY + (place0 + at) * Sh::kTileBytes;
                mbar_expect_tx(bar, Sh::kTileBytes);
                for (int b = 0; b < Sh::kBoxes; ++b)
                    tma_load_3d(dst + b * kBox, map, 64 * b, where.start + y * kTile, yhead, bar);
            }
            ++issued;
            if (KEYS && which == 0) {   // the statistics of Y1's rows
                if (t >= 2 && !warp_wait(st_empty + 8 * (t & 1), ((t >> 1) - 1) & 1, &s_abort, &g_attn_bwd_fault)) break;
                float *dst = reinterpret_cast<float *>(smem + Sh::kOffStats + (t & 1) * 2 * kTile * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    dst[lane + 32 * i] = v[i].x;
                    dst[kTile + lane + 32 * i] = v[i].y;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(st_full + 8 * (t & 1));
            }
            if (++y == y_hi) {
                y = y_lo;
                ++g;
            }
            if (++at == places) {
                at = 0;
                ++before;
            }
        }
        if (n_tiles > 0) {
            if (s_abort != 0) {         // copies in flight land before the memory is given back
                for (int t = max(0, issued - places); t < issued; ++t)
                    mbar_drain(y_full + 8 * place(t, which), turn(t, which) & 1);
                if (which == 0) mbar_drain(x_full, 0);
            }
        }
        __syncwarp();
    } else if (warp == kWatchWarp) {
        // ------ the arrival of Y: the products wait for it and for P at one barrier, as every
        // wait costs a few hundred cycles while the tensor core reads shared memory
        bool ok = n_tiles > 0 && warp_wait(x_full, 0, &s_abort, &g_attn_bwd_fault);
        int y = y0_first;
        for (int t = 0; ok && t <= n_tiles; ++t) {
            if (t < n_tiles) {
                ok = warp_wait(y_full + 8 * place(t, 0), turn(t, 0) & 1, &s_abort, &g_attn_bwd_fault) &&
                     warp_wait(y_full + 8 * place(t, 1), turn(t, 1) & 1, &s_abort, &g_attn_bwd_fault);
                if (!ok) break;
                // streamed rows past the sample's end (another sample's, or anything) are
                // cleared: their weights are zero, but zero times NaN is not
                const int valid = rows - y * kTile;
                if (++y == y_hi) y = y_lo;
                if (valid < kTile) {
                    for (int which = 0; which < 2; ++which) {
                        uint8_t *tile = smem + Sh::kOffY + place(t, which) * Sh::kTileBytes;
                        for (int r = valid + (lane >> 3); r < kTile; r += 4)
                            for (int i = 0; i < Sh::kBoxes; ++i)
                                *reinterpret_cast<uint4 *>(tile + i * kBox + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    __syncwarp();
                }
            }
            // tile t counts towards phase t - 1 of the barrier, once the phase before is over
            if (t >= 2) ok = warp_wait(p_full, (t - 2) & 1, &s_abort, &g_attn_bwd_fault);
            if (ok && lane == 0) mbar_arrive(t == 0 ? first_full : p_full);
            __syncwarp();
        }
    } else if (warp == kMmaWarp) {
        // --------------------------------------------------------- products
        constexpr uint32_t kDescS = mma_desc(kTile, kTile, false), kDescA = mma_desc(kTile, DP, true);
        const uint32_t ubase = uniform(base), utmem = uniform(tmem);
        const uint32_t d_x = desc_lo(ubase, 0), d_y = desc_lo(ubase + Sh::kOffY, 0),
                       d_ymn = desc_lo(ubase + Sh::kOffY, kBox);
        constexpr uint32_t kStep = Sh::kTileBytes >> 4;
        bool ok = true;
        auto wait = [&](uint32_t bar, int phase) {
            if (ok) ok = warp_wait(bar, phase & 1, &s_abort, &g_attn_bwd_fault);
            tc_fence_after();
        };
        // S(t) (which = 0) or dP(t) (1); one elected thread
        auto scores = [&](int t, int which) {
            const uint32_t d = utmem + (which == 0 ? kColS : kColP + (t & 1) * kNextP);
            const uint32_t y = d_y + place(t, which) * kStep;
#pragma unroll
            for (int s = 0; s < DP / 16; ++s) {
                const uint32_t off = ((s / 4) * kBox + (s % 4) * 32) >> 4;
                mma_ss(d, d_x + which * kStep + off, y + off, kDescS, s > 0);
            }
            // (queries: dP of the next tile may be complete before every warp has seen this one)
            tc_commit(which == 0 ? s_full : dp_full + 8 * (t & 1));
            if (!KEYS && which == 1) tc_commit(y_empty + 8 * place(t, which));
        };
        // acc1 += dS Y1 (which = 0) or acc2 += P Y2 (1); one elected thread
        auto accumulate = [&](int t, int which) {
            const uint32_t d = utmem + (which == 0 ? kCol1 : kCol2);
            const uint32_t from = utmem + (which == 0 ? kColP + (t & 1) * kNextP : kColS);
            const uint32_t y = d_ymn + place(t, which) * kStep;
#pragma unroll
            for (int s = 0; s < kTile / 16; ++s)
                mma_ts(d, from + 32 * (s / 2) + 8 * (s % 2), y + s * (2048 >> 4), kDescA, t > 0 || s > 0);
            tc_commit(y_empty + 8 * place(t, which));
            if (KEYS && which == 0) tc_commit(st_empty + 8 * (t & 1));
            if (which == 0 && t + 1 == n_tiles) tc_commit(done);
        };
        if (n_tiles > 0) {
            wait(first_full, 0);
            if (ok && elect_one()) {
                scores(0, 0);
                scores(0, 1);
            }
            __syncwarp();
        }
        for (int t = 0; ok && t < n_tiles; ++t) {
            const bool more = t + 1 < n_tiles;
            if (KEYS || more) wait(p_full, t);
            if (ok && elect_one()) {
                if (KEYS) accumulate(t, 1);
                if (more) scores(t + 1, 0);
                if (!KEYS && more) scores(t + 1, 1);
            }
            __syncwarp();
            wait(ds_full, t);
            if (ok && elect_one()) {
                accumulate(t, 0);
                if (KEYS && more) scores(t + 1, 1);
            }
            __syncwarp();
        }
        if (!ok) {                      // products in flight finish before tensor memory is freed
            if (lane == 0) tc_commit(drain);
            mbar_drain(drain, 0);
        }
        __syncwarp();
    }
    if (n_tiles > 0 && warp < kMmaWarp) {
        // ---------------------------------------------------------- softmax
        // a row of X is four threads', 32 of a tile's columns each
        const int quarter = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + kColS + 32 * quarter, t_p = tmem + lanes + kColP + 32 * quarter;
        const int xi = first + row;                                    // key or query of the sample
        const float c = a.scale * kLog2e;
        float2 mine = make_float2(-INFINITY, 0.0f);
        if (!KEYS && live && xi < rows)
            mine = a.stats[static_cast<int64_t>(xhead) * a.n_tokens + where.start + xi];
        const float2 c2 = make_float2(c, c);
        // The D that comes in is dout . o with o rounded to bf16.  Against the few keys of a
        // sample's first rows that error is as large as the rounding of ds; where all keys of
        // the rows are in one tile, D is taken from them instead, D = sum_j p dP, and kept for
        // the pass over the keys (with n keys the error shrinks as 1 / sqrt(n)).
        const bool single = !KEYS && n_tiles == 1;
        bool &ok = ok_softmax;
        int y = y0_first;
        for (int t = 0; t < n_tiles; ++t) {
            const int y0 = y * kTile + 32 * quarter;                   // this thread's first column
            if (++y == y_hi) y = y_lo;
            const uint32_t st = base + Sh::kOffStats + (t & 1) * 2 * kTile * 4 + 128 * quarter;
            // of its columns, [from, to) are visible: keys of a query row, or queries of a key row
            int from = 0, to = 32;
            bool masked;
            if (KEYS) {
                masked = a.causal && y0 < first + kTile;
                if (a.causal) from = xi - y0;
            } else {
                masked = y0 + 32 > (a.causal ? min(rows, first + 1) : rows);
                to = min(rows, a.causal ? xi + 1 : rows) - y0;
            }
            ok = warp_wait(s_full, t & 1, &s_abort, &g_attn_bwd_fault);
            if (KEYS && ok) ok = warp_wait(st_full + 8 * (t & 1), (t >> 1) & 1, &s_abort, &g_attn_bwd_fault);
            if (!ok && !single) break;         // (a single tile's warps meet below in any case)
            tc_fence_after();
            uint32_t s[32], packed[16];
            tmem_ld32(t_s, s);
            tc_wait_ld(s);
            if (!KEYS) {                                               // S is free
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 nl = KEYS ? smem_load4(st + 4 * j) : make_float4(mine.x, mine.x, mine.x, mine.x);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = j + 2 * h;
                    float2 p = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2,
                                    h == 0 ? make_float2(nl.x, nl.y) : make_float2(nl.z, nl.w));
                    p.x = ex2(p.x);
                    p.y = ex2(p.y);
                    if (masked) {
                        if (e < from || e >= to) p.x = 0.0f;
                        if (e + 1 < from || e + 1 >= to) p.y = 0.0f;
                    }
                    s[e] = __float_as_uint(p.x);
                    s[e + 1] = __float_as_uint(p.y);
                    packed[e / 2] = pack_bf16(p.x, p.y);
                }
            }
            // P and dS take the first half of the columns this thread has read
            if (KEYS) {
                tmem_st16(t_s, packed);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            if (ok) ok = warp_wait(dp_full + 8 * (t & 1), (t >> 1) & 1, &s_abort, &g_attn_bwd_fault);
            if (!ok && !single) break;
            tc_fence_after();
            const uint32_t t_dp = t_p + (t & 1) * kNextP;
            uint32_t dp[32];
            tmem_ld32(t_dp, dp);
            tc_wait_ld(dp);
            if (single) {
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < 32; ++e) sum[e & 1] = fmaf(__uint_as_float(s[e]), __uint_as_float(dp[e]), sum[e & 1]);
                float *swap = reinterpret_cast<float *>(smem + Sh::kOffStats);   // [quarter][row]
                swap[quarter * kTile + row] = sum[0] + sum[1];
                named_barrier(1 + (warp & 3), 128);
                mine.y = -((swap[row] + swap[kTile + row]) + (swap[2 * kTile + row] + swap[3 * kTile + row]));
                if (quarter == 0 && live && xi < rows)
                    a.stats[static_cast<int64_t>(xhead) * a.n_tokens + where.start + xi].y = mine.y;
            }
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 nd = KEYS ? smem_load4(st + 4 * (kTile + j)) : make_float4(mine.y, mine.y, mine.y, mine.y);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = j + 2 * h;
                    const float2 ds = mul2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])),
                                           add2(make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])),
                                                h == 0 ? make_float2(nd.x, nd.y) : make_float2(nd.z, nd.w)));
                    packed[e / 2] = pack_bf16(ds.x, ds.y);
                }
            }
            tmem_st16(t_dp, packed);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
        }
        if (ok && n_tiles > 0) {
            ok = warp_wait(done, 0, &s_abort, &g_attn_bwd_fault);
            tc_fence_after();
        }
    }
    // A cluster's partial dk and dv: the 32-row slices of quarter q go to CTA q * ranks / 4,
    // which adds them in the order of the CTAs.  Y's place takes them, [from][slice][column / 4][row][4].
    const int quarter = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const bool second = KEYS && quarter >= 2;
    constexpr int kCols = KEYS ? DP / 2 : DP / 4;
    const int col0 = (KEYS ? quarter & 1 : quarter) * kCols;
    const uint32_t acc = tmem + lanes + (second ? kCol2 : kCol1) + col0;
    const int owner = KEYS ? quarter * ranks / 4 : 0, slices = 4 / ranks;
    auto part = [&](int from) {
        return base + Sh::kOffY + static_cast<uint32_t>(((from * slices + quarter % slices) * (kCols / 4)) * kTile + row) * 16;
    };
    if (KEYS && ranks > 1 && n_all > 0) {
        cluster_arrive();
        cluster_wait();                 // every CTA is through with its tiles
        if (warp < kMmaWarp && owner != rank) {
            const uint32_t to = part(rank);
#pragma unroll 1
            for (int j = 0; j < kCols / 16; ++j) {
                uint32_t o[16];
                if (n_tiles > 0) {
                    tmem_ld16(acc + 16 * j, o);
                    tc_wait_ld16(o);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (n_tiles > 0)
                        x = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                        __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    cluster_store4(to + (4 * j + e) * kTile * 16, owner, x);
                }
            }
            __syncwarp();
        }
        cluster_arrive();
        cluster_wait();
    }
    if (n_all > 0 && warp < kMmaWarp && owner == rank) {
        // epilogue: dk and dv by two groups each, or a quarter of dq's columns a group
        const int xi = first + row;
        const bool in_use = xi < rows;
        const float mult = second ? 1.0f : a.scale;
        uint32_t v[kCols / 2];
#pragma unroll
        for (int j = 0; j < kCols / 16; ++j) {
            uint32_t o[16];
            __syncwarp();
            if (n_tiles > 0) {
                tmem_ld16(acc + 16 * j, o);
                tc_wait_ld16(o);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = 0u;
            }
            if (KEYS && ranks > 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 own = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int r = 0; r < ranks; ++r) {
                        const float4 x = r == rank ? own : smem_load4(part(r) + (4 * j + e) * kTile * 16);
                        sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
                    }
                    o[4 * e] = __float_as_uint(sum.x);
                    o[4 * e + 1] = __float_as_uint(sum.y);
                    o[4 * e + 2] = __float_as_uint(sum.z);
                    o[4 * e + 3] = __float_as_uint(sum.w);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[8 * j + e] = in_use ? pack_bf16(__uint_as_float(o[2 * e]) * mult, __uint_as_float(o[2 * e + 1]) * mult) : 0u;
        }
        // X is no longer read: its tiles become the warps' scratch
        __nv_bfloat16 *out = second ? a.out2 : a.out1;
        const int64_t ts = second ? a.o2_ts : a.o1_ts, hs = second ? a.o2_hs : a.o1_hs;
        const int row0 = first + 32 * (warp & 3);
        if (ok_softmax && live)
            warp_store_rows<kCols>(base + warp * (64 * kCols), v, a.d - col0, [&](int r) {
                if (row0 + r >= len) return static_cast<__nv_bfloat16 *>(nullptr);
                return out + (where.start + row0 + r) * ts + xhead * hs + col0;
            });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// (-lse log2(e), -D) of every (head, token) row, D = dout . out.  Eight lanes a row, 16
// elements each (head_dim <= 128); HBM-bound.  The grid is resident while the kernel that
// writes out and lse ends, so they are no read-only data: no __ldg and no __restrict__, here
// and where the passes read the statistics.
__global__ void __launch_bounds__(256) attn_stats_kernel(const __nv_bfloat16 *dout, int64_t g_ts, int64_t g_hs,
                                                         const __nv_bfloat16 *out, int64_t o_ts, int64_t o_hs,
                                                         const float *lse, float2 *stats, int n_tokens, int hq, int d)
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
        const uint4 g = *reinterpret_cast<const uint4 *>(dout + tok * g_ts + head * g_hs + col);
        const uint4 o = *reinterpret_cast<const uint4 *>(out + tok * o_ts + head * o_hs + col);
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

// CTAs that share a tile of keys, up to 4.  While all fit the SMs at once, sharing pays from a
// few streamed tiles each on.  Causal tiles of keys are uneven, so that sharing long ones pays
// up to two and a half rounds as well; even ones would only wait for a second round.  CTAs are
// counted by the tiles that samples of any lengths fill on average (slots may stay empty).
// The whole backward by one, two and four a tile, heads of 128 unless stated, causal:
//   one round   500 tokens, 32/8 heads 40.5, 35.5, 33.9 us; 2,000, 8/2 heads 123, 83, 66;
//               8 x 128, 32/8 heads 32, 38, 58 (four tiles each: not shared)
//   more        2,048, 32/8 heads 159, 130, 170; 4,000, 8/2 heads of 64 201, 123, 92;
//               4 x 512, 64/8 heads 127, 134, 164; 4,096, 32/8 heads 379, 393, 482 (not shared)
//   both directions: 3,522 tokens, 10/2 heads of 80 185, 131, 132; 3 x 900, 12/4 heads of 80
//               77, 93, 108 (not shared)
int key_cluster(const AttnProblem &p)
{
    const int64_t n = p.n_seqs > 0 ? p.n_seqs : 1;
    const int64_t ctas = (p.n_tokens + n * (kTile / 2) + kTile - 1) / kTile * p.hkv;
    const int64_t tiles = p.group * ((p.n_tokens / n + kTile - 1) / kTile);
    const auto pays = [&](int ranks) {
        if (ctas * ranks <= kSMs) return tiles >= 4 * ranks;
        return p.causal && 2 * ctas * ranks <= 5 * kSMs && tiles > 16 * ranks;
    };
    int ranks = 1;
    while (ranks < 4 && pays(2 * ranks)) ranks *= 2;
    return ranks;
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
    auto map = [&](CUtensorMap *m, const Rows &r, int heads) {
        const int64_t ext[3] = {p.d, p.n_tokens, heads}, st[3] = {1, r.ts, r.hs};
        const int box[3] = {64, kTile, 1};
        return make_map(m, r.p, 3, ext, st, box);
    };
    if (!map(&a.x1, x1, xh) || !map(&a.x2, x2, xh) || !map(&a.y1, y1, yh) || !map(&a.y2, y2, yh))
        return cudaErrorInvalidValue;
    const Rows &o1 = KEYS ? p.dk : p.dq;
    a.out1 = o1.p;
    a.o1_ts = o1.ts;
    a.o1_hs = o1.hs;
    a.out2 = p.dv.p;
    a.o2_ts = p.dv.ts;
    a.o2_hs = p.dv.hs;
    a.stats = reinterpret_cast<float2 *>(p.stats);
    a.cu = p.cu;
    a.used = p.used;
    a.n_tokens = p.n_tokens;
    a.n_seqs = p.n_seqs;
    a.hq = p.hq;
    a.hkv = p.hkv;
    a.group = p.group;
    a.d = p.d;
    a.causal = p.causal;
    a.n_slots = slot_count(p.n_tokens, p.n_seqs, kTile);
    a.scale = p.scale;
    a.div_tile = make_fastdiv(kTile);
    const int ranks = KEYS ? key_cluster(p) : 1;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    plain_config(cfg, attr[0], static_cast<unsigned>(a.n_slots) * static_cast<unsigned>(xh * ranks), kThreads,
                 Shared<DP>::kBytes, stream);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
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
    // dq first: it improves the statistics that the pass over the keys reads
    err = p.d <= 64 ? launch_pass<64, false>(p, stream) : launch_pass<128, false>(p, stream);
    if (err != cudaSuccess) return err;
    return p.d <= 64 ? launch_pass<64, true>(p, stream) : launch_pass<128, true>(p, stream);
}

int attn_bwd_fault_word(int *word)
{
    return read_fault_word(word, g_attn_bwd_fault);
}

}  // namespace pvr
