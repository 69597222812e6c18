// Attention forward on the tensor cores (GB300, sm_103a): packed samples or a paged cache.
//
// Mathematics.  For each row the running maximum m and sum l of a softmax over key tiles:
//   s = scale q.k;  m' = max(m, max s);  p = exp(s - m');  l' = l exp(m - m') + sum p;
//   o' = o exp(m - m') + p V.  Exponentials are base 2 with scale*log2(e) folded in.
// m is the maximum of the first tile and stays until a later one exceeds it by more than
// 2^30: floating-point weights keep their precision whatever the scale, and sums of 2^24
// weights below 2^30 stay far inside binary32.  So a tile's weights are computed without
// waiting for its maximum, and o is hardly ever rescaled.
//
// Layout.  A CTA owns 256 rows of one key head: two tiles of 128 rows, a row being one
// (token, query head) pair with the G heads that share the key head side by side, so every
// key tile is loaded once for all of them.  Key and value tiles are 128 tokens, brought in by
// TMA through a ring of shared-memory stages.
//   S_x = Q_x K^T      128x128 in tensor memory, both operands from shared memory
//   O_x += P_x V       P as bf16 over S's columns in tensor memory, V from shared memory
// Four warpgroups run the softmax, two to a row tile, a row being two threads' (64 of a tile's
// keys each); one warp issues the products, one the loads, one watches the loads.  While one
// row tile's softmax runs the tensor core works for the other.
//
// Rules on the scores (score_rule.cuh), an instance each.  A prefix only moves the rows' limits.
// Shaped scores (capped, biased) become exponents 32 columns at a time between tensor memory and the
// exponential; with a bias by distance the key tiles go downwards, so that causal rows meet their
// largest exponents first.  They hold the softmax warps, not the tensor core, back: a packed batch of
// 16,384 tokens, 345 us by its operations (another draw of the lengths below, with longer samples), 32/8
// heads of 128, 501-509 us plain, 515 with prefixes of some samples, 557-578 with slopes, 637 capped, 795-800
// both (four warps a scheduler of dependent operations, half of the issue slots taken); 32/32 heads of 64,
// 172 us by its operations, 461, 515, 546, 624 and 837 us.
//
// What it took.  Operands of the tensor core's instructions in uniform registers, issued by an
// elected lane of a converged warp (from one diverged lane each cost 100 cycles).  Hardly a
// register spill (packed: none without slopes, 4-16 bytes stored with them; paged: none with a cap, 4 bytes
// plain, with prefixes or slopes, 8-24 with cap and slopes): with 200 KB
// of shared memory local memory misses to L2, and the softmax loop waits for it.  One wait per
// row tile for the issuing warp: a wait costs some 200 cycles while the tensor core
// reads shared memory, so the arrival of K and V is folded into the barrier of P.
//
// The bound is the tensor core: 1024 cycles a row tile and key tile.  32/8 heads of 128,
// causal: one sample of 32,768 tokens 5.34-5.48 ms, 1,605-1,647 TFLOP/s, over 0.1 s and 5.70
// ms, 1,544, over 0.9 s under the power limit (the library's products sustain 1,705; from pages
// of 128 tokens 5.74 ms); 8,192 tokens 379 and 392 us; packs of short samples are held back by
// the 6,000 cycles before a CTA's first softmax and the 4,000 after its last (16,384 tokens in
// samples of 32-8,192, 309 us by its operations: 474 us, 1,237 TFLOP/s).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "attn_internal.h"
#include "score_rule.cuh"
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace pvr {
namespace {

__device__ int g_attn_fault;            // bounded waits that ran out

constexpr int kThreads = 640;           // four softmax warpgroups, one for products and loads
constexpr int kMmaWarp = 16, kLoadWarp = 17, kWatchWarp = 18;
constexpr int kRows = 128;              // rows of a row tile
constexpr int kKeys = 128;              // keys of a key tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 30.0f;          // log2 growth of the maximum that triggers a rescale
constexpr float kFoldLimit = 4096.0f;   // |m| (log2) up to which it is folded into an FMA: its rounding is 2^-13 at most

struct FwdArgs {
    CUtensorMap q, k, v;
    __nv_bfloat16 *out;
    int64_t out_ts, out_hs;
    float *lse;                         // [hq, T] or NULL
    float *part_o, *part_lse;           // [split][T * hq][d], [split][T * hq], or NULL
    const int32_t *cu, *used;
    const int32_t *table;
    int64_t table_stride;
    int32_t max_pages, page_size, n_pages, box_rows;
    int32_t n_tokens, n_seqs, hq, hkv, group, tile_tokens, d, causal;   // tile_tokens: of one row tile
    int32_t n_slots, splits;
    FastDiv div_cta, div_group;         // by the CTA's tokens, by group
    float scale;
    ScoreRule rule;
};

template <int DP>
struct Shared {
    static constexpr int kBoxes = DP / 64;
    static constexpr int kTileBytes = kKeys * DP * 2;
    static constexpr int kStages = DP == 128 ? 4 : 6;
    static constexpr int kOffKV = 2 * kTileBytes;                     // after the two Q tiles
    static constexpr int kOffBars = kOffKV + kStages * kTileBytes;
    static constexpr int kBytes = kOffBars + 256 + 1024;              // + alignment slack
};

// Capped exponents that stay within +-80 need no maximum, a quarter of K does for all rows: weights
// are within 2^60 and 2^-100, so that they and the sums of 2^24 of them keep their precision in
// binary32; the two halves of a row need not meet.
// Where a maximum makes the largest weight 1, here it is rounded to bf16 too: the output is divided by
// the sum of the rounded weights, so that a row of one key is that key's value (o off by 1.8-2.2e-3 of
// itself, 2.3-2.4e-3 without, for 40 us of 637; lse takes the sum of the weights as they are).
// Their products with values far from 1 may leave binary32 all the same.  A row whose sum is above
// kMostSum or below kLeastSum looks at its output, and where that has overflowed, or holds values so
// small that they may have lost bits, the CTA runs once more, with that row's own lse as its maximum.
// Other rows keep theirs, and their bits (626 -> 637 us, one CTA's work once more where it happens).
// Larger caps are the biased instance's, with slopes of 0 (the packed batch, 32/8 heads of 128: 637 us,
// 797 with the maximum; both in one instance cost the first a quarter).
constexpr bool kFixed = kRule == kRuleCap;
constexpr float kMostSum = 1073741824.0f, kLeastSum = 5.9604645e-8f;   // 2^30, 2^-24
constexpr float kTiny = 7.8886091e-31f; // 2^-100: binary32 holds what is left of such an output to 2^-26

template <int DP, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) attn_fwd_kernel(const __grid_constant__ FwdArgs a)
{
    using Sh = Shared<DP>;
    constexpr int kStages = Sh::kStages;
    constexpr uint32_t kBoxBytes = kKeys * 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_addr(smem);
    const uint32_t bars = base + Sh::kOffBars;
    const uint32_t q_full = bars, s_full = bars + 16, p_full = bars + 32, o_done = bars + 48, kv_full = bars + 64,
                   kv_empty = kv_full + 8 * kStages, first_full = kv_empty + 8 * kStages, drain = first_full + 8;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ float s_start[kFixed ? 2 : 1][kRows];                   // [row tile][row], the fixed maximum
    __shared__ volatile int s_again, s_loads;                          // the CTA is to run once more; tiles that it loaded
    __shared__ TileSlot s_slot;
    __shared__ float s_swap[2][2][2][kRows];                           // [parity][row tile][half][row]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto init_barriers = [&] {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 9);
            mbar_init(o_done + 8 * i, 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(kv_full + 8 * i, 1);
            mbar_init(kv_empty + 8 * i, 1);
        }
        mbar_init(first_full, 1);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    };
    if (threadIdx.x == 0) {
        s_abort = 0;
        if (kFixed) s_again = 0;
        init_barriers();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&s_tmem), 512);
    if (warp == kLoadWarp && lane == 0) {
        tma_prefetch_map(&a.q);
        tma_prefetch_map(&a.k);
        tma_prefetch_map(&a.v);
    }
    if (kFixed && threadIdx.x < 2 * kRows) s_start[threadIdx.x / kRows][threadIdx.x % kRows] = 0.25f * a.rule.k;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int kvh = blockIdx.x % a.hkv;
    const int split = blockIdx.y;
    // causal rows near a sample's end have the most keys: late slots go first
    const int slot = a.n_slots - 1 - static_cast<int>(blockIdx.x) / a.hkv;
    const int cta_tokens = 2 * a.tile_tokens;
    if (warp == 0) {
        const TileSlot f = find_slot(a.cu, a.used, a.n_seqs, a.n_tokens, a.div_cta, slot);
        if (lane == 0) s_slot = f;
    }
    tc_fence_before();
    __syncthreads();
    // With a fixed maximum (kFixed) what follows may run once more: a copy of its own then, as a loop around
    // one leaves the softmax fewer registers (2.6 KB of spills in the paged form).  The other instances have
    // no function around it, which alone cost cap and slopes from pages 374 us for 336.
#if PVR_SCORE_RULE == 2
    auto attend = [&](auto repeats) {
    constexpr bool kRepeated = decltype(repeats)::value;
#else
    constexpr bool kRepeated = false;
#endif
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const TileSlot where = s_slot;
    const int first = where.tile * cta_tokens;                         // token of the sample the CTA starts at
    const int len = where.end - where.start;
    const bool live = where.tile >= 0 && first < len;
    // rows in use, keys, and how far past a row's index its keys go
    int rows_used, keys, offset;
    if (PAGED) {
        const bool inside = where.sample >= 0 && where.sample < a.n_seqs;
        const int kv = max(where.used, -1);
        rows_used = inside ? len : 0;
        keys = inside ? static_cast<int>(min(static_cast<int64_t>(max(kv, 0)),
                                             static_cast<int64_t>(a.max_pages) * a.page_size)) : 0;
        offset = kv - len;
    } else {
        rows_used = min(len, max(where.used, 0));
        keys = rows_used;
        offset = 0;
    }
    const int prefix = prefix_of(a.rule, where.sample, a.n_seqs, keys);
    // keys that row `i` of the sample sees: the first so many
    auto limit = [&](int i) {
        if (i >= rows_used || i + offset < 0) return 0;
        const int own = a.causal ? min(keys, i + offset + 1) : keys;
        return kRuled ? max(own, prefix) : own;
    };
    int count[2], lo_tile = 0, n_tiles = 0;
    {
        int n[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int last = min(first + (x + 1) * a.tile_tokens, rows_used) - 1;
            n[x] = live && last >= first + x * a.tile_tokens ? (limit(last) + kKeys - 1) / kKeys : 0;
        }
        const int all = max(n[0], n[1]);
        const int chunk = a.splits == 1 ? all : (all + a.splits - 1) / a.splits;
        lo_tile = split * chunk;
        const int hi = min(all, lo_tile + chunk);
#pragma unroll
        for (int x = 0; x < 2; ++x) count[x] = max(0, min(n[x], hi) - lo_tile);
        n_tiles = max(count[0], count[1]);
        // biased scores: both row tiles start with the last key tile, the earlier one hiding it
        if (kBias)
            for (int x = 0; x < 2; ++x)
                if (count[x] > 0) count[x] = n_tiles;
    }
    // Key tiles go upwards; with a bias by distance downwards, so that causal rows meet their
    // largest exponents first and hardly ever rescale.
    auto tile_at = [&](int i) { return kBias ? n_tiles - 1 - i : i; };
    constexpr uint32_t kColS = 0, kColO = 256;

    if (n_tiles == 0) {
        // no row of the CTA sees a key (padding, or keys of other splits): zeros, without any
        // of the rest
        const bool joined = PAGED && a.splits > 1;
        const int n_rows = live ? min(cta_tokens, len - first) * a.group : 0;
        for (int i = threadIdx.x; i < n_rows * (DP / 8); i += kThreads) {
            const int r = i / (DP / 8), col = 8 * (i % (DP / 8));
            const int tok_in = static_cast<int>(fast_div(r, a.div_group));
            const int64_t tok = where.start + first + tok_in;
            const int head = kvh * a.group + r - tok_in * a.group;
            if (!joined && col < a.d)
                *reinterpret_cast<uint4 *>(a.out + tok * a.out_ts + head * a.out_hs + col) = make_uint4(0, 0, 0, 0);
            if (col == 0) {
                if (joined) a.part_lse[(static_cast<int64_t>(split) * a.n_tokens + tok) * a.hq + head] = -INFINITY;
                else if (a.lse != nullptr) a.lse[static_cast<int64_t>(head) * a.n_tokens + tok] = -INFINITY;
            }
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            for (int x = 0; x < 2; ++x) {
                if (count[x] == 0) continue;
                mbar_expect_tx(q_full + 8 * x, static_cast<uint32_t>(a.group * a.tile_tokens) * 128 * Sh::kBoxes);
                for (int b = 0; b < Sh::kBoxes; ++b)
                    tma_load_3d(base + x * Sh::kTileBytes + b * kBoxBytes, &a.q, 64 * b, kvh * a.group,
                                where.start + first + x * a.tile_tokens, q_full + 8 * x);
            }
        }
        const int per_tile = kKeys / a.box_rows;                       // boxes down a tile
        const int box = lane % (PAGED ? per_tile : 1), col = lane / (PAGED ? per_tile : 1);
        int issued = 0;
        for (int i = 0; i < n_tiles; ++i) {
            const int key0 = (lo_tile + tile_at(i)) * kKeys;
            int c_slot = where.start + key0, c_page = 0;
            if (PAGED) {
                // keys past the sequence's end read as zero: a page coordinate past the pool's
                const int key = key0 + box * a.box_rows;
                c_page = a.n_pages;
                c_slot = 0;
                if (key < keys) {
                    const int index = key / a.page_size;
                    c_page = __ldg(a.table + where.sample * a.table_stride + index);
                    c_slot = key - index * a.page_size;
                    if (c_page < 0 || c_page >= a.n_pages) c_page = a.n_pages;
                }
            }
            bool ok = true;
            for (int kv = 0; kv < 2; ++kv) {
                const int t = 2 * i + kv, stage = t % kStages;
                if (t >= kStages) ok = warp_wait(kv_empty + 8 * stage, (t / kStages - 1) & 1, &s_abort, &g_attn_fault);
                if (!ok) break;
                const uint32_t bar = kv_full + 8 * stage;
                const uint32_t dst = base + Sh::kOffKV + stage * Sh::kTileBytes + col * kBoxBytes +
                                     static_cast<uint32_t>(box * a.box_rows) * 128;
                if (lane == 0) mbar_expect_tx(bar, Sh::kTileBytes);
                __syncwarp();
                if (col < Sh::kBoxes) tma_load_4d(dst, kv == 0 ? &a.k : &a.v, 64 * col, c_slot, kvh, c_page, bar);
                ++issued;
            }
            if (!ok) break;
        }
        if (s_abort != 0) {             // copies in flight land before the memory is given back
            for (int t = max(0, issued - kStages); t < issued; ++t)
                mbar_drain(kv_full + 8 * (t % kStages), (t / kStages) & 1);
            for (int x = 0; x < 2; ++x)
                if (count[x] > 0)
                    mbar_drain(q_full + 8 * x, 0);
        }
    } else if (warp == kWatchWarp) {
        // ------ the arrival of keys and values: the products wait for them and for P at one
        // barrier, as every wait costs a few hundred cycles while the tensor core reads
        // shared memory
        auto full = [&](int t) {
            return warp_wait(kv_full + 8 * (t % kStages), (t / kStages) & 1, &s_abort, &g_attn_fault);
        };
        bool ok = n_tiles > 0 && full(0);
        for (int x = 0; x < 2; ++x)
            if (ok && count[x] > 0) ok = warp_wait(q_full + 8 * x, 0, &s_abort, &g_attn_fault);
        if (ok && lane == 0) mbar_arrive(first_full);
        __syncwarp();
        for (int i = 0; ok && i < n_tiles; ++i) {
            const int t = 2 * i + 1;
            ok = full(t);
            // value rows past the last key (another sample's, or stale) are cleared: their
            // weights are zero, but zero times NaN is not
            const int valid = keys - (lo_tile + tile_at(i)) * kKeys;
            if (ok && valid < kKeys) {
                uint8_t *v = smem + Sh::kOffKV + (t % kStages) * Sh::kTileBytes;
                for (int r = valid + (lane >> 3); r < kKeys; r += 4)
                    for (int b = 0; b < Sh::kBoxes; ++b)
                        *reinterpret_cast<uint4 *>(v + b * kBoxBytes + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
            }
            if (ok && i + 1 < n_tiles) ok = full(t + 1);
            for (int x = 0; x < 2; ++x) {
                if (i >= count[x]) continue;
                // counts towards phase i, once the phase before is over
                if (ok && i > 0) ok = warp_wait(p_full + 8 * x, (i - 1) & 1, &s_abort, &g_attn_fault);
                if (ok && lane == 0) mbar_arrive(p_full + 8 * x);
                __syncwarp();
            }
        }
    } else if (warp == kMmaWarp) {
        // --------------------------------------------------------- products
        constexpr uint32_t kDescS = mma_desc(kRows, kKeys, false);
        constexpr uint32_t kDescO = mma_desc(kRows, DP, true);
        const uint32_t ubase = uniform(base), utmem = uniform(tmem);
        const uint32_t d_q = desc_lo(ubase, 0), d_k = desc_lo(ubase + Sh::kOffKV, 0),
                       d_v = desc_lo(ubase + Sh::kOffKV, kBoxBytes);
        constexpr uint32_t kStep = Sh::kTileBytes >> 4;
        bool ok = true;
        auto wait = [&](uint32_t bar, int phase) {
            if (ok) ok = warp_wait(bar, phase & 1, &s_abort, &g_attn_fault);
            tc_fence_after();
        };
        // S of row tile x; one elected thread
        auto scores = [&](int x, int stage) {
#pragma unroll
            for (int s = 0; s < DP / 16; ++s) {
                const uint32_t at = ((s / 4) * kBoxBytes + (s % 4) * 32) >> 4;
                mma_ss(utmem + kColS + x * kKeys, d_q + x * kStep + at, d_k + stage * kStep + at, kDescS, s > 0);
            }
            tc_commit(s_full + 8 * x);
        };
        if (n_tiles > 0) {
            wait(first_full, 0);
            if (ok && elect_one()) {
                for (int x = 0; x < 2; ++x)
                    if (count[x] > 0) scores(x, 0);
                tc_commit(kv_empty);
            }
            __syncwarp();
        }
        for (int i = 0; ok && i < n_tiles; ++i) {
            const int sv = (2 * i + 1) % kStages, sk = (2 * i + 2) % kStages;
            for (int x = 0; x < 2; ++x) {
                if (i >= count[x]) continue;
                wait(p_full + 8 * x, i);
                if (ok && elect_one()) {
#pragma unroll
                    for (int s = 0; s < kKeys / 16; ++s)
                        mma_ts(utmem + kColO + x * DP, utmem + kColS + x * kKeys + s * 8 + (kShaped && s >= 4 ? 32 : 0), d_v + sv * kStep + s * (2048 >> 4),
                               kDescO, i > 0 || s > 0);
                    if (i + 1 == count[x]) tc_commit(o_done + 8 * x);
                    else scores(x, sk);
                    if (x == 1 || i >= count[1]) {           // the last to read these stages
                        tc_commit(kv_empty + 8 * sv);
                        if (i + 1 < n_tiles) tc_commit(kv_empty + 8 * sk);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok) {                      // products in flight finish before tensor memory is freed
            if (lane == 0) tc_commit(drain);
            mbar_drain(drain, 0);
        }
        __syncwarp();
    }
    if (n_tiles > 0 && warp < kMmaWarp) {
        // ---------------------------------------------------------- softmax
        // a row is two threads', 64 of a tile's keys each
        const int x = warp >> 3, half = (warp >> 2) & 1;
        const int row = (warp & 3) * 32 + lane;
        const int pair = 1 + x * 4 + (warp & 3);                       // the two warps' barrier
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + kColS + x * kKeys + half * 64;
        // P of a half over S of both; shaped scores: over the half's own S alone
        const uint32_t t_p = tmem + lanes + kColS + x * kKeys + half * (kShaped ? 64 : 32);
        const uint32_t t_o = tmem + lanes + kColO + x * DP + half * (DP / 2);
        const int tok0 = first + x * a.tile_tokens;                    // of the sample
        const int i_tok = tok0 + static_cast<int>(fast_div(row, a.div_group));
        const bool mine = live && row < a.group * a.tile_tokens && i_tok < len;
        const int lim = mine ? limit(i_tok) : 0;
        // from the CTA's first key on: keys that every row of the tile sees, and that this
        // thread's columns of the row see
        const int whole = limit(tok0) - lo_tile * kKeys, visible = lim - lo_tile * kKeys - 64 * half;
        const float c = kShaped ? 1.0f : a.scale * kLog2e;             // shaped scores are exponents of 2
        const float slope2 = !kBias || !mine || a.rule.slopes == nullptr ? 0.0f
            : a.rule.slopes[kvh * a.group + row - static_cast<int>(fast_div(row, a.div_group)) * a.group] * kLog2e;
        const int row_key = i_tok + offset - lo_tile * kKeys - 64 * half;   // this row's own key, from this thread's first
        float m = kFixed ? s_start[x][row] : -INFINITY, l = 0.0f, mc = 0.0f;
        bool ok = true;
        bool folded = false;                                           // m is known, and small (shaped: known)
        bool fold = true;                                              // shaped: m is small
        // 32 of this thread's scores of step i, those it does not see at -infinity
        auto load = [&](int i, int h, uint32_t(&s)[32]) {
            tmem_ld32(t_s + 32 * h, s);
            tc_wait_ld(s);
            if ((tile_at(i) + 1) * kKeys > whole) {
                const int left = visible - tile_at(i) * kKeys - 32 * h;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j >= left) s[j] = 0xff800000u;
            }
        };
        auto highest = [&](const uint32_t(&s)[32]) {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 32; j += 2)
                top[(j >> 1) & 3] = max3(top[(j >> 1) & 3], __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
            return max3(max3(top[0], top[1], top[2]), top[3], top[3]);
        };
        // p = 2^(s c - fixed), packed, and their sum
        auto weights = [&](const uint32_t(&s)[32], uint32_t *p, float fixed) {
            const float2 c2 = make_float2(c, c), fixed2 = make_float2(-fixed, -fixed);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float2 x = fma2(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, fixed2);
                x.x = ex2(x.x);
                x.y = ex2(x.y);
                sum[j & 1] = add2(sum[j & 1], x);
                p[j] = pack_bf16(x.x, x.y);
            }
            return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        };
        // Shaped scores: this thread's 64 of tile step i, 32 at a time, to weights 2^(x - shift): packed
        // into p, or with a fixed maximum to tensor memory as they come.  Returns their sum; high is the
        // largest x.  A large shift is not folded into the exponents' last operation: their rounding
        // would differ from that of the maximum, and the largest weight be far from 1.
        const bool line = a.causal && prefix <= 0;
        float2 rounded = make_float2(0.0f, 0.0f);                       // fixed maximum: sum of the weights as bf16
        auto shaped_pass = [&](auto folds, int i, float shift, uint32_t *p, float &high) {
            constexpr bool kFold = decltype(folds)::value;
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            high = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[32];
                tmem_ld32(t_s + 32 * h, w);
                tc_wait_ld(w);
                const int key0 = tile_at(i) * kKeys + 32 * h;
                float far = static_cast<float>(key0 - row_key);
                asm volatile("" : "+f"(far));    // or the distances of all passes are made at once, in spilled registers
                const int left = visible - key0;
                const bool masked = (tile_at(i) + 1) * kKeys > whole;
                if (kCap && masked) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j >= left) w[j] = 0u;
                }
                by_form(a.rule, w, lim == 0, line, [&](auto form) {
                    shape<decltype(form)::value>(a.rule, w, slope2, far, kFold ? shift : 0.0f);
                });
                if (masked) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j >= left) w[j] = 0xff800000u;
                }
                tmem_loaded(w);                  // (all at once: spread out, what follows would need more registers)
                uint32_t packed[16];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    float2 e = make_float2(__uint_as_float(w[j]), __uint_as_float(w[j + 1]));
                    if (!kFixed) high = max3(high, e.x, e.y);
                    if (!kFold) e = add2(e, twice(-shift));
                    e.x = ex2(e.x);
                    e.y = ex2(e.y);
                    sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], e);
                    (kFixed ? packed[j / 2] : p[16 * h + j / 2]) = pack_bf16(e.x, e.y);
                    if (kFixed)
                        rounded = add2(rounded, make_float2(__uint_as_float(packed[j / 2] << 16), __uint_as_float(packed[j / 2] & 0xffff0000u)));
                }
                if (kFixed) {
                    tmem_st16(t_p + 16 * h, packed);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)  // (a chunk is done before the next one is loaded)
                        asm volatile("" : "+r"(p[16 * h + j]), "+r"(p[16 * h + j + 1]), "+r"(p[16 * h + j + 2]), "+r"(p[16 * h + j + 3]));
                }
            }
            if (kFold) high += shift;
            return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        };
        // this thread's half of the output so far, and its sum, to a new maximum.  S of the tile is
        // complete, and with it every earlier product into O
        auto rescale = [&](int i, float shrink) {
            if (i == 0) return;
            l *= shrink;
#pragma unroll 1
            for (int j = 0; j < DP / 32; ++j) {
                uint32_t o[16];
                tmem_ld16(t_o + 16 * j, o);
                tc_wait_ld16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * shrink);
                tmem_st16(t_o + 16 * j, o);
            }
        };
        // after a wait that ran out the loop goes on without waiting, so that the pair's
        // barriers stay matched
        for (int i = 0; i < count[x]; ++i) {
            if (ok) ok = warp_wait(s_full + 8 * x, i & 1, &s_abort, &g_attn_fault);
            tc_fence_after();
            // with the maximum so far: s c is exact inside the FMA, and m c small enough for its
            // rounding not to matter
            uint32_t p[32];
            float high = -INFINITY, sum = 0.0f;
            if (kFixed) {
                sum = shaped_pass(std::true_type{}, i, m, p, high);
            } else if (kShaped) {
                for (bool settled = false;;) {                         // once more where the maximum has grown too far
                    sum = fold ? shaped_pass(std::true_type{}, i, mc, p, high) : shaped_pass(std::false_type{}, i, mc, p, high);
                    if (settled) break;
                    // (both warps of the pair hold the same rows: they go the same way)
                    if (lim == 0) high = -INFINITY;
                    s_swap[i & 1][x][half][row] = high;
                    named_barrier(pair, 64);
                    high = fmaxf(high, s_swap[i & 1][x][half ^ 1][row]);
                    if (!__any_sync(0xffffffffu, !folded || high - m > kGrow)) break;
                    const float grown = fmaxf(m, high), next = grown == -INFINITY ? 0.0f : grown;
                    const bool small = __all_sync(0xffffffffu, fabsf(next) <= kFoldLimit);
                    if (fold && !small) {                              // the maximum again, without a shift in it
                        fold = false;
                        named_barrier(pair, 64);
                        continue;
                    }
                    rescale(i, m == grown ? 1.0f : ex2(m - grown));
                    m = grown;
                    mc = next;
                    fold = small;
                    settled = folded = true;
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t s[32];
                    load(i, h, s);
                    high = fmaxf(high, highest(s));
                    if (folded) sum += weights(s, p + 16 * h, mc);
                }
                // rows that see no key may hold anything: they take no part in the warp's decisions
                if (lim == 0) high = -INFINITY;
                s_swap[i & 1][x][half][row] = high;
                // past the barrier both warps have read their scores, and P may overwrite them
                tc_fence_before();
                named_barrier(pair, 64);
                tc_fence_after();
                high = fmaxf(high, s_swap[i & 1][x][half ^ 1][row]);
                if (__any_sync(0xffffffffu, !folded || (high - m) * c > kGrow)) {
                    // a new maximum; both warps of the pair come here, as they hold the same rows
                    const float grown = fmaxf(m, high);
                    rescale(i, m == grown ? 1.0f : ex2((m - grown) * c));
                    m = grown;
                    const float shift = m == -INFINITY ? 0.0f : m;
                    mc = shift * c;
                    folded = __all_sync(0xffffffffu, fabsf(mc) <= kFoldLimit);
                    sum = 0.0f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t s[32];
                        load(i, h, s);
#pragma unroll
                        for (int j = 0; j < 32; ++j) s[j] = __float_as_uint(__uint_as_float(s[j]) - shift);
                        sum += weights(s, p + 16 * h, 0.0f);
                    }
                    tc_fence_before();
                    named_barrier(pair, 64);
                    tc_fence_after();
                }
            }
            if (!kFixed) tmem_st32(t_p, p);
            l += sum;
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 8 * x);
        }
        float norm = 0.0f;
        if (count[x] > 0) {
            if (ok) ok = warp_wait(o_done + 8 * x, 0, &s_abort, &g_attn_fault);
            tc_fence_after();
            s_swap[count[x] & 1][x][half][row] = l;
            if (kFixed) s_swap[count[x] & 1 ^ 1][x][half][row] = norm = rounded.x + rounded.y;
            named_barrier(pair, 64);
            l += s_swap[count[x] & 1][x][half ^ 1][row];
            if (kFixed) norm += s_swap[count[x] & 1 ^ 1][x][half ^ 1][row];
        }
        if (kFixed && !kRepeated) {
            const bool low = l < kLeastSum, far = lim > 0 && l > 0.0f && (low || l > kMostSum);
            if (__any_sync(0xffffffffu, far)) {
                bool off = false;
#pragma unroll 1
                for (int j = 0; j < DP / 32; ++j) {
                    uint32_t o[16];
                    tmem_ld16(t_o + 16 * j, o);
                    tc_wait_ld16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float size = fabsf(__uint_as_float(o[e]));
                        off = off || (half * (DP / 2) + 16 * j + e < a.d && (!(size < INFINITY) || (low && size < kTiny)));
                    }
                }
                if (far && off) {                                      // (either of the row's threads, or both alike)
                    s_start[x][row] = m + log2f(l);
                    s_loads = 2 * n_tiles;
                    s_again = 1;
                }
            }
        }
        // epilogue: rows outside the pack, and rows that see no key, are zero (tiles that all
        // rows in use see whole are not masked, so such rows may have summed anything).  No
        // weight is l == 0, not !(l > 0): a NaN score makes l NaN, and that must come out
        if (lim == 0) l = 0.0f;
        const int tok = where.start + i_tok;
        const int head = kvh * a.group + (row - static_cast<int>(fast_div(row, a.div_group)) * a.group);
        const float inv = l == 0.0f ? 0.0f : 1.0f / (kFixed ? norm : l);
        const bool joined = PAGED && a.splits > 1;
        const int64_t at = static_cast<int64_t>(tok) * a.hq + head;
        if (ok && mine && half == 0) {
            if (joined) {
                a.part_lse[static_cast<int64_t>(split) * a.n_tokens * a.hq + at] =
                    l == 0.0f ? -INFINITY : m * c + log2f(l);
            } else if (a.lse != nullptr) {
                a.lse[static_cast<int64_t>(head) * a.n_tokens + tok] = l == 0.0f ? -INFINITY : (kShaped ? m * kLn2 : m * a.scale) + kLn2 * log2f(l);
            }
        }
        const int col0 = half * (DP / 2);
        if (joined) {
#pragma unroll
            for (int j = 0; j < DP / 64; ++j) {
                const int col = col0 + 32 * j;
                uint32_t o[32];
                __syncwarp();
                if (count[x] > 0) {
                    tmem_ld32(t_o + 32 * j, o);
                    tc_wait_ld(o);
                }
                if (!ok || !mine || l == 0.0f) continue;
                float4 *dst = reinterpret_cast<float4 *>(a.part_o + (static_cast<int64_t>(split) * a.n_tokens * a.hq + at) *
                                                                        a.d + col);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col + 4 * e < a.d)
                        dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                             __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
            }
        } else {
            uint32_t w[DP / 4];
#pragma unroll
            for (int j = 0; j < DP / 64; ++j) {
                uint32_t o[32];
                __syncwarp();
                if (count[x] > 0) {
                    tmem_ld32(t_o + 32 * j, o);
                    tc_wait_ld(o);
                }
                if (count[x] == 0 || l == 0.0f) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    w[16 * j + e] = pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            }
            // Q is no longer read: its tile becomes the scratch of the eight warps
            const int row0 = 32 * (warp & 3);
            if (ok && live)
                warp_store_rows<DP / 2>(base + x * Sh::kTileBytes + (warp & 7) * (32 * DP), w, a.d - col0, [&](int r) {
                    const int tok_in = static_cast<int>(fast_div(row0 + r, a.div_group));
                    const int to = tok0 + tok_in;
                    if (row0 + r >= a.group * a.tile_tokens || to >= len) return static_cast<__nv_bfloat16 *>(nullptr);
                    return a.out + (where.start + to) * a.out_ts +
                           (kvh * a.group + row0 + r - tok_in * a.group) * a.out_hs + col0;
                });
        }
        tc_fence_before();
    }
#if PVR_SCORE_RULE == 2
    };
    attend(std::false_type{});
    __syncthreads();
    if (s_again != 0 && s_abort == 0) {
        // All copies have landed and all products are done, as the waits above have seen; what may still be
        // on its way are reports of places that are free.  Past them the barriers begin anew.
        fence_async_smem();             // the rows of the output were in Q's place
        if (warp == kMmaWarp)
            for (int t = max(0, s_loads - kStages); t < s_loads; ++t)
                warp_wait(kv_empty + 8 * (t % kStages), (t / kStages) & 1, &s_abort, &g_attn_fault);
        __syncthreads();
        if (s_abort == 0) {
            if (threadIdx.x == 0) {
                for (uint32_t bar = bars; bar <= drain; bar += 8) mbar_inval(bar);
                init_barriers();
            }
            tc_fence_before();
            __syncthreads();
            attend(std::true_type{});
            __syncthreads();
        }
    }
    const uint32_t tmem = s_tmem;
#else
    __syncthreads();
#endif
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

#if PVR_SCORE_RULE == 0
// Joins the partial results of the splits: o = sum_i w_i o_i, w_i = 2^(lse_i - lse).  One
// warp a row, 4 elements a lane.  A part whose lse is -infinity holds no weight and nothing
// was written for it; one of NaN (which the maximum passes over) makes the row NaN.  The grid
// is resident while the kernel that writes the parts ends: no __ldg and no __restrict__.
__global__ void __launch_bounds__(128) attn_join_kernel(const float *part_o, const float *part_lse,
                                                        __nv_bfloat16 *out, int64_t out_ts, int64_t out_hs,
                                                        int n_rows, int hq, int d, int splits)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= n_rows) return;
    float m = -INFINITY;
    for (int i = lane; i < splits; i += 32) m = fmaxf(m, part_lse[static_cast<int64_t>(i) * n_rows + row]);
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.0f;
    for (int i0 = 0; i0 < splits; i0 += 32) {
        const float mine = i0 + lane < splits ? part_lse[static_cast<int64_t>(i0 + lane) * n_rows + row] : -INFINITY;
        const int n = min(32, splits - i0);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float lse = __shfl_sync(0xffffffffu, mine, i);
            if (lse == -INFINITY) continue;
            const float w = exp2f(lse - m);
            l += w;
            if (4 * lane < d) {
                const float4 o = *reinterpret_cast<const float4 *>(
                    part_o + (static_cast<int64_t>(i0 + i) * n_rows + row) * d + 4 * lane);
                acc.x += w * o.x; acc.y += w * o.y; acc.z += w * o.z; acc.w += w * o.w;
            }
        }
    }
    if (4 * lane >= d) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int tok = row / hq, head = row % hq;
    *reinterpret_cast<uint2 *>(out + tok * out_ts + head * out_hs + 4 * lane) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

#endif

template <int DP, bool PAGED>
cudaError_t launch_fwd(const FwdArgs &a, cudaStream_t stream)
{
    static std::atomic<uint64_t> sized{0};
    const cudaError_t err = allow_smem(attn_fwd_kernel<DP, PAGED>, Shared<DP>::kBytes, sized);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n_slots) * static_cast<unsigned>(a.hkv), static_cast<unsigned>(a.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shared<DP>::kBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_fwd_kernel<DP, PAGED>, a);
}

}  // namespace

#if PVR_SCORE_RULE == 0
// Splits of the keys: enough CTAs to fill the GPU, at least two key tiles a split.
int attn_fwd_splits(const AttnProblem &p, int64_t max_kv)
{
    const int tile = kRows / p.group;
    const int64_t ctas = static_cast<int64_t>(slot_count(p.n_tokens, p.n_seqs, 2 * tile)) * p.hkv;
    const int64_t tiles = (max_kv + kKeys - 1) / kKeys;
    int64_t want = kSMs / ctas;
    if (want > tiles / 2) want = tiles / 2;
    return static_cast<int>(want < 1 ? 1 : want > 128 ? 128 : want);
}

cudaError_t launch_attn_fwd(const AttnProblem &p, int splits, float *workspace, cudaStream_t stream)
{
    int rule = p.rule();
    constexpr float kFixedLimit = 80.0f;                     // of K
    if (rule == kRuleCap && !(p.cap * kLog2e <= kFixedLimit)) rule |= kRuleBias;
    return for_rule(rule, [&](auto rule) { return launch_attn_fwd_rule<decltype(rule)::value>(p, splits, workspace, stream); });
}
#endif

template <>
cudaError_t launch_attn_fwd_rule<kRule>(const AttnProblem &p, int splits, float *workspace, cudaStream_t stream)
{
    FwdArgs a;
    const int dp = p.d <= 64 ? 64 : 128;
    const int tile = kRows / p.group;
    a.tile_tokens = tile;
    if (!make_q_map(&a.q, p, tile)) return cudaErrorInvalidValue;
    a.box_rows = kKeys;
    if (p.paged) {
        // the largest power of two that divides a page: boxes never straddle pages
        a.box_rows = p.pages.page_size & -p.pages.page_size;
        if (a.box_rows > kKeys) a.box_rows = kKeys;
        if (!make_page_maps(&a.k, &a.v, p, a.box_rows)) return cudaErrorInvalidValue;
    } else {
        const int64_t ext[4] = {p.d, p.n_tokens, p.hkv, 1};
        const int64_t ks[4] = {1, p.k.ts, p.k.hs, 0}, vs[4] = {1, p.v.ts, p.v.hs, 0};
        const int box[4] = {64, kKeys, 1, 1};
        if (!make_map(&a.k, p.k.p, 4, ext, ks, box) || !make_map(&a.v, p.v.p, 4, ext, vs, box))
            return cudaErrorInvalidValue;
    }
    a.out = p.out.p;
    a.out_ts = p.out.ts;
    a.out_hs = p.out.hs;
    a.lse = p.lse;
    a.cu = p.cu;
    a.used = p.used;
    a.table = p.pages.table;
    a.table_stride = p.pages.table_stride;
    a.max_pages = p.pages.max_pages;
    a.page_size = p.pages.page_size;
    a.n_pages = p.pages.n_pages;
    a.n_tokens = p.n_tokens;
    a.n_seqs = p.n_seqs;
    a.hq = p.hq;
    a.hkv = p.hkv;
    a.group = p.group;
    a.d = p.d;
    a.causal = p.causal;
    a.n_slots = slot_count(p.n_tokens, p.n_seqs, 2 * tile);
    a.splits = splits;
    a.div_group = make_fastdiv(static_cast<uint32_t>(p.group));
    a.div_cta = make_fastdiv(static_cast<uint32_t>(2 * tile));
    a.scale = p.scale;
    a.rule = rule_of(p);
    const int64_t rows = static_cast<int64_t>(p.n_tokens) * p.hq;
    a.part_o = workspace;
    a.part_lse = splits > 1 ? workspace + splits * rows * p.d : nullptr;
    cudaError_t err;
    if (p.paged) err = dp == 64 ? launch_fwd<64, true>(a, stream) : launch_fwd<128, true>(a, stream);
    else err = dp == 64 ? launch_fwd<64, false>(a, stream) : launch_fwd<128, false>(a, stream);
    if (err != cudaSuccess || splits <= 1) return err;
    return launch_attn_join(a.part_o, a.part_lse, p, splits, stream);
}

template <>
int attn_fwd_fault_of<kRule>(int *word)
{
    return read_fault_word(word, g_attn_fault);
}

#if PVR_SCORE_RULE == 0
cudaError_t launch_attn_join(const float *part_o, const float *part_lse, const AttnProblem &p, int splits,
                             cudaStream_t stream)
{
    const int rows = p.n_tokens * p.hq;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel, part_o, part_lse, p.out.p, p.out.ts, p.out.hs, rows, p.hq, p.d,
                              splits);
}

int attn_fault_word(int *word)
{
    return sum_fault_words(word, [](auto rule, int *w) { return attn_fwd_fault_of<decltype(rule)::value>(w); });
}
#endif

}  // namespace pvr
