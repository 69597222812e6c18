// Rotation by several position axes (GB300, sm_103a): in place or out of place, forward or
// backward, and with the append of keys and values to a paged cache.
//
// Mathematics.  y = x*cos + rotate_half(x)*sin with the angle of frequency j
// phi = position[axis(j)] * w_j (one binary32 product); the arithmetic after the angle is that
// of the rotation by one axis, bit for bit.
//
// One CTA owns a tile of consecutive tokens and moves every head of them: the first 16-byte
// loads go out before anything is known, then the tile's positions on all axes, then its rows of
// (cos, sin), shared by all heads, then the heads stream through.  Every element is read once
// and written once: the bound is HBM for long packs (16,384 tokens of 32/8 heads of 128, 336 MB a
// direction: 54 us, 6.2 TB/s, the evaluation of 64 angles a token beside 640 units of 32 bytes; an
// append of 17,043 tokens of 64/8 heads 116.5 us, 6.0 TB/s; 4,520 tokens of 16/16 heads of 80, which
// stay in L2, 12.7 us, one wave of CTAs), the chain of dependent loads for a decoding step (8 tokens
// 4.1 us, 11 through Python).  Registers are held to 11 resident CTAs an SM (the append: 10): 108 us
// for both directions where 9 CTAs took 113 and the compiler's choice 122.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fastdiv.cuh"
#include "host_checks.h"
#include "paged_checks.h"
#include "rope_axes.h"
#include "rope_core.cuh"

namespace {

using namespace pvr;

constexpr int kThreads = 128;
constexpr int kUnits = 2;               // 16-byte pair units in flight per thread
constexpr int kTileUnits = 640;         // about as many pair units a tile
constexpr int kMaxTile = 16;            // tokens per tile
constexpr int kSMs = 152;
constexpr int kMaxStaged = 256;         // sequences whose cu_seqlens and kv_lens are staged

struct AxesArgs {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_out, *v_out;   // the append's k_out and v_out: the pages
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
    int64_t kp_ps, kp_ts, kp_hs, vp_ps, vp_ts, vp_hs;
    const int32_t *cu, *kv_lens, *table;
    int64_t table_stride;
    const void *ids;
    int64_t ids_stride;
    const float4 *cache;                // cos/sin rows, or NULL
    int32_t cache_rows;
    int32_t max_pages, n_pages, page_size;
    int32_t n_seqs, n_tokens, staged;
    int32_t hq, hkv, h_tot, cph, tile, n_axes, ids64;
    int32_t in_place, bwd;
    int32_t rows_at_once;               // (cos, sin) rows that a CTA's threads make at a time
    FastDiv div_htot, div_cph, div_row;
    float w[kMaxHalf];
    uint8_t axis[kMaxHalf];
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

// Every (cos, sin) of a tile is one thread's: thread i has frequency i % (d/2), whatever the token, so
// that its frequency and axis are read once, and its position on that axis alone.
template <bool APPEND>
__global__ void __launch_bounds__(kThreads, APPEND ? 10 : 11) rope_axes_kernel(const __grid_constant__ AxesArgs a)
{
    extern __shared__ __align__(16) float4 s_cs[];
    __shared__ int s_row[kMaxTile];                          // 0: the token is left out
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
                                 : !APPEND || head < a.hq + a.hkv ? a.k + (t * a.k_ts + (head - a.hq) * a.k_hs)
                                                                  : a.v + (t * a.v_ts + (head - a.hq - a.hkv) * a.v_hs);
        return p + 8 * w.chunk;
    };
    // where the unit goes; NULL: nowhere
    auto target = [&](const Where &w) -> __nv_bfloat16 * {
        const int64_t t = t0 + static_cast<int64_t>(w.tok);
        const int head = static_cast<int>(w.head);
        if (head < a.hq || !APPEND) {
            if (a.in_place && s_row[w.tok] == 0) return nullptr;
            return (head < a.hq ? a.q_out + (t * a.qo_ts + head * a.qo_hs)
                                : a.k_out + (t * a.ko_ts + (head - a.hq) * a.ko_hs)) + 8 * w.chunk;
        }
        const bool key = head < a.hq + a.hkv;
        const int64_t slot = key ? s_slot_k[w.tok] : s_slot_v[w.tok];
        if (slot < 0) return nullptr;
        return (key ? a.k_out + (slot + (head - a.hq) * a.kp_hs)
                    : a.v_out + (slot + (head - a.hq - a.hkv) * a.vp_hs)) + 8 * w.chunk;
    };

    // this thread's place in a token's (cos, sin) row, which is in the cache's [quad][chunk] order
    const int per_row = 2 * row4;                            // frequencies, d / 2
    const int my_row = static_cast<int>(fast_div(threadIdx.x, a.div_row)), at = static_cast<int>(threadIdx.x) - my_row * per_row;
    const int quad = static_cast<int>(fast_div(static_cast<uint32_t>(at) >> 1, a.div_cph));
    const int freq = 8 * ((at >> 1) - quad * cph) + 2 * quad + (at & 1);
    const float w_j = a.w[freq];
    const int64_t axis = a.axis[freq];

    // the grid may be scheduled while the kernel before it drains: nothing is read earlier
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    Where unit[kUnits];
    uint4 lo[kUnits], hi[kUnits];
    auto load = [&](uint32_t base) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const uint32_t u = base + threadIdx.x + k * kThreads;
            if (u >= units) continue;
            unit[k] = where(u);
            const __nv_bfloat16 *src = source(unit[k]);
            lo[k] = load_stream(src);
            hi[k] = load_stream(src + h);
        }
    };
    auto id_of = [&](int64_t x, int t) {
        return a.ids64 ? static_cast<const int64_t *>(a.ids)[x * a.ids_stride + t]
                       : static_cast<int64_t>(static_cast<const int32_t *>(a.ids)[x * a.ids_stride + t]);
    };
    load(0);

    // which tokens are left out, and where they go, one thread per token
    int32_t *s_cu = reinterpret_cast<int32_t *>(s_cs + a.tile * row4);
    if (APPEND && a.staged) {
        for (int i = threadIdx.x; i < 2 * a.n_seqs + 1; i += kThreads)
            s_cu[i] = i <= a.n_seqs ? a.cu[i] : a.kv_lens[i - a.n_seqs - 1];
        __syncthreads();
    }
    if (static_cast<int>(threadIdx.x) < tt) {
        const int t = t0 + static_cast<int>(threadIdx.x);
        bool in = true;
        for (int x = 0; x < a.n_axes; ++x) {
            const int64_t p = id_of(x, t);
            in = in && p >= 0 && p < kMaxTokens;
        }
        if (APPEND) {
            const int32_t *cu = a.staged ? s_cu : a.cu, *kv = a.staged ? s_cu + a.n_seqs + 1 : a.kv_lens;
            int64_t slot_k = -1, slot_v = -1;
            const int s = sequence_of(cu, a.n_seqs, t);
            int pos = -1;
            if (s >= 0) {
                const int64_t p = static_cast<int64_t>(kv[s]) - (static_cast<int64_t>(cu[s + 1]) - t);
                if (p >= 0 && p < kMaxTokens && cu[s] >= 0) pos = static_cast<int>(p);
            }
            in = in && pos >= 0;
            if (in) {
                const int index = pos / a.page_size;
                const int in_page = pos - index * a.page_size;
                const int page = index < a.max_pages ? a.table[s * a.table_stride + index] : -1;
                if (page >= 0 && page < a.n_pages) {
                    slot_k = page * a.kp_ps + in_page * a.kp_ts;
                    slot_v = page * a.vp_ps + in_page * a.vp_ts;
                }
            }
            s_slot_k[threadIdx.x] = slot_k;
            s_slot_v[threadIdx.x] = slot_v;
        }
        s_row[threadIdx.x] = in ? 1 : 0;
    }

    // (cos, sin) rows of the tile; what a token left out gets here is not used
    if (my_row < a.rows_at_once) {
        float2 *dst = reinterpret_cast<float2 *>(s_cs);
        for (int i = my_row; i < tt; i += a.rows_at_once) {
            const int64_t id = id_of(axis, t0 + i);
            const int pos = id >= 0 && id < kMaxTokens ? static_cast<int>(id) : 0;
            float2 cs = pos < a.cache_rows
                            ? __ldg(reinterpret_cast<const float2 *>(a.cache + static_cast<int64_t>(pos) * row4) + at)
                            : cos_sin_at(pos, w_j);
            if (a.bwd) cs.y = -cs.y;
            dst[i * per_row + at] = cs;
        }
    }
    __syncthreads();

    auto finish = [&](const Where &w, uint4 x, uint4 y) {
        __nv_bfloat16 *dst = target(w);
        if (dst == nullptr) return;
        if ((!APPEND || static_cast<int>(w.head) < a.hq + a.hkv) && s_row[w.tok] != 0) {
            const float4 *cs = s_cs + w.tok * row4 + w.chunk;
            rotate2(x.x, y.x, cs[0]);
            rotate2(x.y, y.y, cs[cph]);
            rotate2(x.z, y.z, cs[2 * cph]);
            rotate2(x.w, y.w, cs[3 * cph]);
        }
        if (APPEND) {                   // read again soon, by the attention
            *reinterpret_cast<uint4 *>(dst) = x;
            *reinterpret_cast<uint4 *>(dst + h) = y;
        } else {
            __stcs(reinterpret_cast<uint4 *>(dst), x);
            __stcs(reinterpret_cast<uint4 *>(dst + h), y);
        }
    };
    for (uint32_t base = 0;;) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
            if (base + threadIdx.x + k * kThreads < units) finish(unit[k], lo[k], hi[k]);
        base += kUnits * kThreads;
        if (base >= units) break;
        load(base);
    }
}

// Sections, flags and positions of the axes; fills the arguments' frequencies.
int check_axes(const rope_axes &x, int64_t T, int32_t head_dim, double theta, double scale,
               const rope_cos_sin_cache *cache, AxesArgs &a)
{
    constexpr int kKnown = ROPE_AXES_INTERLEAVED | ROPE_AXES_OWN_FREQUENCIES | ROPE_AXES_IDS_INT64;
    if (x.n_axes < 1 || x.n_axes > ROPE_MAX_AXES) return ROPE_ERR_SHAPE;
    if ((x.flags & ~kKnown) != 0) return ROPE_ERR_UNSUPPORTED;
    const int half = head_dim / 2;
    int64_t sum = 0;
    for (int i = 0; i < ROPE_MAX_AXES; ++i) {
        if (i < x.n_axes ? x.sections[i] < 1 : x.sections[i] != 0) return ROPE_ERR_SHAPE;
        sum += x.sections[i];
    }
    if (sum != half) return ROPE_ERR_SHAPE;
    if ((x.flags & ROPE_AXES_OWN_FREQUENCIES) != 0 && cache != nullptr) return ROPE_ERR_CACHE;
    if (T > 0) {
        if (x.position_ids == nullptr) return ROPE_ERR_NULL;
        if (!aligned(x.position_ids, (x.flags & ROPE_AXES_IDS_INT64) != 0 ? 8 : 4)) return ROPE_ERR_ALIGN;
        if (x.n_axes > 1 && (x.position_stride < 0 || x.position_stride > (int64_t(1) << 56))) return ROPE_ERR_SHAPE;
    }
    host_inv_freq(theta, head_dim, scale, a.w);
    int had[ROPE_MAX_AXES] = {};
    for (int j = 0, turn = 0; j < half; ++j) {
        while (had[turn] == x.sections[turn]) turn = (turn + 1) % x.n_axes;
        a.axis[j] = static_cast<uint8_t>(turn);
        if ((x.flags & ROPE_AXES_OWN_FREQUENCIES) != 0)
            a.w[j] = static_cast<float>(std::pow(theta, -static_cast<double>(had[turn]) / x.sections[turn]) / scale);
        ++had[turn];
        if ((x.flags & ROPE_AXES_INTERLEAVED) != 0) turn = (turn + 1) % x.n_axes;
    }
    a.ids = x.position_ids;
    a.ids_stride = x.position_stride;
    a.ids64 = (x.flags & ROPE_AXES_IDS_INT64) != 0;
    a.n_axes = x.n_axes;
    return ROPE_OK;
}

template <bool APPEND>
int launch(AxesArgs &a, int64_t T, int64_t d, const rope_cos_sin_cache *cs, void *stream)
{
    a.cache = cs != nullptr && cs->rows > 0 ? reinterpret_cast<const float4 *>(cs->data) : nullptr;
    a.cache_rows = a.cache != nullptr ? static_cast<int32_t>(cs->rows) : 0;
    a.n_tokens = static_cast<int32_t>(T);
    a.h_tot = a.hq + (APPEND ? 2 : 1) * a.hkv;
    a.cph = static_cast<int32_t>(d / 16);
    a.div_htot = make_fastdiv(static_cast<uint32_t>(a.h_tot));
    a.div_cph = make_fastdiv(static_cast<uint32_t>(a.cph));
    a.div_row = make_fastdiv(static_cast<uint32_t>(d / 2));
    a.rows_at_once = static_cast<int32_t>(kThreads / (d / 2));   // d <= 256: at least one
    // Tokens a tile: kTileUnits of them, so that all threads evaluate (two tokens of 40 heads of 128; one
    // token a tile took 128 us for what two take 113); fewer where the tiles would not fill the GPU
    const int64_t per_token = static_cast<int64_t>(a.h_tot) * a.cph;
    int64_t fit = kTileUnits / per_token, spread = T / (kSMs * 8);
    if (fit > spread) fit = spread;
    a.tile = static_cast<int32_t>(fit < 1 ? 1 : fit > kMaxTile ? kMaxTile : fit);
    const size_t smem = static_cast<size_t>(a.tile) * 4 * a.cph * sizeof(float4) +
                        (APPEND && a.staged ? (2 * static_cast<size_t>(a.n_seqs) + 1) * sizeof(int32_t) : 0);
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
    return cudaLaunchKernelEx(&cfg, rope_axes_kernel<APPEND>, a) == cudaSuccess ? ROPE_OK : ROPE_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int rope_axes_apply(const rope_qk_desc *dp, const rope_axes *axes, void *stream)
{
    if (dp == nullptr || axes == nullptr) return ROPE_ERR_NULL;
    const rope_qk_desc &p = *dp;
    const int64_t T = p.total_tokens, d = p.head_dim;
    if (T < 0 || p.n_q_heads < 1 || p.n_kv_heads < 1 || p.n_q_heads > (1 << 20) || p.n_kv_heads > (1 << 20))
        return ROPE_ERR_SHAPE;
    if (p.cu_seqlens != nullptr || p.position_ids != nullptr || p.seq_used != nullptr || p.segments != nullptr ||
        p.n_seqs != 0 || p.n_segments != 0 || p.token_offset != 0 || p.flags != 0 || p.reserved != 0)
        return ROPE_ERR_UNSUPPORTED;
    int rc;
    if ((rc = check_head_dim(p.head_dim)) != ROPE_OK || (rc = check_theta(p.theta)) != ROPE_OK ||
        (rc = check_scale(p.position_scale)) != ROPE_OK)
        return rc;
    AxesArgs a{};
    if ((rc = check_axes(*axes, T, p.head_dim, p.theta, p.position_scale, p.cos_sin_cache, a)) != ROPE_OK) return rc;
    if ((rc = check_cache(p.cos_sin_cache, p.head_dim, p.theta, p.position_scale)) != ROPE_OK) return rc;
    if (T > INT32_MAX / 2) return ROPE_ERR_UNSUPPORTED;
    if (T == 0) return ROPE_OK;
    const View q{p.q, T, p.n_q_heads, p.q_stride_token, p.q_stride_head, d};
    const View k{p.k, T, p.n_kv_heads, p.k_stride_token, p.k_stride_head, d};
    const bool in_place = p.q_out == nullptr && p.k_out == nullptr;
    if (!in_place && (p.q_out == nullptr || p.k_out == nullptr)) return ROPE_ERR_NULL;
    const View qo = in_place ? q : View{p.q_out, T, p.n_q_heads, p.q_out_stride_token, p.q_out_stride_head, d};
    const View ko = in_place ? k : View{p.k_out, T, p.n_kv_heads, p.k_out_stride_token, p.k_out_stride_head, d};
    for (const View *v : {&q, &k, &qo, &ko})
        if ((rc = check_view(*v)) != ROPE_OK) return rc;
    if (!views_disjoint(q, k)) return ROPE_ERR_OVERLAP;
    if (!in_place) {
        if (!views_disjoint(qo, ko)) return ROPE_ERR_OVERLAP;
        for (const View *o : {&qo, &ko})
            for (const View *i : {&q, &k})
                if (overlap(o->base, o->bytes(), i->base, i->bytes())) return ROPE_ERR_OVERLAP;
    }
    if ((rc = check_cache_device(p.cos_sin_cache)) != ROPE_OK) return rc;
    a.q = static_cast<const __nv_bfloat16 *>(q.base);
    a.k = static_cast<const __nv_bfloat16 *>(k.base);
    a.q_out = static_cast<__nv_bfloat16 *>(const_cast<void *>(qo.base));
    a.k_out = static_cast<__nv_bfloat16 *>(const_cast<void *>(ko.base));
    a.q_ts = q.ts; a.q_hs = q.hs; a.k_ts = k.ts; a.k_hs = k.hs;
    a.qo_ts = qo.ts; a.qo_hs = qo.hs; a.ko_ts = ko.ts; a.ko_hs = ko.hs;
    a.hq = p.n_q_heads;
    a.hkv = p.n_kv_heads;
    a.in_place = in_place ? 1 : 0;
    a.bwd = p.backward ? 1 : 0;
    return launch<false>(a, T, d, p.cos_sin_cache, stream);
}

int rope_kv_append_axes(const rope_kv_append_desc *dp, const rope_axes *axes, void *stream)
{
    if (dp == nullptr || axes == nullptr) return ROPE_ERR_NULL;
    const rope_kv_append_desc &p = *dp;
    const rope_paged_kv &c = p.cache;
    const int64_t T = p.total_tokens;
    AppendViews w;
    int rc = check_append(p, w);
    if (rc != ROPE_OK) return rc;
    AxesArgs a{};
    if ((rc = check_axes(*axes, T, c.head_dim, p.theta, p.position_scale, p.cos_sin_cache, a)) != ROPE_OK) return rc;
    if (T == 0) return ROPE_OK;
    a.q = static_cast<const __nv_bfloat16 *>(p.q);
    a.k = static_cast<const __nv_bfloat16 *>(p.k);
    a.v = static_cast<const __nv_bfloat16 *>(p.v);
    a.q_out = static_cast<__nv_bfloat16 *>(const_cast<void *>(w.q_out.base));
    a.k_out = static_cast<__nv_bfloat16 *>(c.k);
    a.v_out = static_cast<__nv_bfloat16 *>(c.v);
    a.q_ts = w.q.ts; a.q_hs = w.q.hs; a.k_ts = w.k.ts; a.k_hs = w.k.hs; a.v_ts = w.v.ts; a.v_hs = w.v.hs;
    a.qo_ts = w.q_out.ts; a.qo_hs = w.q_out.hs;
    a.kp_ps = c.k_stride_page; a.kp_ts = c.k_stride_token; a.kp_hs = c.k_stride_head;
    a.vp_ps = c.v_stride_page; a.vp_ts = c.v_stride_token; a.vp_hs = c.v_stride_head;
    a.cu = p.cu_seqlens; a.kv_lens = p.kv_lens; a.table = p.page_table;
    a.table_stride = p.page_table_stride;
    a.max_pages = p.max_pages;
    a.n_pages = static_cast<int32_t>(c.n_pages);
    a.page_size = c.page_size;
    a.n_seqs = p.n_seqs;
    a.staged = p.n_seqs < kMaxStaged ? 1 : 0;
    a.hq = p.n_q_heads;
    a.hkv = c.n_kv_heads;
    a.in_place = p.q_out == nullptr ? 1 : 0;
    return launch<true>(a, T, c.head_dim, p.cos_sin_cache, stream);
}

}  // extern "C"
