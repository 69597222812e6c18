// Attention in its plainest form: one warp per query row (forward, dq) or key row (dk,
// dv), binary32 throughout, one key or query at a time with the running maximum and sum.
// Bound by its shuffles: about 20 instructions per (row, key).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_internal.h"

namespace pvr {
namespace {

constexpr int kWarps = 8;

struct Sample {
    int start, rows, keys, offset;   // rows: query rows; key j is visible to row i when j <= i + offset
};

// The sample of token t: false outside the pack and past the rows in use.
__device__ bool sample_of(const AttnProblem &p, int t, Sample &s)
{
    const int n = p.n_seqs;
    if (n <= 0 || t < p.cu[0] || t >= p.cu[n]) return false;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int a = p.cu[lo], b = min(p.cu[lo + 1], p.n_tokens);
    if (a < 0 || t < a || t >= b) return false;
    s.start = a;
    if (p.paged) {
        s.rows = b - a;
        s.keys = static_cast<int>(min(static_cast<int64_t>(max(p.used[lo], 0)),
                                      static_cast<int64_t>(p.pages.max_pages) * p.pages.page_size));
        s.offset = p.used[lo] - (p.cu[lo + 1] - a);
        if (t - a + s.offset < 0) return false;
    } else {
        s.rows = p.used != nullptr ? min(b - a, p.used[lo]) : b - a;
        if (t - a >= s.rows) return false;
        s.keys = s.rows;
        s.offset = 0;
    }
    return true;
}

__device__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ void store4(__nv_bfloat16 *p, float4 v)
{
    __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
}

__device__ float dot(float4 a, float4 b)
{
    float x = a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

__device__ void axpy(float4 &y, float a, float4 x)
{
    y.x += a * x.x; y.y += a * x.y; y.z += a * x.z; y.w += a * x.w;
}

__device__ float4 zero4() { return make_float4(0.f, 0.f, 0.f, 0.f); }

// Key and value of position j of a sample (4 elements a lane, zero past head_dim).
__device__ void key_value(const AttnProblem &p, const Sample &s, int seq_row, int j, int kvh, int e, float4 &k, float4 &v)
{
    k = zero4();
    v = zero4();
    if (e >= p.d) return;
    if (!p.paged) {
        const int64_t t = s.start + j;
        k = load4(p.k.p + t * p.k.ts + kvh * p.k.hs + e);
        v = load4(p.v.p + t * p.v.ts + kvh * p.v.hs + e);
        return;
    }
    const Pages &g = p.pages;
    const int page = g.table[seq_row * g.table_stride + j / g.page_size];
    if (page < 0 || page >= g.n_pages) return;
    const int64_t slot = j % g.page_size;
    k = load4(g.k + page * g.k_ps + slot * g.k_ts + kvh * g.k_hs + e);
    v = load4(g.v + page * g.v_ps + slot * g.v_ts + kvh * g.v_hs + e);
}

__global__ void simple_bwd_dq(const AttnProblem p)
{
    const int64_t w = blockIdx.x * int64_t(kWarps) + threadIdx.x / 32;
    const int t = static_cast<int>(w / p.hq), head = static_cast<int>(w % p.hq), e = (threadIdx.x & 31) * 4;
    if (t >= p.n_tokens) return;
    Sample s;
    float4 dq = zero4();
    float delta = 0.f;
    if (sample_of(p, t, s)) {
        const bool in = e < p.d;
        const float4 q = in ? load4(p.q.p + t * p.q.ts + head * p.q.hs + e) : zero4();
        const float4 g = in ? load4(p.dout.p + t * p.dout.ts + head * p.dout.hs + e) : zero4();
        const float4 o = in ? load4(p.out.p + t * p.out.ts + head * p.out.hs + e) : zero4();
        delta = dot(g, o);
        const float lse = p.lse[static_cast<int64_t>(head) * p.n_tokens + t];
        const int last = p.causal ? t - s.start + 1 : s.keys;
        for (int j = 0; j < last; ++j) {
            float4 k, v;
            key_value(p, s, 0, j, head / p.group, e, k, v);
            const float pj = expf(dot(q, k) * p.scale - lse);
            axpy(dq, pj * (dot(g, v) - delta) * p.scale, k);
        }
    }
    if (e < p.d) store4(p.dq.p + t * p.dq.ts + head * p.dq.hs + e, dq);
    if (e == 0) p.delta[static_cast<int64_t>(head) * p.n_tokens + t] = delta;
}

__global__ void simple_bwd_dkv(const AttnProblem p)
{
    const int64_t w = blockIdx.x * int64_t(kWarps) + threadIdx.x / 32;
    const int t = static_cast<int>(w / p.hkv), kvh = static_cast<int>(w % p.hkv), e = (threadIdx.x & 31) * 4;
    if (t >= p.n_tokens) return;
    Sample s;
    float4 dk = zero4(), dv = zero4();
    if (sample_of(p, t, s)) {
        float4 k, v;
        key_value(p, s, 0, t - s.start, kvh, e, k, v);
        for (int g = 0; g < p.group; ++g) {
            const int head = kvh * p.group + g;
            for (int i = p.causal ? t - s.start : 0; i < s.rows; ++i) {
                const int64_t r = s.start + i, st = static_cast<int64_t>(head) * p.n_tokens + r;
                const float4 q = e < p.d ? load4(p.q.p + r * p.q.ts + head * p.q.hs + e) : zero4();
                const float4 o = e < p.d ? load4(p.dout.p + r * p.dout.ts + head * p.dout.hs + e) : zero4();
                const float pj = expf(dot(q, k) * p.scale - p.lse[st]);
                axpy(dv, pj, o);
                axpy(dk, pj * (dot(o, v) - p.delta[st]) * p.scale, q);
            }
        }
    }
    if (e >= p.d) return;
    store4(p.dk.p + t * p.dk.ts + kvh * p.dk.hs + e, dk);
    store4(p.dv.p + t * p.dv.ts + kvh * p.dv.hs + e, dv);
}

unsigned grid_of(int64_t warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_attn_simple_bwd(const AttnProblem &p, cudaStream_t stream)
{
    simple_bwd_dq<<<grid_of(int64_t(p.n_tokens) * p.hq), 32 * kWarps, 0, stream>>>(p);
    simple_bwd_dkv<<<grid_of(int64_t(p.n_tokens) * p.hkv), 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pvr
