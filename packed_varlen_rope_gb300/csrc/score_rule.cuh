// Rules on attention scores, compiled into instances of the attention kernels: PVR_SCORE_RULE is
// 0 (none), or a sum of the bits below; every instance but 0 honours a prefix, the sequence's
// first keys that all its rows see.
//
//   y_ij = cap tanh(scale q_i.k_j / cap) - slope_h |i - j|
//
// Scores become exponents of 2 before the softmax, x = y log2(e): K tanh(s a) with K = cap
// log2(e) and a = scale / cap for capped ones, s c with c = scale log2(e) for others.  tanh is
// u P(u^2) for |u| <= 1 (fit_tanh.py: relative error 7.2e-6, 2.8e-4 of a score capped at 50,
// against the 2^-9 that rounding a weight to bf16 moves), and 1 - 2 / (1 + 2^(2 log2(e) u))
// beyond, whose error of about 2^-22 of the cap is small against a score that large.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "attn_internal.h"
#include "tensor_core.cuh"

#ifndef PVR_SCORE_RULE
#define PVR_SCORE_RULE 0
#endif

namespace pvr {
namespace {

constexpr int kRule = PVR_SCORE_RULE;
constexpr int kRulePrefix = 1, kRuleCap = 2, kRuleBias = 4;
constexpr bool kRuled = kRule != 0;
constexpr bool kCap = (kRule & kRuleCap) != 0, kBias = (kRule & kRuleBias) != 0;
constexpr bool kShaped = kCap || kBias;      // scores are exponents of 2 before the softmax

// What a kernel knows of the rule.
struct ScoreRule {
    float a, k, a2;                          // capped scores: scale / cap, cap log2(e), 2 log2(e) scale / cap
    float c;                                 // others: scale log2(e)
    int32_t fixed;                           // capped exponents within +-80: no maximum is needed
    const float *slopes;                     // [hq]
    const int32_t *prefix;                   // [n_seqs], or NULL
};

constexpr float kTanh0 = 9.999928679e-01f, kTanh1 = -3.329738354e-01f, kTanh2 = 1.303347757e-01f, kTanh3 = -4.476498296e-02f,
                kTanh4 = 9.010406017e-03f;

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Both halves of a pair alike.
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// tanh of two scores times a.  wide: some score of the warp is past the fit, so each takes the form
// that is right for it (no branch of its own: what follows is for converged warps).  The factor is
// 1 - tanh^2, the gradient's.
template <bool WIDE>
__device__ __forceinline__ float2 tanh2(const ScoreRule &r, float2 s, float2 &factor)
{
    const float2 u = mul2(s, twice(r.a)), z = mul2(u, u);
    float2 p = fma2(z, twice(kTanh4), twice(kTanh3));
    p = fma2(z, p, twice(kTanh2));
    p = fma2(z, p, twice(kTanh1));
    p = fma2(z, p, twice(kTanh0));
    float2 t = mul2(u, p);
    factor = fma2(t, mul2(t, twice(-1.0f)), twice(1.0f));
    if (WIDE) {
        const float qx = rcp(1.0f + ex2(s.x * r.a2)), qy = rcp(1.0f + ex2(s.y * r.a2));
        // (a NaN score takes the second form, and stays one)
        const bool nx = fabsf(u.x) <= 1.0f, ny = fabsf(u.y) <= 1.0f;
        t.x = nx ? t.x : fmaf(-2.0f, qx, 1.0f);
        t.y = ny ? t.y : fmaf(-2.0f, qy, 1.0f);
        factor.x = nx ? factor.x : 4.0f * qx * (1.0f - qx);
        factor.y = ny ? factor.y : 4.0f * qy * (1.0f - qy);
    }
    return t;
}

// The largest magnitude of N scores (NaN is passed over).
template <int N>
__device__ __forceinline__ float largest(const uint32_t (&s)[N])
{
    float top[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < N; j += 2)
        top[(j >> 1) & 1] = max3(top[(j >> 1) & 1], fabsf(__uint_as_float(s[j])), fabsf(__uint_as_float(s[j + 1])));
    return fmaxf(top[0], top[1]);
}

// Biases of a thread's columns, a pair at a time, the first one `distance` past the row's own
// place: -slope2 |distance|.  Distances are whole numbers and exact.
struct Bias {
    float2 at, slope;
    __device__ __forceinline__ Bias(float slope2, float distance)
        : at(make_float2(distance, distance + 1.0f)), slope(twice(-slope2)) {}
    __device__ __forceinline__ float2 next()
    {
        const float2 x = mul2(slope, make_float2(fabsf(at.x), fabsf(at.y)));
        at = add2(at, twice(2.0f));
        return x;
    }
};

// N scores, columns from `distance` past the row on, to exponents of 2, in place.
template <bool WIDE, int N>
__device__ __forceinline__ void shape(const ScoreRule &r, uint32_t (&s)[N], float slope2, float distance)
{
    Bias bias(slope2, distance);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        float2 x = make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), factor;
        if (kCap) x = tanh2<WIDE>(r, x, factor);
        const float2 scale = twice(kCap ? r.k : r.c);
        x = kBias ? fma2(x, scale, bias.next()) : mul2(x, scale);
        s[j] = __float_as_uint(x.x);
        s[j + 1] = __float_as_uint(x.y);
    }
}

// Whether some score of a converged warp is past the fit of the tanh.  A thread that holds one may
// have it in a place that nobody sees: the two forms give a score within the fit the same bits.
template <int N>
__device__ __forceinline__ bool any_wide(const ScoreRule &r, const uint32_t (&s)[N])
{
    return __any_sync(0xffffffffu, largest(s) * r.a > 1.0f);
}

template <int N>
__device__ __forceinline__ void shape_any(const ScoreRule &r, uint32_t (&s)[N], float slope2, float distance)
{
    if (kCap && any_wide(r, s)) shape<true>(r, s, slope2, distance);
    else shape<false>(r, s, slope2, distance);
}

// The keys at the start of a sequence that all its rows see.
__device__ __forceinline__ int prefix_of(const ScoreRule &r, int sample, int n_seqs, int keys)
{
    if (!kRuled || r.prefix == nullptr || sample < 0 || sample >= n_seqs) return 0;
    return min(r.prefix[sample], keys);
}

// Host side: the rule of a problem.
inline ScoreRule rule_of(const AttnProblem &p)
{
    constexpr float kLog2 = 1.4426950408889634f;
    ScoreRule r{};
    if (p.cap > 0.0f) {
        r.a = p.scale / p.cap;
        r.k = p.cap * kLog2;
        r.a2 = 2.0f * kLog2 * r.a;
    }
    r.c = p.scale * kLog2;
    r.fixed = p.cap > 0.0f && p.slopes == nullptr && r.k <= 80.0f;
    r.slopes = p.slopes;
    r.prefix = p.prefix;
    return r;
}

}  // namespace
}  // namespace pvr
