// Rules on attention scores, compiled into instances of the attention kernels: PVR_SCORE_RULE is
// 0 (none), or a sum of the bits below; every instance but 0 honours a prefix, the sequence's
// first keys that all its rows see.
//
//   y_ij = cap tanh(scale q_i.k_j / cap) - slope_h |i - j|
//
// Scores become exponents of 2 before the softmax, x = y log2(e): K tanh(u) with K = cap log2(e) and
// u = s scale / cap for capped ones, s c with c = scale log2(e) for others.  The tanh takes one of
// four forms:
//
//   kSmall  K u P(u^2), degree 5: 4 packed operations for two scores, absolute error 5.6e-6 of the cap
//           (fit_tanh.py); for caps up to 128, where no score of the warp's chunk is past half the cap
//   kNear   the same of degree 7, 5 operations, 6.7e-6; where none is past 0.8 caps
//   kAny    K (1 - 2 q), q = 1 / (1 + e^2u), off by about 2^-22 K: 3 packed operations, but two special
//           functions a score; for such caps elsewhere
//   kLarge  caps past 128: u P(u^2), degree 11, relative error 6.1e-7, for |u| <= 1, so that scores far
//           below the cap keep theirs; kAny's beyond; chosen score by score
//
// 16,384 tokens of a packed batch, 32/8 heads of 128, forward and backward: nearly all chunks kSmall
// (scores of deviation 6, cap 50) 637 and 2,250-2,290 us (kNear in its place: 8 and 1 % more), nearly
// all kAny (cap 20) 901-915 and 2,815 us, kLarge 1,212-1,219 and 3,270 us; without a cap 501-509 and 1,686-1,713 us.  kAny
// for every second, third or fourth pair among kNear, to spread the work over the pipes, took 20 to
// 25 % more forward and 0 to 3 % backward.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

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
    float near[4], near_limit;               // kNear: x = s sum near_i s^2i, for |s| up to the limit
    float small[3], small_limit;             // kSmall
    float unit;                              // of the gradient's factor, unit (tanh^2 - 1): K^2, as kNear has K tanh; 1 with kLarge
    float dq_scale;                          // what dq and dk are multiplied by at the end: -scale / unit
    int32_t large;                           // the cap takes kLarge
    const float *slopes;                     // [hq]
    const int32_t *prefix;                   // [n_seqs], or NULL
};

constexpr float kNearCap = 128.0f, kNearEnd = 0.8f;
constexpr float kNear0 = 9.999243658e-01f, kNear1 = -3.317269685e-01f, kNear2 = 1.238189323e-01f, kNear3 = -3.164692249e-02f;
constexpr float kSmallEnd = 0.5f;
constexpr float kSmall0 = 9.999222584e-01f, kSmall1 = -3.308141013e-01f, kSmall2 = 1.124106519e-01f;
constexpr float kTanh0 = 9.999993948e-01f, kTanh1 = -3.332895137e-01f, kTanh2 = 1.328072065e-01f, kTanh3 = -5.158598840e-02f,
                kTanh4 = 1.672085518e-02f, kTanh5 = -3.058229038e-03f;

// (kLine: uncapped scores, biased, of rows that see keys on one side of them alone)
enum Form { kSmall, kNear, kAny, kLarge, kLine };
template <Form FORM>
using FormTag = std::integral_constant<Form, FORM>;

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Both halves of a pair alike.
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// The largest magnitude of three.
__device__ __forceinline__ float max3_abs(float a, float b, float c)
{
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two scores to exponents of 2, plus an offset: K tanh(a s) + offset or s c + offset.  top is the
// offset, K + offset for kAny.  factor: unit (tanh^2 - 1), of the gradient.
template <Form FORM>
__device__ __forceinline__ float2 exponent2(const ScoreRule &r, float2 s, float2 top, float2 &factor)
{
    if (!kCap) return fma2(s, twice(r.c), top);
    if (FORM == kNear || FORM == kSmall) {
        const float2 z = mul2(s, s);
        float2 p;
        if (FORM == kSmall) {
            p = fma2(z, twice(r.small[2]), twice(r.small[1]));
            p = fma2(z, p, twice(r.small[0]));
        } else {
            p = fma2(z, twice(r.near[3]), twice(r.near[2]));
            p = fma2(z, p, twice(r.near[1]));
            p = fma2(z, p, twice(r.near[0]));
        }
        const float2 y = mul2(s, p);
        factor = fma2(y, y, twice(-r.unit));
        return fma2(s, p, top);
    }
    const float2 e = mul2(s, twice(r.a2));
    const float2 d = add2(make_float2(ex2(e.x), ex2(e.y)), twice(1.0f));
    const float2 q = make_float2(rcp(d.x), rcp(d.y));
    float2 x = FORM == kAny ? fma2(q, twice(-2.0f * r.k), top) : add2(fma2(q, twice(-2.0f * r.k), twice(r.k)), top);
    factor = mul2(q, fma2(q, twice(4.0f * r.unit), twice(-4.0f * r.unit)));
    if (FORM == kLarge) {
        const float2 u = mul2(s, twice(r.a)), z = mul2(u, u);
        float2 p = fma2(z, twice(kTanh5), twice(kTanh4));
        p = fma2(z, p, twice(kTanh3));
        p = fma2(z, p, twice(kTanh2));
        p = fma2(z, p, twice(kTanh1));
        p = fma2(z, p, twice(kTanh0));
        const float2 t = mul2(u, p), y = fma2(t, twice(r.k), top);
        const float2 f = fma2(t, t, twice(-1.0f));           // (unit is 1)
        if (fabsf(u.x) <= 1.0f) { x.x = y.x; factor.x = f.x; }
        if (fabsf(u.y) <= 1.0f) { x.y = y.y; factor.y = f.y; }
    }
    return x;
}

// What exponent2 takes as `top` for a thread's columns, a pair at a time, the first one `distance`
// past the row's own place: -slope2 |distance| + offset, and K with kAny.  Distances are whole numbers
// and exact.  With kLine the visible columns are on one side, and slope2 has its sign: the bias is
// slope2 distance, a sum from 16 columns to the next.
template <Form FORM>
struct Tops {
    float first, slope1, offset;
    float2 at, slope, base;
    __device__ __forceinline__ Tops(const ScoreRule &r, float slope2, float distance, float offset_)
        : first(distance), slope1(slope2), offset(offset_), at(make_float2(distance, distance + 1.0f)),
          slope(twice(FORM == kLine ? 2.0f * slope2 : -slope2)), base(twice(kCap && FORM == kAny ? r.k + offset_ : offset_)) {}
    __device__ __forceinline__ float2 next(int j)
    {
        if (!kBias) return base;
        float2 x;
        if (FORM == kLine) {
            if (j % 16 == 0) {
                at.x = fmaf(slope1, first + j, offset);
                at.y = at.x + slope1;
            }
            x = at;
            at = add2(at, slope);
        } else {
            x = fma2(slope, make_float2(fabsf(at.x), fabsf(at.y)), base);
            at = add2(at, twice(2.0f));
        }
        return x;
    }
};

// N scores, columns from `distance` past the row on, to exponents of 2 less `shift`, in place.
template <Form FORM, int N>
__device__ __forceinline__ void shape(const ScoreRule &r, uint32_t (&s)[N], float slope2, float distance, float shift)
{
    Tops<FORM> tops(r, slope2, distance, -shift);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        float2 factor;
        const float2 x = exponent2<FORM>(r, make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), tops.next(j), factor);
        s[j] = __float_as_uint(x.x);
        s[j + 1] = __float_as_uint(x.y);
    }
}

// Calls fn(FormTag<FORM>) with the form for N scores of every thread of a converged warp.  Scores
// that nobody sees must not decide (hidden: the thread's row is none): they are 0 here.  line: the
// rows see keys on one side alone.
template <int N, typename Fn>
__device__ __forceinline__ void by_form(const ScoreRule &r, const uint32_t (&s)[N], bool hidden, bool line, Fn fn)
{
    if (!kCap) {
        if (kBias && line) fn(FormTag<kLine>{});
        else fn(FormTag<kNear>{});
        return;
    }
    if (r.large) {
        fn(FormTag<kLarge>{});
        return;
    }
    float top[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < N; j += 2)
        top[(j >> 1) & 1] = max3_abs(top[(j >> 1) & 1], __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
    // (a NaN is passed over, and comes through every form)
    const float most = hidden ? 0.0f : fmaxf(top[0], top[1]);
    if (!__any_sync(0xffffffffu, most > r.small_limit)) fn(FormTag<kSmall>{});
    else if (!__any_sync(0xffffffffu, most > r.near_limit)) fn(FormTag<kNear>{});
    else fn(FormTag<kAny>{});
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
        // (the powers of a have to be normal numbers, and K^2 p dP)
        r.large = !(p.cap <= kNearCap) || !(r.a >= 1e-5f && r.a <= 1e5f) || !(r.k >= 1e-6f);
        r.near_limit = kNearEnd / r.a;
        r.small_limit = kSmallEnd / r.a;
        const float fit[4] = {kNear0, kNear1, kNear2, kNear3}, small[3] = {kSmall0, kSmall1, kSmall2};
        double power = static_cast<double>(r.k) * r.a;
        for (int i = 0; i < 4 && !r.large; ++i, power *= static_cast<double>(r.a) * r.a) {
            r.near[i] = static_cast<float>(power * fit[i]);
            if (i < 3) r.small[i] = static_cast<float>(power * small[i]);
        }
        r.unit = r.large ? 1.0f : r.k * r.k;
        r.dq_scale = -p.scale / r.unit;
    }
    r.c = p.scale * kLog2;
    r.slopes = p.slopes;
    r.prefix = p.prefix;
    return r;
}

}  // namespace
}  // namespace pvr
