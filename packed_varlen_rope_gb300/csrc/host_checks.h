// Host-side argument checks and frequencies shared by the entry points.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <utility>

#include "rope_qk.h"

namespace pvr {

constexpr int kMaxHalf = 128;           // head_dim <= 256
constexpr int64_t kMaxTokens = int64_t(1) << 24;   // positions < 2^24 are exact in fp32

// w_j = RN32( pow(theta, -(2j)/d) / scale ), binary64 until the one rounding; a linear
// position rescale by `scale` (position p acts as p / scale) divides every frequency.
inline void host_inv_freq(double theta, int d, double scale, float *w)
{
    for (int j = 0; j < d / 2; ++j)
        w[j] = static_cast<float>(std::pow(theta, -(2.0 * static_cast<double>(j)) / static_cast<double>(d)) / scale);
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    if (na <= 0 || nb <= 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + static_cast<uintptr_t>(nb) && pb < pa + static_cast<uintptr_t>(na);
}

inline int check_head_dim(int32_t head_dim)
{
    if (head_dim < 16 || head_dim > 2 * kMaxHalf || head_dim % 16 != 0) return ROPE_ERR_HEAD_DIM;
    return ROPE_OK;
}

inline int check_theta(double theta)
{
    if (!(theta > 0.0) || !std::isfinite(theta)) return ROPE_ERR_THETA;
    return ROPE_OK;
}

inline int check_scale(double scale)
{
    if (!(scale > 0.0) || !std::isfinite(scale)) return ROPE_ERR_THETA;
    return ROPE_OK;
}

// A strided bf16 view of `rows` x `heads` blocks of head_dim contiguous elements.
struct View {
    const void *base;
    int64_t rows, heads, ts, hs, d;

    int64_t span_elems() const { return (rows - 1) * ts + (heads - 1) * hs + d; }
    int64_t bytes() const { return span_elems() * 2; }
};

// Distinct (row, head) pairs address disjoint blocks: with the two dimensions sorted by
// stride, the smaller stride covers a block and the larger one covers every block of
// the smaller dimension.  A dimension of extent 1 is ignored.
inline bool view_injective(const View &v)
{
    int64_t s1 = v.ts, n1 = v.rows, s2 = v.hs, n2 = v.heads;
    if (n1 <= 1) { s1 = s2; n1 = n2; s2 = 0; n2 = 1; }
    if (n2 > 1 && s2 < s1) { std::swap(s1, s2); std::swap(n1, n2); }
    if (n1 > 1 && s1 < v.d) return false;
    if (n2 > 1 && s2 < n1 * s1) return false;
    return true;
}

// Two views share no element.  True when their address ranges are disjoint, or when
// both step tokens by the same stride S, each token's block fits in S, and the second
// view's block sits after the first's inside every period of S (the Q and K slices of
// a fused QKV projection output).
inline bool views_disjoint(const View &a, const View &b)
{
    if (!overlap(a.base, a.bytes(), b.base, b.bytes())) return true;
    if (a.rows != b.rows || a.ts != b.ts || a.ts <= 0 || a.rows < 1) return false;
    const int64_t S = a.ts;
    const int64_t ea = (a.heads - 1) * a.hs + a.d;
    const int64_t eb = (b.heads - 1) * b.hs + b.d;
    if (ea > S || eb > S) return false;
    const int64_t delta_bytes = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.base)) -
                                static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.base));
    if (delta_bytes % 2 != 0) return false;
    const int64_t r = ((delta_bytes / 2) % S + S) % S;
    return r >= ea && r + eb <= S;
}

// The view's span in elements, computed without wrapping, stays below 2^56 (so that
// the int64 span, byte counts and overlap tests below cannot overflow).
inline bool span_fits(const View &v)
{
    const __int128 span = static_cast<__int128>(v.rows - 1) * v.ts + static_cast<__int128>(v.heads - 1) * v.hs + v.d;
    return span < (static_cast<__int128>(1) << 56);
}

inline int check_view(const View &v)
{
    if (v.base == nullptr) return ROPE_ERR_NULL;
    if (!aligned(v.base, 16) || v.ts % 8 != 0 || v.hs % 8 != 0) return ROPE_ERR_ALIGN;
    if (v.ts < 0 || v.hs < 0 || !span_fits(v)) return ROPE_ERR_SHAPE;
    if (!view_injective(v)) return ROPE_ERR_OVERLAP;
    return ROPE_OK;
}

// Check word of a cache descriptor: FNV-1a (64-bit) over the bytes of every other
// field, so that a descriptor not written by the build, or changed after it, is caught.
inline uint64_t cache_check_word(const rope_cos_sin_cache &c)
{
    uint64_t h = 1469598103934665603ull;
    auto mix = [&h](const void *p, size_t n) {
        const unsigned char *b = static_cast<const unsigned char *>(p);
        for (size_t i = 0; i < n; ++i) {
            h ^= b[i];
            h *= 1099511628211ull;
        }
    };
    const uintptr_t data = reinterpret_cast<uintptr_t>(c.data);
    mix(&data, sizeof data);
    mix(&c.rows, sizeof c.rows);
    mix(&c.head_dim, sizeof c.head_dim);
    mix(&c.device, sizeof c.device);
    mix(&c.theta, sizeof c.theta);
    mix(&c.position_scale, sizeof c.position_scale);
    return h;
}

// The cache serves this rotation: written by the build, for the same head_dim, theta
// and position_scale, with a table inside the limits the build enforces.
inline int check_cache(const rope_cos_sin_cache *c, int32_t head_dim, double theta, double scale)
{
    if (c == nullptr) return ROPE_OK;
    if (c->check != cache_check_word(*c)) return ROPE_ERR_CACHE;
    if (c->head_dim != head_dim || !(c->theta == theta) || !(c->position_scale == scale)) return ROPE_ERR_CACHE;
    if (c->rows < 0 || c->rows > kMaxTokens || (c->rows > 0 && c->data == nullptr)) return ROPE_ERR_CACHE;
    if (c->data != nullptr && !aligned(c->data, 16)) return ROPE_ERR_ALIGN;
    return ROPE_OK;
}

// A cache with rows is read by kernels of the current device only.
inline int check_cache_device(const rope_cos_sin_cache *c)
{
    if (c == nullptr || c->rows == 0) return ROPE_OK;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ROPE_ERR_LAUNCH;
    return dev == c->device ? ROPE_OK : ROPE_ERR_CACHE;
}

}  // namespace pvr
