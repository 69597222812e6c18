// The rotation's device arithmetic for kernels beside the rotation kernel (rope_qk.cu has
// its own): cos and sin of a position, streaming loads, and the rotation of two bf16
// pairs.  Step for step the same binary32 operations, so the results carry the same bits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cos_sin.cuh"

namespace pvr {

// (cos phi, sin phi) of a binary32 angle in binary64, each rounded once to binary32.
static __device__ __noinline__ float2 cos_sin_binary64(float phi)
{
    double s, c;
    sincos(static_cast<double>(phi), &s, &c);
    return make_float2(__double2float_rn(c), __double2float_rn(s));
}

// (cos phi, sin phi) with phi = RN32(pos * w): the angle is one binary32 multiply; the
// cosine and sine are the binary64 values rounded once to binary32, obtained in
// binary32 double-float arithmetic where its rounding is certain (all but a few cases
// in a million) and in binary64 otherwise.
__device__ __forceinline__ float2 cos_sin_of(float phi)
{
    float c, s;
    if (cos_sin_binary32(phi, c, s)) return make_float2(c, s);
    return cos_sin_binary64(phi);
}

__device__ __forceinline__ float2 cos_sin_at(int pos, float w)
{
    return cos_sin_of(__fmul_rn(__int2float_rn(pos), w));
}

__device__ __forceinline__ uint4 load_stream(const __nv_bfloat16 *p)
{
    return __ldcs(reinterpret_cast<const uint4 *>(p));
}

__device__ __forceinline__ uint32_t bf162_bits(__nv_bfloat162 v)
{
    return *reinterpret_cast<uint32_t *>(&v);
}

__device__ __forceinline__ __nv_bfloat162 bits_bf162(uint32_t u)
{
    return *reinterpret_cast<__nv_bfloat162 *>(&u);
}

// Rotate two bf16 pairs: a = first-half elements, b = second-half elements, with
// (c0, s0, c1, s1) for the two frequencies.  lo' = a*c - b*s, hi' = b*c + a*s.
__device__ __forceinline__ void rotate2(uint32_t &lo, uint32_t &hi, float4 cs)
{
    const __nv_bfloat162 a = bits_bf162(lo);
    const __nv_bfloat162 b = bits_bf162(hi);
    const float a0 = __low2float(a), a1 = __high2float(a);
    const float b0 = __low2float(b), b1 = __high2float(b);
    const float y0 = __fsub_rn(__fmul_rn(a0, cs.x), __fmul_rn(b0, cs.y));
    const float z0 = __fadd_rn(__fmul_rn(b0, cs.x), __fmul_rn(a0, cs.y));
    const float y1 = __fsub_rn(__fmul_rn(a1, cs.z), __fmul_rn(b1, cs.w));
    const float z1 = __fadd_rn(__fmul_rn(b1, cs.z), __fmul_rn(a1, cs.w));
    lo = bf162_bits(__floats2bfloat162_rn(y0, y1));
    hi = bf162_bits(__floats2bfloat162_rn(z0, z1));
}

}  // namespace pvr
