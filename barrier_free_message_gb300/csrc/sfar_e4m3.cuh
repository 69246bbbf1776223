// sfar_e4m3.cuh -- e4m3 arithmetic shared by the 8-bit kernels.
//
// e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; no infinities, NaN is
// 0x7f or 0xff, largest finite value 448 = 1.75 * 2^8.
#pragma once
#include <cuda_fp16.h>

#include "sfar_prims.cuh"

// The exponent e of the scale 2^e of values whose largest finite magnitude has
// the bf16 bits `amax` (sign clear): the least e >= -100 with amax <= 448 *
// 2^e.  amax = 1.f * 2^(E - 127), so e = E - 135, and one more if 1.f > 1.75
// (mantissa bits above 0x60).
__device__ __forceinline__ int sfar_scale_exponent(uint32_t amax)
{
    const int e = (int)(amax >> 7) - 135 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
    return e < -100 ? -100 : e;
}
__device__ __forceinline__ float sfar_exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// largest magnitude of two packed bf16 values, per half
__device__ __forceinline__ uint32_t sfar_max_abs2(uint32_t m, uint32_t v) { return __vmaxu2(m, v & 0x7fff7fffu); }

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// two binary32 to two e4m3 (lo in bits 0-7), nearest even, |x| <= 448
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// two e4m3 to two binary16 (exact; NaN stays NaN)
__device__ __forceinline__ uint32_t cvt_f16x2_e4m3(uint32_t v)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t v)
{
    const uint32_t h = cvt_f16x2_e4m3(v);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The binary32 result y of an operation, given what the exact result has beyond it (its sign): of the two binary32 values
// around the exact one, that with an odd significand, so that a second rounding to far fewer bits goes as a single one would.
__device__ __forceinline__ float sfar_to_odd(float y, float beyond)
{
    uint32_t b = __float_as_uint(y);
    if (beyond < 0.f || beyond > 0.f) {
        if ((__float_as_uint(beyond) ^ b) >> 31)
            --b;                           // towards zero: y is beyond the exact result, and so not 0
        b |= 1u;
    }
    return __uint_as_float(b);
}

// How x / scale is formed for a scale: a product with the exact reciprocal of
// a power of two, a division otherwise (a scale > 0 that the caller brought),
// rounded to odd.
struct SfarInv {
    float s, inv;
    bool pow2;
    __device__ __forceinline__ explicit SfarInv(float scale) : s(scale)
    {
        const uint32_t b = __float_as_uint(scale);
        const int e = (int)(b >> 23) - 127;
        pow2 = (b & 0x7fffffu) == 0 && e >= -126 && e <= 126;
        inv = pow2 ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.f;
    }
    __device__ __forceinline__ float operator()(float x) const
    {
        if (pow2)
            return x * inv;
        const float y = __fdiv_rn(x, s);
        return sfar_to_odd(y, fmaf(-y, s, x));
    }
};

__device__ __forceinline__ float sfar_times(float by, float x) { return by * x; }
__device__ __forceinline__ float sfar_times(const SfarInv &by, float x) { return by(x); }
// Eight bf16 (one 16-byte vector) as eight e4m3 of x / scale (by: the scale's
// SfarInv, or the inverse of a power of two); `special`: some value of the
// group is infinite or NaN, and such values become NaN.
template <class By> __device__ __forceinline__ uint2 sfar_quantize8(const uint4 &v, const By &by, bool special)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p[i] = cvt_e4m3x2(sfar_times(by, bf16_lo(w[i])), sfar_times(by, bf16_hi(w[i])));
    if (special) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if ((w[i] & 0x7f80u) == 0x7f80u)
                p[i] = (p[i] & 0xff00u) | 0x7fu;
            if ((w[i] & 0x7f800000u) == 0x7f800000u)
                p[i] = (p[i] & 0x00ffu) | 0x7f00u;
        }
    }
    return make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
}

// Clears the infinities and NaN of two packed bf16 magnitudes.
__device__ __forceinline__ uint32_t sfar_finite_abs2(uint32_t v)
{
    v &= 0x7fff7fffu;
    if ((v & 0x7f80u) == 0x7f80u)
        v &= 0xffff0000u;
    if ((v & 0x7f800000u) == 0x7f800000u)
        v &= 0x0000ffffu;
    return v;
}
__device__ __forceinline__ uint32_t sfar_max_half(uint32_t m) { return max(m & 0xffffu, m >> 16); }
