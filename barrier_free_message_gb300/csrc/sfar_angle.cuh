// sfar_angle.cuh -- cosine and sine of position * frequency.
//
// The angle in turns, n f / (2 pi), is needed modulo 1, so far positions need
// more than binary32: n = 65536 n1 + n0 is exact in two numbers, f / (2 pi) is
// formed as h + l (48 bits), and the products n1 h, n0 h are split without
// error by fma; whole turns leave each part as soon as it is there.  About 25
// binary32 instructions; binary64 would be three, at a rate of two a clock and
// SM.
#pragma once
#include "sfar_prims.cuh"

// n >= 0
__device__ __forceinline__ float sfar_turns(int n, float f)
{
    constexpr float ih = 0.15915494f, il = (float)(0.15915494309189533577 - (double)0.15915494f);
    const float h = f * ih, l = fmaf(f, il, fmaf(f, ih, -h));
    const float n1 = (float)(n & 0x7fff0000), n0 = (float)(n & 0xffff);
    const float a = n1 * h, b = n0 * h, ae = fmaf(n1, h, -a), be = fmaf(n0, h, -b);
    const float far = (ae - rintf(ae)) + fmaf(n1, l, fmaf(n0, l, be));
    const float near = (a - rintf(a)) + (b - rintf(b));
    const float t = (near - rintf(near)) + (far - rintf(far));
    return t - rintf(t);
}
__device__ __forceinline__ float2 sfar_cos_sin(int n, float f)
{
    float2 r;
    sincospif(2.f * sfar_turns(n, f), &r.y, &r.x);
    return r;
}
