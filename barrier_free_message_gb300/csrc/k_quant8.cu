// k_quant8.cu -- bf16 rows to e4m3 with a power-of-two scale for each block of
// 128: the input of the 8-bit projection.
//
// A half warp takes a block: 16 lanes of 8 elements.  The largest magnitude
// (integer maxima of the bf16 patterns) fixes the exponent, and the values
// never leave the registers between.  HBM-bound: 3 bytes per element.
// Consecutive warps take consecutive rows, so their scales, [block][row],
// share sectors.
#include "sfar_e4m3.cuh"
#include "sfar_kv_args.h"

__global__ void __launch_bounds__(256) k_quant8(const __grid_constant__ SfarQuantArgs a)
{
    const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    const long long pairs = (a.kb + 1) / 2, units = pairs * a.m;
    const int r = blockIdx.y;
    pdl_wait();
    const uint16_t *x = a.x[r];
    for (long long u = blockIdx.x * 8ll + (threadIdx.x >> 5); u < units; u += gridDim.x * 8ll) {
        const long long row = u % a.m, b = 2 * (u / a.m) + half;
        const long long k0 = b * 128 + l * 8;
        const uint16_t *src = x + row * a.ldx + k0;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (a.vec && k0 + 8 <= a.k) {
            v = ld_nc_v4(src);
        } else {
            uint32_t *w = &v.x;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k0 + e < a.k)
                    w[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
        }
        uint32_t m = sfar_max_half(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(v.x & 0x7fff7fffu, v.y), v.z), v.w));
#pragma unroll
        for (int d = 8; d; d >>= 1)
            m = max(m, __shfl_xor_sync(SFAR_FULL, m, d));
        const bool special = m >= 0x7f80u;
        if (__any_sync(SFAR_FULL, special)) {
            uint32_t f = sfar_max_half(__vmaxu2(__vmaxu2(sfar_finite_abs2(v.x), sfar_finite_abs2(v.y)),
                                                __vmaxu2(sfar_finite_abs2(v.z), sfar_finite_abs2(v.w))));
#pragma unroll
            for (int d = 8; d; d >>= 1)
                f = max(f, __shfl_xor_sync(SFAR_FULL, f, d));
            m = f;
        }
        if (b >= a.kb)
            continue;
        const float scale = sfar_exp2i(sfar_scale_exponent(m));
        if (l == 0)
            a.sx[r][b * a.m + row] = scale;
        const uint2 q = sfar_quantize8(v, SfarInv(scale), special);
        uint8_t *dst = a.x8[r] + row * a.ldx8 + k0;
        if (a.vec && k0 + 8 <= a.k) {
            st_v2u32(dst, q.x, q.y);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k0 + e < a.k)
                    dst[e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
        }
    }
}

const void *sfar_kernel_quantize() { return (const void *)k_quant8; }
