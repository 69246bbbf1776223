// k_quant8.cu -- bf16 rows to e4m3 with a power-of-two scale for each block of
// 128: the input of the 8-bit projection.
//
// A half warp takes a block: 16 lanes of 8 elements.  The largest magnitude
// (integer maxima of the bf16 patterns) fixes the exponent, and the values
// never leave the registers between.  HBM-bound: 3 bytes per element.  A warp
// has four pairs of blocks of one row in flight (one at a time ran at 3.7 TB/s
// for 2048 rows of 3584, four at 4.9, 36 us for 8 ranks; the conversions and
// shuffles then take 0.71 of the issue slots); the warps of a CTA take consecutive rows, so their
// scales, [block][row], share sectors.
#include "sfar_e4m3.cuh"
#include "sfar_kv_args.h"

namespace {
constexpr int kPairs = 4;                       // pairs of blocks a warp has in flight
}

__global__ void __launch_bounds__(256) k_quant8(const __grid_constant__ SfarQuantArgs a)
{
    const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    const int r = blockIdx.z;
    const long long row = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const long long b0 = (long long)blockIdx.y * (2 * kPairs) + half;       // this half warp's first block
    pdl_wait();
    if (row >= a.m)
        return;
    const uint16_t *src = a.x[r] + row * a.ldx + l * 8;
    uint8_t *dst = a.x8[r] + row * a.ldx8 + l * 8;
    uint4 v[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const long long k0 = (b0 + 2 * i) * 128, k = k0 + l * 8;
        v[i] = make_uint4(0, 0, 0, 0);
        if (a.vec && k + 8 <= a.k) {
            v[i] = ld_nc_v4(src + k0);
        } else {
            uint32_t *w = &v[i].x;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < a.k)
                    w[e >> 1] |= (uint32_t)src[k0 + e] << (16 * (e & 1));
        }
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const long long b = b0 + 2 * i, k0 = b * 128, k = k0 + l * 8;
        uint32_t m = sfar_max_half(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(v[i].x & 0x7fff7fffu, v[i].y), v[i].z), v[i].w));
#pragma unroll
        for (int d = 8; d; d >>= 1)
            m = max(m, __shfl_xor_sync(SFAR_FULL, m, d));
        const bool special = m >= 0x7f80u;
        if (__any_sync(SFAR_FULL, special)) {
            uint32_t f = sfar_max_half(__vmaxu2(__vmaxu2(sfar_finite_abs2(v[i].x), sfar_finite_abs2(v[i].y)),
                                                __vmaxu2(sfar_finite_abs2(v[i].z), sfar_finite_abs2(v[i].w))));
#pragma unroll
            for (int d = 8; d; d >>= 1)
                f = max(f, __shfl_xor_sync(SFAR_FULL, f, d));
            m = f;
        }
        const int e = sfar_scale_exponent(m);
        const uint2 q = sfar_quantize8(v[i], sfar_exp2i(-e), special);
        if (b < a.kb) {
            if (l == 0)
                a.sx[r][b * a.m + row] = sfar_exp2i(e);
            if (a.vec && k + 8 <= a.k) {
                st_v2u32(dst + k0, q.x, q.y);
            } else {
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    if (k + n < a.k)
                        dst[k0 + n] = (uint8_t)((n < 4 ? q.x : q.y) >> (8 * (n & 3)));
            }
        }
    }
}

const void *sfar_kernel_quantize() { return (const void *)k_quant8; }
