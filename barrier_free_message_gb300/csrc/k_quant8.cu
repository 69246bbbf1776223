// k_quant8.cu -- bf16 rows to e4m3 with a power-of-two scale for each block of
// 128: the input of the 8-bit projection.
//
// Eight lanes take a block: two vectors of 8 elements each, so that four blocks
// of a row pass through a warp at a time.  The largest magnitude (integer
// maxima of the bf16 patterns) fixes the exponent, and the values never leave
// the registers between.  HBM-bound: 3 bytes per element; the warps of a CTA
// take consecutive rows, so their scales, [block][row], share sectors.  Measured,
// 8 ranks of 2048 rows of 3584: 30 us, 5.9 TB/s; sixteen lanes to a block and a
// vector each took 36 (twice the shuffles and exponents), one block at a time 48.  Rows of odd
// length: 1024 of 3583, 23 us, 3.8 TB/s; element by element they ran at 1.0.
#include "sfar_e4m3.cuh"
#include "sfar_kv_args.h"

namespace {

constexpr int kGroups = 2;                      // groups of four blocks a warp has in flight

// Eight elements from an address that is a multiple of 2 only, out of the two aligned vectors they lie in.
__device__ __forceinline__ uint4 load_shifted(uintptr_t at)
{
    const uint16_t *base = reinterpret_cast<const uint16_t *>(at & ~(uintptr_t)15);
    const uint4 a = ld_nc_v4(base), b = ld_nc_v4(base + 8);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const uint32_t off = (uint32_t)at & 15u;
    if (off & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i)
            w[i] = w[i + 2];
    }
    if (off & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i)
            w[i] = w[i + 1];
    }
    const uint32_t bits = 8u * (off & 2u);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}

}  // namespace

__global__ void __launch_bounds__(256) k_quant8(const __grid_constant__ SfarQuantArgs a)
{
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int r = blockIdx.z;
    const long long row = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const long long b0 = (long long)blockIdx.y * (4 * kGroups) + (lane >> 3);       // this lane's first block
    pdl_wait();
    if (row >= a.m)
        return;
    const long long k0 = b0 * 128 + l * 8;      // its first element
    const uint16_t *src = a.x[r] + row * a.ldx + k0;
    uint8_t *dst = a.x8[r] + row * a.ldx8 + k0;
    float *sx = a.sx[r] + b0 * a.m + row;
    const bool inside = (blockIdx.y + 1ll) * (512 * kGroups) <= a.k;        // all the warp's blocks are
    uint4 v[kGroups][2];
    if (inside && a.vec) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                v[i][j] = ld_nc_v4(src + 512 * i + 64 * j);
    } else {
        // rows that begin on no 16 bytes: the vectors around eight elements are read whole where both are the tensor's
        const uintptr_t from = (uintptr_t)a.x[r], to = from + 2 * ((a.m - 1) * a.ldx + a.k);
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = 512 * i + 64 * j;
                const uintptr_t here = (uintptr_t)(src + at), base = here & ~(uintptr_t)15;
                v[i][j] = make_uint4(0, 0, 0, 0);
                if (a.vec && k0 + at + 8 <= a.k) {
                    v[i][j] = ld_nc_v4(src + at);
                } else if (k0 + at + 8 <= a.k && base >= from && base + 32 <= to) {
                    v[i][j] = load_shifted(here);
                } else {
                    uint32_t *w = &v[i][j].x;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (k0 + at + e < a.k)
                            w[e >> 1] |= (uint32_t)src[at + e] << (16 * (e & 1));
                }
            }
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            m = sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(m, v[i][j].x), v[i][j].y), v[i][j].z), v[i][j].w);
        m = sfar_max_half(m);
#pragma unroll
        for (int d = 4; d; d >>= 1)
            m = max(m, __shfl_xor_sync(SFAR_FULL, m, d));
        const bool special = m >= 0x7f80u;
        if (__any_sync(SFAR_FULL, special)) {
            uint32_t f = 0;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                f = __vmaxu2(f, __vmaxu2(__vmaxu2(sfar_finite_abs2(v[i][j].x), sfar_finite_abs2(v[i][j].y)),
                                         __vmaxu2(sfar_finite_abs2(v[i][j].z), sfar_finite_abs2(v[i][j].w))));
            f = sfar_max_half(f);
#pragma unroll
            for (int d = 4; d; d >>= 1)
                f = max(f, __shfl_xor_sync(SFAR_FULL, f, d));
            m = f;
        }
        const int e = sfar_scale_exponent(m);
        const float by = sfar_exp2i(-e);
        const bool in = b0 + 4 * i < a.kb;      // the last blocks' lanes stay for the others' shuffles
        if (in && l == 0)
            sx[4 * i * a.m] = sfar_exp2i(e);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = 512 * i + 64 * j;
            const uint2 q = sfar_quantize8(v[i][j], by, special);
            if (a.vec8 && (inside || (in && k0 + at + 8 <= a.k))) {
                st_v2u32(dst + at, q.x, q.y);
            } else {
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    if (k0 + at + n < a.k)
                        dst[at + n] = (uint8_t)((n < 4 ? q.x : q.y) >> (8 * (n & 3)));
            }
        }
    }
}

const void *sfar_kernel_quantize() { return (const void *)k_quant8; }
