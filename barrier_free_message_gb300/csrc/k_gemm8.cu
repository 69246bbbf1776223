// k_gemm8.cu -- the e4m3 row-parallel projection of several tokens, with a
// scale for each block of 128: a tile of 16 tokens x 64 outputs per CTA,
// operands widened to binary32 in shared memory.
#include "sfar_e4m3.cuh"
#include "sfar_kv_args.h"

__global__ void __launch_bounds__(256) k_gemm8(const __grid_constant__ SfarGemm8Args a)
{
    constexpr int TM = 16, TN = 64, TK = 32;
    __shared__ float xs[TM][TK + 1], ws[TN][TK + 1];
    const int tid = threadIdx.x, r = blockIdx.z;
    const long long m0 = (long long)blockIdx.y * TM, n0 = (long long)blockIdx.x * TN;
    const int i = tid >> 4, j = tid & 15;
    const long long kb = (a.k + 127) / 128;
    pdl_wait();
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    for (long long b = 0; b < kb; ++b) {
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        for (long long k0 = b * 128; k0 < b * 128 + 128 && k0 < a.k; k0 += TK) {
            __syncthreads();
            for (int e = tid; e < (TM + TN) * TK; e += 256) {
                const int row = e / TK, c = e % TK;
                const bool is_x = row < TM;
                const long long at = is_x ? m0 + row : n0 + row - TM;
                float v = 0.f;
                if (k0 + c < a.k && at < (is_x ? a.m : a.n))
                    v = e4m3x2_to_float2(is_x ? a.x8[r][at * a.ldx + k0 + c] : a.w8[r][at * a.ldw + k0 + c]).x;
                (is_x ? xs[row] : ws[row - TM])[c] = v;
            }
            __syncthreads();
#pragma unroll 8
            for (int c = 0; c < TK; ++c)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    part[u] = fmaf(xs[i][c], ws[j + 16 * u][c], part[u]);
        }
        if (m0 + i < a.m)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const long long n = n0 + j + 16 * u;
                if (n < a.n)
                    y[u] = fmaf(part[u], a.sx[r][b * a.m + m0 + i] * a.sw[r][(n / 128) * kb + b], y[u]);
            }
    }
    if (m0 + i < a.m)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long n = n0 + j + 16 * u;
            if (n < a.n)
                a.y[r][(m0 + i) * a.n + n] = __bfloat16_as_ushort(__float2bfloat16_rn(y[u]));
        }
}

const void *sfar_kernel_gemm8() { return (const void *)k_gemm8; }
