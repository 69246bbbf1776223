// k_kv_attn.cu -- attention of the step's tokens over the paged 8-bit cache,
// one warp for each (rank, token, query head): the definition, read off.
#include "sfar_e4m3.cuh"
#include "sfar_kv_args.h"
#include "sfar_kv_device.cuh"

template <int D>
__global__ void __launch_bounds__(128) k_kv_attn(const __grid_constant__ SfarAttnArgs a)
{
    constexpr int kE = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = blockIdx.x * 4ll + (threadIdx.x >> 5);
    const int r = blockIdx.y;
    pdl_wait();
    if (row >= (long long)a.T * a.Hq)
        return;
    const int t = (int)(row / a.Hq), h = (int)(row % a.Hq), hk = h / a.G;
    uint16_t *dst = a.out[r] + t * a.ots + h * a.ohs + lane * kE;
    float o[kE] = {}, q[kE];
    float top = -INFINITY, sum = 0.f;
    if (t < a.starts[a.B]) {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.starts[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        const int b = lo;
        const uint16_t *src = a.q[r] + t * a.qts + h * a.qhs + lane * kE;
#pragma unroll
        for (int e = 0; e < kE; ++e)
            q[e] = __uint_as_float((uint32_t)src[e] << 16) * a.scale;
        const long long most = min((long long)a.W << a.shift, (long long)INT_MAX);
        long long len = a.lens[b];
        if (len < 0 || len > most) {
            sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_LENGTH);
            len = len < 0 ? 0 : most;
        }
        const long long pos = len - (a.starts[b + 1] - t);
        const long long first = a.window ? max(0ll, pos - a.window + 1) : 0;
        for (long long j = first; j <= pos; ++j) {
            const int p = a.table[(size_t)b * a.W + (j >> a.shift)];
            if ((unsigned)p >= (unsigned)a.pages) {
                sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_PAGE);
                continue;
            }
            const long long page = (long long)p * a.Hk + hk;
            const long long at = ((page << a.shift) + (j & ((1 << a.shift) - 1))) * D + lane * kE;
            float s = 0.f, v[kE];
#pragma unroll
            for (int e = 0; e < kE; e += 2) {
                const float2 kx = e4m3x2_to_float2(*reinterpret_cast<const uint16_t *>(a.k[r] + at + e));
                const float2 vx = e4m3x2_to_float2(*reinterpret_cast<const uint16_t *>(a.v[r] + at + e));
                s += q[e] * kx.x + q[e + 1] * kx.y;
                v[e] = vx.x;
                v[e + 1] = vx.y;
            }
#pragma unroll
            for (int d = 16; d; d >>= 1)
                s += __shfl_xor_sync(SFAR_FULL, s, d);
            s *= a.ks[r][page];
            const float now = fmaxf(top, s), keep = top == -INFINITY ? 0.f : expf(top - now), w = expf(s - now);
            const float wv = w * a.vs[r][page];
            sum = sum * keep + w;
#pragma unroll
            for (int e = 0; e < kE; ++e)
                o[e] = o[e] * keep + wv * v[e];
            top = now;
        }
    }
    const float inv = top == -INFINITY ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < kE; ++e)
        dst[e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * inv));
}

const void *sfar_kernel_kv_attn(int head_dim)
{
    return head_dim == 64 ? (const void *)k_kv_attn<64> : (const void *)k_kv_attn<128>;
}
