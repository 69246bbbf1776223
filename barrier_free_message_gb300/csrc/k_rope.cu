// k_rope.cu -- rotary positions (include/sfar_rope.h).
//
// HBM-bound: every element is read and written once, 6 flops a pair beside it.
// A CTA takes one token: its angles (rot / 2, shared by all heads and ranks)
// are turned into cosines and sines once, in shared memory; then a thread
// takes 8 pairs of one (rank, head) at a time, two or four 16-byte vectors in
// and out.  A pair's two elements are in one thread, so an output may be its
// input.  Few tokens (decode) would leave SMs idle, so a token's work is then
// cut over several CTAs, each with its own table.
#include "sfar_angle.cuh"
#include "sfar_latent_args.h"

namespace {

// 8 elements as binary32
__device__ __forceinline__ void load8(float (&v)[8], const uint16_t *p)
{
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(float (&v)[8], const float *p)
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8])
{
    st_v4(p, make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7])));
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace

template <class E, bool Inter> __global__ void __launch_bounds__(SFAR_ROPE_THREADS) k_rope(const __grid_constant__ SfarRopeArgs a)
{
    extern __shared__ float2 turn[];               // [half]
    pdl_wait();
    const int t = blockIdx.x, n = a.pos[t];
    if (n < 0)
        return;
    for (int i = threadIdx.x; i < a.half; i += SFAR_ROPE_THREADS) {
        const float2 cs = sfar_cos_sin(n, a.freq[i]);
        turn[i] = make_float2(cs.x * a.scale, cs.y * a.scale);
    }
    __syncthreads();
    // items: (rank, query or key head, 8 pairs), the pairs first
    const int chunks = a.half / 8, heads = a.H[0] + a.H[1], all = a.R * heads * chunks;
    const int end = min(all, (int)(blockIdx.y + 1) * a.span);
    for (int i = blockIdx.y * a.span + threadIdx.x; i < end; i += SFAR_ROPE_THREADS) {
        const int row = i / chunks, c = i - row * chunks, r = row / heads, head = row - r * heads;
        const int key = head >= a.H[0], h = head - (key ? a.H[0] : 0);
        const E *in = static_cast<const E *>(a.in[key][r]) + t * a.its[key] + h * a.ihs[key];
        E *out = static_cast<E *>(a.out[key][r]) + t * a.ots[key] + h * a.ohs[key];
        const int first = Inter ? 16 * c : 8 * c, second = Inter ? first + 8 : first + a.half;
        float x[8], y[8], u[8], v[8];
        load8(x, in + first);
        load8(y, in + second);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 cs = turn[8 * c + j];
            if (Inter) {
                const float p = j < 4 ? x[2 * j & 7] : y[2 * j & 7], q = j < 4 ? x[(2 * j + 1) & 7] : y[(2 * j + 1) & 7];
                float(&to)[8] = j < 4 ? u : v;
                to[2 * j & 7] = p * cs.x - q * cs.y;
                to[(2 * j + 1) & 7] = q * cs.x + p * cs.y;
            } else {
                u[j] = x[j] * cs.x - y[j] * cs.y;
                v[j] = y[j] * cs.x + x[j] * cs.y;
            }
        }
        store8(out + first, u);
        store8(out + second, v);
    }
}

const void *sfar_kernel_rope(int dt, int interleaved)
{
    if (dt == 0)
        return interleaved ? (const void *)k_rope<uint16_t, true> : (const void *)k_rope<uint16_t, false>;
    return interleaved ? (const void *)k_rope<float, true> : (const void *)k_rope<float, false>;
}
