// k_rope.cu -- rotary positions (include/sfar_rope.h).
//
// HBM-bound: every element is read and written once, 6 flops a pair beside it.
// A CTA takes rows of one token, a row a (rank, head): the token's angles
// (rot / 2, shared by all of them) are turned into cosines and sines once, in
// shared memory, while the rows are on their way; a thread takes 8 pairs of
// one row, two or four 16-byte vectors in and out.  A pair's two elements are
// in one thread, so an output may be its input.  Threads do no more than that,
// in 32 registers, so that 64 warps are in flight on an SM (40 registers and 48
// warps: 39 us where this takes 34; several rows to a thread: 45).
//
// Measured: 8 ranks, 5003 tokens, 20 heads and a key of 64 elements in 192,
// bf16: 215 MB in 34.4 us, 6.3 TB/s or 0.92 of a copy's rate; 64 elements side
// by side 0.94, 20012 tokens 0.96.  64 tokens of 8 heads and a key of 128: 3.2 us,
// the latency of position, angles and rows.
#include "sfar_angle.cuh"
#include "sfar_latent_args.h"
#include "sfar_tc.cuh"

namespace {

// 8 elements as they lie, as four binary32 pairs, and back
struct Bf16 {
    using E = uint16_t;
    uint4 x;
    __device__ __forceinline__ void load(const E *p) { x = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ uint64_t pair(int i) const
    {
        const uint32_t w = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
        return tc::pack2u(w << 16, w & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(E *p, const uint64_t (&v)[4])
    {
        const float2 a = tc::unpack2(v[0]), b = tc::unpack2(v[1]), c = tc::unpack2(v[2]), d = tc::unpack2(v[3]);
        st_v4(p, make_uint4(tc::bf16x2(a.x, a.y), tc::bf16x2(b.x, b.y), tc::bf16x2(c.x, c.y), tc::bf16x2(d.x, d.y)));
    }
};
struct Fp32 {
    using E = float;
    uint4 x, y;
    __device__ __forceinline__ void load(const E *p)
    {
        x = reinterpret_cast<const uint4 *>(p)[0];
        y = reinterpret_cast<const uint4 *>(p)[1];
    }
    __device__ __forceinline__ uint64_t pair(int i) const
    {
        return i == 0 ? tc::pack2u(x.x, x.y) : i == 1 ? tc::pack2u(x.z, x.w) : i == 2 ? tc::pack2u(y.x, y.y) : tc::pack2u(y.z, y.w);
    }
    static __device__ __forceinline__ void store(E *p, const uint64_t (&v)[4])
    {
        const float2 a = tc::unpack2(v[0]), b = tc::unpack2(v[1]), c = tc::unpack2(v[2]), d = tc::unpack2(v[3]);
        reinterpret_cast<float4 *>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
        reinterpret_cast<float4 *>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
    }
};

}  // namespace

template <class V, bool Inter> __global__ void __launch_bounds__(SFAR_ROPE_THREADS, 8) k_rope(const __grid_constant__ SfarRopeArgs a)
{
    using E = typename V::E;
    // cosine and sine of each pair, two pairs to 16 bytes, 8 to 80: no two chunks of a quarter-warp meet in a bank
    extern __shared__ __align__(16) unsigned char turn[];
    const int t = blockIdx.x, chunks = a.half / 8, heads = a.H[0] + a.H[1];
    const int row = threadIdx.x / chunks, c = threadIdx.x - row * chunks, at = blockIdx.y * a.span + row;
    const bool mine = row < a.span && at < a.R * heads;
    const int first = Inter ? 16 * c : 8 * c, second = Inter ? 8 : a.half;     // second: from the first vector on
    E *out = nullptr;
    V x, y;
    pdl_wait();
    const int n = a.pos[t];
    if (mine) {
        const int r = at / heads, h = at - r * heads, key = h >= a.H[0], k = h - (key ? a.H[0] : 0);
        const E *in = static_cast<const E *>(a.in[key][r]) + t * a.its[key] + k * a.ihs[key] + first;
        out = static_cast<E *>(a.out[key][r]) + t * a.ots[key] + k * a.ohs[key] + first;
        x.load(in);
        y.load(in + second);
    }
    if (n < 0)
        return;
    for (int k = threadIdx.x; k < a.half; k += blockDim.x) {
        const float2 cs = sfar_cos_sin(n, a.freq[k]);
        *reinterpret_cast<float2 *>(turn + (k >> 3) * 80 + (k & 7) * 8) = make_float2(cs.x * a.scale, cs.y * a.scale);
    }
    __syncthreads();
    if (!mine)
        return;
    uint64_t u[4], v[4];
    const float4 *w = reinterpret_cast<const float4 *>(turn + c * 80);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 z = w[j];                     // pairs 2 j and 2 j + 1
        if (Inter) {
            // four pairs in each vector
            const V &e = j < 2 ? x : y;
            const uint64_t p = e.pair(2 * j & 3), q = e.pair((2 * j & 3) + 1);
            const float2 f = tc::unpack2(p), g = tc::unpack2(q);
            uint64_t(&to)[4] = j < 2 ? u : v;
            to[2 * j & 3] = tc::fma2(tc::pack2(f.y, f.x), tc::pack2(-z.y, z.y), tc::mul2(p, tc::pack2(z.x, z.x)));
            to[(2 * j & 3) + 1] = tc::fma2(tc::pack2(g.y, g.x), tc::pack2(-z.w, z.w), tc::mul2(q, tc::pack2(z.z, z.z)));
        } else {
            const uint64_t p = x.pair(j), q = y.pair(j), cs = tc::pack2(z.x, z.z);
            u[j] = tc::fma2(q, tc::pack2(-z.y, -z.w), tc::mul2(p, cs));
            v[j] = tc::fma2(p, tc::pack2(z.y, z.w), tc::mul2(q, cs));
        }
    }
    V::store(out, u);
    V::store(out + second, v);
}

const void *sfar_kernel_rope(int dt, int interleaved)
{
    if (dt == 0)
        return interleaved ? (const void *)k_rope<Bf16, true> : (const void *)k_rope<Bf16, false>;
    return interleaved ? (const void *)k_rope<Fp32, true> : (const void *)k_rope<Fp32, false>;
}
