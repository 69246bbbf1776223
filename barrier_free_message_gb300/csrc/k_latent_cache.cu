// k_latent_cache.cu -- the paged latent cache written and read back
// (include/sfar_latent.h).
//
// Append: a warp takes a token's row of one rank: latents of 8 or 16 a lane,
// their sum of squares by shuffles, the rotated key's pairs an angle to a lane.
// The row is asked for before its slot is known; 40 registers, so that 48 warps
// are in flight on an SM.  (Rows of two or four ranks to a warp, with the angle
// in common: 30 and 37 us where this takes 26.)
//
// Gather: a warp takes four neighbouring rows, finds the first one's request
// by a search of 32 places at a time and the others from there by steps that
// double, and copies all of them at once.
//
// Both are HBM-bound for prompts (4 bytes an element), latency-bound for a few
// tokens.  Measured, rows of 576: append of 16384 tokens, 4 ranks: 152 MB in 25.6
// us, 0.88 of a copy's rate, of 48 tokens, 8 ranks, 2.6 us; gather of 30000 rows,
// 8 ranks: 622 MB in 91.8 us, the copy's rate, of three short requests 2.6 us.
#include "sfar_angle.cuh"
#include "sfar_kv_device.cuh"
#include "sfar_latent_args.h"
#include "sfar_tc.cuh"

namespace {

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float l, float h)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(h), "f"(l));
    return r;
}

}  // namespace

template <int L>
__global__ void __launch_bounds__(32 * SFAR_LATENT_APPEND_WARPS, 6) k_latent_append(const __grid_constant__ SfarLatentAppendArgs a)
{
    constexpr int kV = L / 256;                    // 16-byte vectors of latents per lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const long long item = (long long)blockIdx.x * SFAR_LATENT_APPEND_WARPS + warp;
    const int t = (int)(item / a.R), r = (int)(item - (long long)t * a.R);
    if (t >= a.T)
        return;
    const int slot = a.slots[t], n = a.pos[t];
    const uint16_t *x = a.x[r] + t * a.ts;
    uint4 v[kV], w[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        v[i] = ld_nc_v4(x + 256 * i + 8 * lane);
        w[i] = ld_nc_v4(a.weight + 256 * i + 8 * lane);
    }
    // the key: pair `lane` of rope / 2
    const int half = a.rope / 2, first = a.inter ? 2 * lane : lane, second = a.inter ? first + 1 : lane + half;
    const bool pair = lane < half;
    uint32_t k = 0;
    float freq = 0.f;
    if (pair) {
        freq = a.freq[lane];
        k = a.inter ? *reinterpret_cast<const uint32_t *>(x + L + first) : x[L + first] | (uint32_t)x[L + second] << 16;
    }
    if (slot < -1 || slot >= a.slot_end) {
        if (lane == 0)
            sfar_kv_fault(a.ctl, t, SFAR_KV_BAD_SLOT);
        return;
    }
    if (slot < 0 || n < 0)
        return;
    const float2 cs = sfar_cos_sin(n, freq);
    uint64_t two = 0;                              // two sums at once
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t y = tc::pack2(lo(u[j]), hi(u[j]));
            two = tc::fma2(y, y, two);
        }
    }
    const float2 both = tc::unpack2(two);
    float s = both.x + both.y;
#pragma unroll
    for (int e = 16; e; e >>= 1)
        s += __shfl_xor_sync(SFAR_FULL, s, e);
    const float by = rsqrtf(fmaf(s, 1.f / L, a.eps));
    const uint64_t by2 = tc::pack2(by, by);
    uint16_t *to = a.cache[r] + (long long)slot * (L + a.rope);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, g[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 z = tc::unpack2(tc::mul2(tc::mul2(tc::pack2(lo(u[j]), hi(u[j])), by2), tc::pack2(lo(g[j]), hi(g[j]))));
            y[j] = pack(z.x, z.y);
        }
        st_v4(to + 256 * i + 8 * lane, make_uint4(y[0], y[1], y[2], y[3]));
    }
    if (pair) {
        const float c = cs.x * a.scale, d = cs.y * a.scale, p = lo(k), q = hi(k);
        const uint32_t y = pack(p * c - q * d, q * c + p * d);
        if (a.inter) {
            *reinterpret_cast<uint32_t *>(to + L + first) = y;
        } else {
            to[L + first] = (uint16_t)y;
            to[L + second] = (uint16_t)(y >> 16);
        }
    }
}

__global__ void __launch_bounds__(32 * SFAR_GATHER_WARPS) k_latent_gather(const __grid_constant__ SfarLatentGatherArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y;
    pdl_wait();
    const long long t0 = ((long long)blockIdx.x * SFAR_GATHER_WARPS + warp) * SFAR_GATHER_ROWS;
    if (t0 >= a.T)
        return;
    // the last request b with starts[b] <= t0, in [at, at + n)
    int at = 0, n = a.B;
    while (n > 1) {
        const int step = (n + 31) / 32, j = at + lane * step;
        const unsigned in = __ballot_sync(SFAR_FULL, lane * step < n && a.starts[j] <= t0);
        const int k = in ? 31 - __clz(in) : 0;
        at += k * step;
        n = min(step, n - k * step);
    }
    // lane i < 4: row t0 + i
    int b = at, slot = -1;
    if (lane < SFAR_GATHER_ROWS && t0 + lane < a.T) {
        const int t = (int)t0 + lane;
        // the last request that begins at or before t: mostly this one or the next, but many may have no rows
        int step = 1;
        for (; b + step < a.B && a.starts[b + step] <= t; step *= 2)
            b += step;
        while (step /= 2)
            if (b + step < a.B && a.starts[b + step] <= t)
                b += step;
        const int from = a.starts[b], to = a.starts[b + 1];
        if (from < 0 || to > a.T || from > to) {
            sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_TOKENS);
        } else if (t >= from && t < to) {
            const int i = t - from;
            if (i >= a.lens[b] || (i >> a.shift) >= a.W) {
                sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_TOKENS);
            } else {
                const int page = a.table[(size_t)b * a.W + (i >> a.shift)];
                if ((unsigned)page >= (unsigned)a.pages)
                    sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_PAGE);
                else
                    slot = (page << a.shift) + (i & ((1 << a.shift) - 1));
            }
        }
    }
    const uint16_t *cache = a.cache[r];
    uint16_t *out = a.out[r] + t0 * a.ots;
    constexpr int kMost = (SFAR_GATHER_ROWS * 72 + 31) / 32;       // rows of up to 576 elements
    uint4 v[kMost];
    int row[kMost], c[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const int i = 32 * k + lane;
        row[k] = i / a.vecs;
        c[k] = i - row[k] * a.vecs;
        const int s = __shfl_sync(SFAR_FULL, slot, row[k] & 31);
        if (row[k] >= SFAR_GATHER_ROWS || s < 0)
            row[k] = -1;
        else
            v[k] = ld_nc_v4(cache + ((long long)s * a.vecs + c[k]) * 8);
    }
#pragma unroll
    for (int k = 0; k < kMost; ++k)
        if (row[k] >= 0)
            st_v4(out + row[k] * a.ots + c[k] * 8, v[k]);
}

const void *sfar_kernel_latent_append(int latent)
{
    return latent == 256 ? (const void *)k_latent_append<256> : (const void *)k_latent_append<512>;
}
const void *sfar_kernel_latent_gather() { return (const void *)k_latent_gather; }
