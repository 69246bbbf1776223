// k_kv_append.cu -- new keys and values into the paged 8-bit cache.
//
// A run is the new tokens of one page: neighbours in the step with
// consecutive slots.  One warp takes a run of one (rank, head, keys or values)
// plane: the largest magnitude over the run fixes the scale's exponent, held
// tokens of the page are rewritten if it grew, the run is quantised and
// stored.  No two warps share a page's plane, so nothing is atomic and the
// result does not depend on any order.  The first 16 vectors a lane loads
// (all of a run of up to 32 tokens of 128) stay in registers between the
// maximum and the stores; longer runs read the rest again, from L2.
//
// HBM-bound for prompts (3 bytes per element), latency-bound for a decode
// step.  A CTA of 8 warps covers 8 planes of a window of tokens: single
// tokens when there are few (a decode step then has 8 warps per token and
// plane group in flight), up to 32 for prompts, where only one token in a
// page begins a run and a CTA per token would spend its time on launches.
// Measured: 4 ranks of two heads of 128, 9 prompts of 1501 to 2139 tokens (102
// MB) 21 us, 4.8 TB/s; 8 ranks of one head, 64 single tokens 2.7 us.
#include "sfar_e4m3.cuh"
#include "sfar_kv_args.h"
#include "sfar_kv_device.cuh"

template <int D>
__global__ void __launch_bounds__(32 * SFAR_APPEND_WARPS) k_kv_append(const __grid_constant__ SfarKvAppendArgs a)
{
    constexpr int kVec = D / 8;            // 16-byte vectors (8 bf16) of a token
    constexpr int kTok = 32 / kVec;        // tokens one step of the warp covers
    constexpr int kKeep = 16;              // vectors a lane keeps in registers
    const int lane = threadIdx.x & 31;
    const int plane = blockIdx.y * SFAR_APPEND_WARPS + (threadIdx.x >> 5);
    const int P = 1 << a.shift;
    pdl_wait();
    if (plane >= 2 * a.R * a.H)
        return;
    const int kv = plane & 1, h = (plane >> 1) % a.H, r = (plane >> 1) / a.H;

    // The window's runs: a token begins one if it does not continue its neighbour's page.  A run may go on past the
    // window, by less than a page: bit l of goes[w] says that token 32 w + l of the window and what follows continues
    // the one before it.
    const int t_base = blockIdx.x * a.window;
    const int words = 1 + ((P + 31) >> 5);
    int slot = -1;
    bool leads = false;
    uint32_t goes[5];
    {
        int s[5], before[5];
#pragma unroll
        for (int w = 0; w < 5; ++w) {
            const int t = t_base + 32 * w + lane;
            const bool in = w < words && t >= t_base && t < a.T;
            s[w] = in ? a.slots[t] : -1;
            before[w] = in && t > 0 ? a.slots[t - 1] : -1;
        }
        slot = s[0];
        if (lane < a.window && t_base + lane < a.T && (slot < -1 || (slot >= 0 && (slot >> a.shift) >= a.pages))) {
            sfar_kv_fault(a.ctl, t_base + lane, SFAR_KV_BAD_SLOT);
            slot = -1;
        }
#pragma unroll
        for (int w = 0; w < 5; ++w)
            goes[w] = __ballot_sync(SFAR_FULL, s[w] >= 0 && s[w] == before[w] + 1 && (s[w] & (P - 1)) != 0 && before[w] >= 0);
        leads = lane < a.window && slot >= 0 && !(goes[0] >> lane & 1u);
    }
    const uint16_t *src = a.x[kv][r] + (long long)h * a.hs[kv];
    const long long ts = a.ts[kv];
    uint8_t *cache = a.cache[kv][r];
    float *scales = a.scale[kv][r];
    for (unsigned todo = __ballot_sync(SFAR_FULL, leads); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1;
        const int t0 = t_base + from;
        const int s0 = __shfl_sync(SFAR_FULL, slot, from);
        const int page = s0 >> a.shift, first = s0 & (P - 1);
        int n = 1;                         // the run's tokens: at most what is left of the page
#pragma unroll
        for (int w = 0; w < 5; ++w) {
            // places of word w after `from` that end the run
            const uint32_t after = w ? SFAR_FULL : from == 31 ? 0u : SFAR_FULL << (from + 1);
            const uint32_t end = ~goes[w] & after;
            if (end) {
                n = 32 * w + __ffs(end) - 1 - from;
                break;
            }
        }
        const uint16_t *x = src + (long long)t0 * ts + (lane % kVec) * 8;
        const int tok = lane / kVec;       // of the step's tokens, this lane's
        auto load = [&](int step) { return ld_nc_v4(x + (long long)(step * kTok + tok) * ts); };
        uint4 keep[kKeep];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            if (i * kTok + tok < n)
                keep[i] = load(i);
            else
                keep[i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            m = sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(m, keep[i].x), keep[i].y), keep[i].z), keep[i].w);
        for (int i = kKeep; i * kTok + tok < n; ++i) {
            const uint4 v = load(i);
            m = sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(m, v.x), v.y), v.z), v.w);
        }
        uint32_t amax = __reduce_max_sync(SFAR_FULL, sfar_max_half(m));
        const bool special = amax >= 0x7f80u;
        if (special) {                     // infinities and NaN do not count
            m = 0;
            for (int i = 0; i * kTok + tok < n; ++i) {
                const uint4 v = load(i);
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(sfar_finite_abs2(v.x), sfar_finite_abs2(v.y)),
                                         __vmaxu2(sfar_finite_abs2(v.z), sfar_finite_abs2(v.w))));
            }
            amax = __reduce_max_sync(SFAR_FULL, sfar_max_half(m));
        }
        const long long at = (long long)page * a.H + h;
        uint8_t *base = cache + (at << a.shift) * D;
        const float old = first ? scales[at] : 0.f;
        const float scale = fmaxf(old, sfar_exp2i(sfar_scale_exponent(amax)));
        __syncwarp();
        if (lane == 0)
            scales[at] = scale;
        if (first && scale > old) {
            const float ratio = __fdiv_rn(old, scale);
            uint4 *held = reinterpret_cast<uint4 *>(base);
#pragma unroll 4
            for (int i = lane; i < first * (D / 16); i += 32) {
                uint4 w = held[i];
                uint32_t *p = &w.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 lo = e4m3x2_to_float2(p[j]), hi = e4m3x2_to_float2(p[j] >> 16);
                    p[j] = cvt_e4m3x2(lo.x * ratio, lo.y * ratio) | cvt_e4m3x2(hi.x * ratio, hi.y * ratio) << 16;
                }
                held[i] = w;
            }
        }
        const SfarInv by(scale);
        uint8_t *dst = base + (long long)(first + tok) * D + (lane % kVec) * 8;
        auto store = [&](auto how) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (i * kTok + tok < n) {
                    const uint2 q = sfar_quantize8(keep[i], how, special);
                    st_v2u32(dst + i * kTok * D, q.x, q.y);
                }
            for (int i = kKeep; i * kTok + tok < n; ++i) {
                const uint2 q = sfar_quantize8(load(i), how, special);
                st_v2u32(dst + i * kTok * D, q.x, q.y);
            }
        };
        if (by.pow2)
            store(by.inv);
        else
            store(by);
    }
}

const void *sfar_kernel_kv_append(int head_dim)
{
    return head_dim == 64 ? (const void *)k_kv_append<64> : (const void *)k_kv_append<128>;
}
