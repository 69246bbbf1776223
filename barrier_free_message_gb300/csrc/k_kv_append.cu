// k_kv_append.cu -- new keys and values into the paged 8-bit cache.
//
// A run is the new tokens of one page: neighbours in the step with consecutive
// slots.  A team of warps (one, unless a page is long) takes a run of one
// (rank, head, keys or values) plane: the largest magnitude over the run fixes
// the scale's exponent, held tokens of the page are rewritten if it grew, the
// run is quantised and stored.  No two teams share a page's plane, so nothing
// is atomic and the result does not depend on any order.
//
// HBM-bound for prompts (3 bytes per element), latency-bound for a decode step.
// A CTA of 8 warps covers the planes of 8 teams' warps and a window of tokens.
//  many tokens: windows of up to 32 (only one token in a page begins a run, and
//    a CTA per token would spend its time on launches), and as many vectors
//    kept per lane (up to 16) and warps to a team as a whole page needs: a run
//    is read once, and a short page holds no registers it does not use.
//  few tokens: windows of one token, so that a decode step has a warp per token
//    and plane in flight, 8 vectors kept per lane; what a longer run has beyond
//    is read twice, in batches (80 registers, 52 bytes of them spilled: three
//    CTAs per SM).
//
// Measured: 4 ranks of two heads of 128, pages of 32, 9 prompts of 1501 to 2139
// tokens (102 MB) 20.9 us, 4.9 TB/s; 8 ranks, 16 prompts of 500 to 1000: 4.4
// TB/s with pages of 64 and 4.8 with 16 (3.2 and 3.6 with one warp and 16
// vectors for every page); 64 single tokens 2.4 us; 128 single tokens of 8 ranks
// of four heads 6.3 us (in windows of two tokens 8.9).
#include "sfar_e4m3.cuh"
#include "sfar_kv_args.h"
#include "sfar_kv_device.cuh"

namespace {

// Sixteen e4m3, each by `how`.
template <class F> __device__ __forceinline__ uint4 times(uint4 w, F how)
{
    uint32_t *p = &w.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 lo = e4m3x2_to_float2(p[j]), hi = e4m3x2_to_float2(p[j] >> 16);
        p[j] = cvt_e4m3x2(how(lo.x), how(lo.y)) | cvt_e4m3x2(how(hi.x), how(hi.y)) << 16;
    }
    return w;
}
// A run beside a scale that is no power of two (the caller's): what the kernel does with the others, its values read again.
// Held values take products of more than 24 bits, new ones a division, both rounded to odd.  Out of line: inside, its code
// and registers cost a decode step of 64 tokens 0.3 us of 2.4.
template <int D>
__device__ __noinline__ void append_any(const uint16_t *x, long long ts, uint8_t *page, int first, int n, float old, float scale, bool special,
                                        int member, int team)
{
    constexpr int kVec = D / 8, kTok = 32 / kVec;
    const int lane = threadIdx.x & 31;
    if (first && scale > old) {
        const float ratio = __fdiv_rn(old, scale);           // exact: the new scale is a power of two
        uint4 *held = reinterpret_cast<uint4 *>(page);
        for (int i = lane + 32 * member; i < first * (D / 16); i += 32 * team)
            held[i] = times(held[i], [&](float v) { return sfar_to_odd(v * ratio, fmaf(v, ratio, -(v * ratio))); });
    }
    const SfarInv by(scale);
    for (int t = member * kTok + lane / kVec; t < n; t += kTok * team) {
        const uint2 q = sfar_quantize8(ld_nc_v4(x + t * ts + (lane % kVec) * 8), by, special);
        st_v2u32(page + (first + t) * D + (lane % kVec) * 8, q.x, q.y);
    }
}

}  // namespace

// Keep: vectors a lane holds between the maximum and the stores; Team: warps to
// a run; Whole: a page has no more than Keep * Team * 32 vectors.
template <int D, int Keep, int Team, bool Whole>
__global__ void __launch_bounds__(32 * SFAR_APPEND_WARPS, Keep > 8 ? 2 : Whole ? 4 : 3) k_kv_append(const __grid_constant__ SfarKvAppendArgs a)
{
    constexpr int kVec = D / 8;            // 16-byte vectors (8 bf16) of a token
    constexpr int kTok = 32 / kVec;        // tokens one step of a warp covers
    constexpr int kBatch = 8;              // steps in flight beyond those kept
    constexpr int kTeams = SFAR_APPEND_WARPS / Team;
    __shared__ int s_slot[kTeams][32];
    __shared__ uint32_t s_runs[kTeams][6];
    __shared__ uint32_t s_max[2][SFAR_APPEND_WARPS], s_fin[2][SFAR_APPEND_WARPS];       // by the run's parity
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, member = warp % Team;
    const int plane = blockIdx.y * kTeams + warp / Team;
    const int P = 1 << a.shift;
    pdl_wait();
    if (plane >= 2 * a.R * a.H)
        return;
    const int kv = plane & 1, h = (plane >> 1) % a.H, r = (plane >> 1) / a.H;
    auto team_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / Team), "n"(32 * Team) : "memory"); };
    // the largest of the team's warps; one barrier a call, since calls alternate between two places
    auto of_team = [&](uint32_t m, uint32_t (&at)[SFAR_APPEND_WARPS]) {
        m = __reduce_max_sync(SFAR_FULL, m);
        if constexpr (Team > 1) {
            if (lane == 0)
                at[warp] = m;
            team_sync();
#pragma unroll
            for (int i = 0; i < Team; ++i)
                m = max(m, at[warp - member + i]);
        }
        return m;
    };
    // The window's runs: a token begins one if it does not continue its neighbour's page.  A run may go on past the
    // window, by less than a page: bit l of goes[w] says that token 32 w + l of the window and what follows continues
    // the one before it.
    const int t_base = blockIdx.x * a.window;
    const int words = 1 + ((P + 31) >> 5);
    int slot = -1;
    uint32_t goes[5], todo;                // todo: the window's tokens that begin a run
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
        todo = __ballot_sync(SFAR_FULL, lane < a.window && slot >= 0 && !(goes[0] >> lane & 1u));
    }
    if constexpr (Team > 1) {
        // a team goes by what its first warp has read: its barriers meet whatever happens to the slots
        uint32_t *runs = s_runs[warp / Team];
        if (member == 0) {
            s_slot[warp / Team][lane] = slot;
            if (lane == 0) {
#pragma unroll
                for (int w = 0; w < 5; ++w)
                    runs[w] = goes[w];
                runs[5] = todo;
            }
        }
        team_sync();
        slot = s_slot[warp / Team][lane];
#pragma unroll
        for (int w = 0; w < 5; ++w)
            goes[w] = runs[w];
        todo = runs[5];
    }
    const uint16_t *src = a.x[kv][r] + (long long)h * a.hs[kv];
    const long long ts = a.ts[kv];
    uint8_t *cache = a.cache[kv][r];
    float *scales = a.scale[kv][r];
    int parity = 0;
    for (; todo; todo &= todo - 1) {
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
        const int tok = lane / kVec;       // of the step's tokens, this lane's
        const uint16_t *x = src + (long long)(t0 + member * kTok + tok) * ts + (lane % kVec) * 8;
        const long long hop = ts * (kTok * Team);
        auto holds = [&](int i) { return (i * Team + member) * kTok + tok < n; };
        auto load = [&](int i) { return holds(i) ? ld_nc_v4(x + i * hop) : make_uint4(0, 0, 0, 0); };
        const bool longer = !Whole && n > Keep * Team * kTok;
        const long long at = (long long)page * a.H + h;
        const float old = first ? scales[at] : 0.f;
        uint4 keep[Keep];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < Keep; ++i)
            keep[i] = load(i);
#pragma unroll
        for (int i = 0; i < Keep; ++i)
            m = sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(m, keep[i].x), keep[i].y), keep[i].z), keep[i].w);
        // what comes after the kept steps, a batch at a time
        auto rest = [&](auto what) {
            if (longer)
#pragma unroll 1
                for (int i = Keep; i * Team * kTok < n; i += kBatch) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int y = 0; y < kBatch; ++y)
                        v[y] = load(i + y);
#pragma unroll
                    for (int y = 0; y < kBatch; ++y)
                        what(i + y, v[y]);
                }
        };
        rest([&](int, const uint4 &v) { m = sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(m, v.x), v.y), v.z), v.w); });
        parity ^= 1;
        uint32_t amax = of_team(sfar_max_half(m), s_max[parity]);
        const bool special = amax >= 0x7f80u;
        if (special) {                     // infinities and NaN do not count
            m = 0;
            for (int i = 0; i * Team * kTok < n; ++i) {
                const uint4 v = load(i);
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(sfar_finite_abs2(v.x), sfar_finite_abs2(v.y)),
                                         __vmaxu2(sfar_finite_abs2(v.z), sfar_finite_abs2(v.w))));
            }
            amax = of_team(sfar_max_half(m), s_fin[parity]);
        }
        uint8_t *base = cache + (at << a.shift) * D;
        const float scale = fmaxf(old, sfar_exp2i(sfar_scale_exponent(amax)));
        __syncwarp();                      // every lane (with a team, every warp) has read the old one
        if (lane == 0 && member == 0)
            scales[at] = scale;
        const bool grows = first && scale > old;
        const SfarInv by(scale);
        if (!by.pow2 || (grows && !SfarInv(old).pow2)) {
            append_any<D>(src + (long long)t0 * ts, ts, base, first, n, old, scale, special, member, Team);
            continue;
        }
        if (grows) {
            const float ratio = old * by.inv;
            uint4 *held = reinterpret_cast<uint4 *>(base);
#pragma unroll 4
            for (int i = lane + 32 * member; i < first * (D / 16); i += 32 * Team)
                held[i] = times(held[i], [&](float v) { return v * ratio; });
        }
        uint8_t *dst = base + (long long)(first + member * kTok + tok) * D + (lane % kVec) * 8;
        auto one = [&](int i, const uint4 &v) {
            if (holds(i)) {
                const uint2 q = sfar_quantize8(v, by.inv, special);
                st_v2u32(dst + i * (kTok * Team * D), q.x, q.y);
            }
        };
#pragma unroll
        for (int i = 0; i < Keep; ++i)
            one(i, keep[i]);
        rest(one);
    }
}

const void *sfar_kernel_kv_append(int head_dim, int page_tokens, int few, int *team)
{
    *team = 1;
    if (few)
        return head_dim == 64 ? (const void *)k_kv_append<64, 8, 1, false> : (const void *)k_kv_append<128, 8, 1, false>;
    // vectors of a page per lane: 4 to 64
    switch (page_tokens * head_dim / 256) {
    case 4: return (const void *)k_kv_append<64, 4, 1, true>;
    case 8: return head_dim == 64 ? (const void *)k_kv_append<64, 8, 1, true> : (const void *)k_kv_append<128, 8, 1, true>;
    case 16: return head_dim == 64 ? (const void *)k_kv_append<64, 16, 1, true> : (const void *)k_kv_append<128, 16, 1, true>;
    case 32: *team = 2; return head_dim == 64 ? (const void *)k_kv_append<64, 16, 2, true> : (const void *)k_kv_append<128, 16, 2, true>;
    default: *team = 4; return (const void *)k_kv_append<128, 16, 4, true>;
    }
}
