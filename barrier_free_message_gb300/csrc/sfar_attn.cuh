// sfar_attn.cuh -- what the attention kernels share.  A: a kernel's parameters.
#pragma once
#include "sfar_kv_args.h"
#include "sfar_kv_device.cuh"
#include "sfar_tc.cuh"

constexpr float kNoScale = 0x1p-100f;  // value scales up to it count as 0: what the append gives to a page of zeros
// log2 by which a score may pass its running reference.  The weights' reference stands 2^kAttnDeep lower: in binary16 they
// reach 2^15.9 (65504 is the most), keep all their bits down to 2^-22 of a row's largest and some down to 2^-33.  A row moves
// its reference for itself, so moves add up over the rows of a warp: three prompt chunks take 4% more with 6 and 9, 0.7% less
// with 8.9 and 7.
constexpr float kAttnLift = 7.9f, kAttnDeep = 8.f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// a / b for a >= 0, b > 0, in 32 bits where they fit (a 64-bit division takes some hundred instructions)
__device__ __forceinline__ long long sfar_div(long long a, long long b)
{
    return (a | b) >> 32 == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
// The first token that position `pos` attends to (below 0: a row of nothing, for which a window near 2^31 would wrap).
__device__ __forceinline__ int sfar_attn_from(const SfarAttnArgs &a, int pos)
{
    return a.window ? max(0, max(pos, -1) - a.window + 1) : 0;
}
// Request b: its context, how many new tokens it has and the row of the first.
template <class A> __device__ __forceinline__ void sfar_attn_request(const A &a, int b, int &len, int &count, int &first)
{
    const long long most = min((long long)a.W << a.shift, (long long)INT_MAX - 1024);
    len = (int)max(0ll, min((long long)a.lens[b], most));
    const int s = a.starts[b], e = a.starts[b + 1];
    first = s;
    count = s < 0 || e < s || e > a.T ? 0 : e - s;
}
// Records what sfar_attn_request had to correct.
template <class A> __device__ __forceinline__ void sfar_attn_check(const A &a, int b, int len, int count, int first)
{
    if (a.lens[b] != len)
        sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_LENGTH);
    if (first < 0 || a.starts[b + 1] - first != count)
        sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_TOKENS);
}
// Offsets in no order can give the requests more row tiles together than the
// step has (and the line more units than its 32-bit sums hold, which the host
// bounds for a step's): nothing is computed then.
template <class A> __device__ __forceinline__ bool sfar_attn_many(const A &a, long long row_tiles)
{
    if (row_tiles > a.most && blockIdx.x == 0 && threadIdx.x == 0)
        sfar_kv_fault(a.ctl, a.B, SFAR_KV_BAD_TOKENS);
    return row_tiles > a.most;
}
// Zeros for the rows past the last request, by the whole grid; this thread is
// `thread` of the `threads` that its CTA has for it (or of fewer than another's).
template <int D, class A> __device__ __forceinline__ void sfar_attn_padding(const A &a, int thread, int threads)
{
    const long long rows = (long long)(a.T - max(0, min(a.starts[a.B], a.T))) * a.Hq * a.R;
    for (long long i = blockIdx.x + (long long)thread * gridDim.x; i < rows; i += (long long)gridDim.x * threads) {
        const int h = (int)(i % a.Hq), r = (int)(i / a.Hq % a.R);
        uint16_t *dst = a.out[r] + (a.T - 1 - i / a.Hq / a.R) * a.ots + h * a.ohs;
        for (int e = 0; e < D; e += 8)
            st_v4(dst + e, make_uint4(0, 0, 0, 0));
    }
}

// Parts of a row's softmax, joined: the references first, then the parts in
// their order.  o = sum of weights * values, relative to 2^wtop; sum relative
// to 2^top.
template <int E> struct SfarAttnState {
    float top = -INFINITY, wtop = -INFINITY, sum = 0.f, o[E] = {};
    __device__ __forceinline__ void reference(float t, float w)
    {
        top = fmaxf(top, t);
        wtop = fmaxf(wtop, w);
    }
    // adds a part's sum; returns what its o is to be multiplied by
    __device__ __forceinline__ float add(float t, float s, float w)
    {
        sum += t == -INFINITY ? s : ex2(t - top) * s;         // s is 0 then, or NaN
        return w == -INFINITY ? 1.f : ex2(w - wtop);          // o is 0 then, or NaN
    }
    __device__ __forceinline__ void add4(int e, float by, const float4 &v)
    {
        o[e] += by * v.x;
        o[e + 1] += by * v.y;
        o[e + 2] += by * v.z;
        o[e + 3] += by * v.w;
    }
    // 0 for a row that attends to nothing
    __device__ __forceinline__ float factor() const
    {
        return sum == 0.f ? 0.f : wtop == -INFINITY ? 1.f / sum : ex2(wtop - top) / sum;
    }
};

// How the parts of a row tile that lies in CTAs c0 .. c1 are joined: always in
// the order of the CTAs, by whichever of them comes last -- of a group of
// `radix` neighbours, which leaves its result in the place of its first, and
// then of the groups (one CTA would read 76 parts of 16 rows for 40 us; two
// levels of 9 take 5).  Up to `flat` parts are one group.
struct SfarJoin {
    int c0, c1;
    int lo, hi, step;               // parts lo, lo + step .. hi are joined next
    int *counter;                   // of those that have come
    template <class A> __device__ __forceinline__ SfarJoin(const A &a, int kind, int first, int last, int me, int flat = 8) : c0(first), c1(last)
    {
        // three sets of counters: of groups that begin a row tile, of others (their first CTA begins no other row
        // tile's second group), of the groups of a row tile; index: the first CTA
        int *set = a.arrived + kind * 3 * a.arrived_stride;
        const int parts = c1 - c0 + 1;
        lo = c0, hi = c1, step = 1, counter = set + c0;
        if (parts > flat) {
            const int radix = max(8, (int)ceilf(sqrtf((float)parts)));
            lo = c0 + (me - c0) / radix * radix;
            hi = min(lo + radix - 1, c1);
            counter = lo == c0 ? set + a.arrived_stride + c0 : set + 2 * a.arrived_stride + lo;
            up = radix;
        }
    }
    int up = 0;                     // the groups' size, if there are groups to join after these
    // by one thread, after the CTA's writes: whether this CTA is the last
    __device__ __forceinline__ bool last() const
    {
        const int all = (hi - lo) / step;
        int come;                   // releases all the CTA's writes: a barrier has ordered them before it
        asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(come) : "l"(counter), "r"(all) : "memory");
        return come == all;         // the last has set the counter back to 0, for the next call
    }
    // on to the groups; false: these were all
    template <class A> __device__ __forceinline__ bool next(const A &a, int kind)
    {
        if (!up)
            return false;
        lo = c0, hi = c0 + (c1 - c0) / up * up, step = up, up = 0;
        counter = a.arrived + kind * 3 * a.arrived_stride + c0;
        return true;
    }
};
