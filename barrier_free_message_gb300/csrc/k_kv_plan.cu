// k_kv_plan.cu -- block tables, slot map and token offsets of a step, built on
// the GPU from the requests' lengths.
//
// Request b goes from len to len' = max(0, len + delta) tokens and so from
// have = ceil(len / P) to want = ceil(len' / P) pages.  Three exclusive sums
// over the requests place everything: of the pages that are lacking (where in
// the ring of free pages a request's begin), of the pages given back (where
// behind the free ones they go) and of the new tokens (the rows of the step).
// Free pages leave the ring at its head and return behind its tail, so what
// is read and what is written never meet, in whatever order the CTAs work.
//
// Latency-bound: a few KB.  One launch of one cluster; every CTA forms the
// sums over all requests itself (they fit its shared memory), so that the
// CTAs exchange nothing, and takes its share of the outputs.  The one cluster
// barrier, between the reads of the lengths and the ring's state and the
// writes of the new ones, lets both be updated in place.  Measured: 256
// requests of one new token each 3.3 us (4.7 with four slots to every thread),
// 2039 requests of mixed changes (0 to 61 new tokens, every 7th leaving) 9.6.
#include <cooperative_groups.h>

#include "sfar_kv_args.h"
#include "sfar_prims.cuh"
#include "sfar_kv_device.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kMostWarps = SFAR_PLAN_THREADS / 32;

struct Sums {
    long long need, back, count;
};

__device__ __forceinline__ long long up(long long v, int shift) { return (v + (1ll << shift) - 1) >> shift; }

__device__ __forceinline__ void warp_scan(Sums &v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long a = __shfl_up_sync(SFAR_FULL, v.need, d), b = __shfl_up_sync(SFAR_FULL, v.back, d),
                        c = __shfl_up_sync(SFAR_FULL, v.count, d);
        if (lane >= d) {
            v.need += a;
            v.back += b;
            v.count += c;
        }
    }
}
// inclusive sums over the CTA's threads, on top of *carry, which goes on to include them
__device__ __forceinline__ Sums block_scan(Sums v, Sums *carry, Sums *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
    warp_scan(v);
    if (lane == 31)
        warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        Sums s = {0, 0, 0};
        if (lane < warps)
            s = warp_sums[lane];
        warp_scan(s);
        if (lane < warps)
            warp_sums[lane] = s;
    }
    __syncthreads();
    Sums before = *carry;
    if (warp > 0) {
        const Sums s = warp_sums[warp - 1];
        before = {before.need + s.need, before.back + s.back, before.count + s.count};
    }
    const Sums all = warp_sums[warps - 1];
    *carry = {carry->need + all.need, carry->back + all.back, carry->count + all.count};
    __syncthreads();
    return {v.need + before.need, v.back + before.back, v.count + before.count};
}

}  // namespace

__global__ void __launch_bounds__(SFAR_PLAN_THREADS) k_kv_plan(const __grid_constant__ SfarKvPlanArgs a)
{
    extern __shared__ int mem[];
    int *s_start = mem;                     // [B + 1] first row of a request's new tokens, at most T
    int *s_len = s_start + a.B + 1;         // [B] tokens held before
    int *s_new = s_len + a.B;               // [B] tokens held after (before, if refused)
    int *s_off = s_new + a.B;               // [B] ring offset of its pages taken or given back; -1 refused
    __shared__ Sums warp_sums[kMostWarps];
    __shared__ int s_used;
    const int tid = threadIdx.x, lane = tid & 31, kThreads = blockDim.x;
    const int shift = a.shift;
    const int crank = blockIdx.x, csize = gridDim.x;
    if (tid == 0)
        s_used = 0;
    pdl_wait();

    int head = a.state[0], freec = a.state[1];
    if (head < 0 || head >= a.pages || freec < 0 || freec > a.pages) {
        if (tid == 0 && crank == 0)
            sfar_kv_fault(a.ctl, 0, SFAR_KV_BAD_RING);
        head = 0;
        freec = 0;
    }
    const long long most = min((long long)a.W << shift, (long long)INT_MAX);
    Sums carry = {0, 0, 0};
    int next_len = 0, next_d = 0;          // of the round after, read while this one's sums are formed
    if (tid < a.B) {
        next_len = a.lens[tid];
        next_d = a.delta[tid];
    }
    for (int base = 0; base < a.B; base += kThreads) {
        const int i = base + tid;
        long long len = next_len, after = 0;
        int d = next_d;
        if (i + kThreads < a.B) {
            next_len = a.lens[i + kThreads];
            next_d = a.delta[i + kThreads];
        }
        Sums v = {0, 0, 0};
        bool fits = true;
        if (i < a.B) {
            if (len < 0 || len > most) {
                if (crank == 0)
                    sfar_kv_fault(a.ctl, i, SFAR_KV_BAD_LENGTH);
                len = len < 0 ? 0 : most;
            }
            after = max(0ll, len + d);
            const long long have = up(len, shift), want = up(after, shift);
            fits = after <= most;
            v.need = d > 0 && fits ? want - have : 0;
            v.back = d < 0 ? have - want : 0;
            v.count = max(d, 0);
        }
        const Sums t = block_scan(v, &carry, warp_sums);
        const bool ok = d <= 0 || (fits && (v.need == 0 || t.need <= freec));
        const int upto = ok && v.need > 0 ? (int)t.need : 0;
        const int best = __reduce_max_sync(SFAR_FULL, upto);
        if (lane == 0 && best > 0)
            atomicMax(&s_used, best);
        if (i < a.B) {
            s_start[i] = (int)min(t.count - v.count, (long long)a.T);
            s_len[i] = (int)len;
            s_new[i] = (int)(ok ? after : len);
            s_off[i] = !ok ? -1 : v.need > 0 ? (int)(t.need - v.need) : (int)min(t.back - v.back, (long long)a.pages);
        }
    }
    if (tid == 0) {
        s_start[a.B] = (int)min(carry.count, (long long)a.T);
        if (crank == 0 && carry.count > a.T)
            sfar_kv_fault(a.ctl, a.B, SFAR_KV_BAD_TOKENS);
    }
    // every CTA has read the lengths and the state; from here on they may change
    cg::this_cluster().sync();

    const int used = s_used;
    const unsigned pages = (unsigned)a.pages;
    auto ring_at = [&](unsigned i) {       // the free page i places behind the head
        unsigned p = (unsigned)head + i;
        return p >= pages ? p - pages : p;
    };
    for (int i = crank * kThreads + tid; i < a.B; i += csize * kThreads) {
        a.lens_out[i] = s_new[i];
        a.taken[i] = s_off[i] >= 0;
        a.starts[i] = s_start[i];
    }
    if (crank == 0 && tid == 0) {
        a.starts[a.B] = s_start[a.B];
        const int held = a.pages - freec;       // the ring has room for no more, whatever is taken
        if (carry.back > held)
            sfar_kv_fault(a.ctl, 0, SFAR_KV_BAD_RING);
        a.state_out[0] = (int)ring_at((unsigned)used);
        a.state_out[1] = freec - used + (int)min(carry.back, (long long)held);
    }
    // Table entries of new pages, ring entries of pages given back: a few lanes per request (most gain a page or none, a
    // large step has ones that leave with many), four pages in flight.
    const int share = kThreads > 256 ? 8 : 4;
    const int part = tid % share;
    for (int b = (crank * kThreads + tid) / share; b < a.B; b += csize * kThreads / share) {
        const int off = s_off[b];
        if (off < 0)
            continue;
        const int have = (int)up(s_len[b], shift), want = (int)up(s_new[b], shift);
        int *row = a.table + (size_t)b * a.W;
        for (int j = have + part; j < want; j += share) {
            int p = a.ring[ring_at((unsigned)(off + j - have))];
            if ((unsigned)p >= pages) {
                sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_PAGE);
                p = -1;
            }
            row[j] = p;
        }
        for (int j0 = want + part; j0 < have; j0 += 4 * share) {
            int p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p[i] = j0 + i * share < have ? row[j0 + i * share] : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long at = (long long)off + j0 + i * share - want;
                if (j0 + i * share >= have || at >= (long long)a.pages - freec)
                    continue;               // more than the pool has: recorded above, and not counted
                if ((unsigned)p[i] >= pages) {
                    sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_PAGE);
                    p[i] = -1;              // its place holds no page
                }
                unsigned to = (unsigned)head + (unsigned)freec;
                to = (to >= pages ? to - pages : to) + (unsigned)at;
                a.ring[to >= pages ? to - pages : to] = p[i];
            }
        }
    }
    // Slots: a thread finds its first token's request and walks on from there, over one token if all can be taken at
    // once, else four.  The last CTA begins: with few requests and tokens others have the table.
    const int total = s_start[a.B], per = a.T <= csize * kThreads ? 1 : 4;
    for (long long t0 = (long long)per * ((csize - 1 - crank) * kThreads + tid); t0 < a.T; t0 += (long long)per * csize * kThreads) {
        int out[4];
        int b = 0;
        if (t0 < total) {
            int lo = 0, hi = a.B;           // the last b with starts[b] <= t0
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_start[mid] <= t0)
                    lo = mid;
                else
                    hi = mid;
            }
            b = lo;
        }
        int last = -1, page = -1;          // neighbours mostly share a page: its number is read once
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const long long t = t0 + e;
            int slot = -1;
            if (e < per && t < total) {
                while (t >= s_start[b + 1]) {
                    ++b;
                    last = -1;
                }
                const int off = s_off[b];
                if (off >= 0) {
                    const int len = s_len[b], pos = len + (int)(t - s_start[b]);
                    const int j = pos >> shift;
                    if (j != last) {
                        const int have = (int)up(len, shift);
                        page = j < have ? a.table[(size_t)b * a.W + j] : a.ring[ring_at((unsigned)(off + j - have))];
                        last = j;
                        if ((unsigned)page >= pages)
                            sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_PAGE);
                    }
                    if ((unsigned)page < pages)
                        slot = (page << shift) + (pos & ((1 << shift) - 1));
                }
            }
            out[e] = slot;
        }
        if (per == 4 && t0 + 4 <= a.T && ((uintptr_t)a.slots & 15u) == 0) {
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(out[0], out[1], out[2], out[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < per && t0 + e < a.T)
                    a.slots[t0 + e] = out[e];
        }
    }
}

const void *sfar_kernel_kv_plan() { return (const void *)k_kv_plan; }
