// k_kv_attn.cu -- attention of the step's tokens over the paged 8-bit cache
// (include/sfar_kv.h), for few query rows per request: decode steps.
//
// The G query heads that share a key head and a request's new tokens are the
// rows of one matrix, taken 16 at a time.  One pass over the keys with the
// running maximum and sum of the softmax: per 16 rows and tile of 64 cached
// tokens S = Q K^T, p = exp2(S - max), O = O * correction + p V.  HBM-bound:
// every cached byte is read once, 2 D bytes per token and key head, against 64
// flops per byte at 16 rows -- far below what mma.sync does, so the tile stays
// in the layout of the warp-wide instruction and nothing waits on a CTA.
//
// Numbers: e4m3 is exact in binary16, so keys and values are widened on the
// way into the registers and never rounded.  A query row is brought into
// binary16's range by a power of two (bf16's 8 bits are exact there; only
// elements 2^-29 below the row's largest lose bits) that goes back into the
// score's factor, with the page's scale.  Scores, maxima, sums and the
// accumulator are binary32.  A value's weight, p times its page's scale, is
// rounded to binary16 for the second product (2^-11, where the bf16 result has
// 2^-8); it is taken relative to a running reference of its own, so that the
// scales' size does not matter.  Both references move only when they are
// passed by 2^6: the accumulator is seldom rescaled, and weights stay below
// 2^6.
//
// Work: the tiles of all (rank, key head, request, 16 rows) form one line that
// is cut into equal pieces, one per CTA, wherever the cuts fall: a batch of
// unequal contexts and a single long one load the GPU alike, and the host
// needs no length.  Rows whose tiles lie in several CTAs are joined by the
// last of them to finish, in the order of the pieces (the result does not
// depend on which that is), from partial results in the handle's workspace.
//
// A CTA: one producer warp (page numbers, TMA copies of tiles into a ring of
// stages with the swizzle that the fragment loads want, page scales, query
// rows), four consumer warps of 16 tokens of each tile with running states of
// their own, joined through shared memory once per piece of 16 rows.
#include "sfar_e4m3.cuh"
#include "sfar_attn.cuh"
#include "sfar_tc.cuh"

namespace {

constexpr int kTile = SFAR_ATTN_TILE;              // cached tokens per stage
constexpr int kConsumers = 4, kThreads = 32 * (kConsumers + 1);
constexpr int kStages = SFAR_ATTN_STAGES;
constexpr int kRows = 16;

// Shared memory of a CTA, after the prefix sums.
template <int D> struct Lay {
    static constexpr int kStage = 2 * kTile * D;
    static constexpr int kRow = D + 16;            // floats of a row in the join buffer, padded against bank conflicts
    static constexpr int kJoin = kConsumers * kRows * kRow * 4;
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kBytes = kStages * kStage + kJoin + 2 * kQ;
};
struct Meta {                                      // of a stage
    float ks[kTile / 16], vs[kTile / 16];          // scales of each 16 tokens' page
    int bad;                                       // bit i: tokens 16 i .. are on no page of the pool
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Byte of (token, 16-byte chunk) in a tile as TMA wrote it: 128-byte rows with
// the 128-byte swizzle, 64-byte rows with the 64-byte one.
template <int D> __device__ __forceinline__ uint32_t at_chunk(int token, int chunk)
{
    return D == 128 ? token * 128 + ((chunk ^ (token & 7)) << 4) : token * 64 + ((chunk ^ ((token >> 1) & 3)) << 4);
}
// The token (of 8) that stands in column n of an 8-column fragment.  For
// 64-byte rows an order in which neither the key loads (rows n, n + 1) nor the
// value loads (columns 0 2 4 6, then 1 3 5 7) meet in a bank.
template <int D> __device__ __forceinline__ int token_of(int n)
{
    return D == 128 ? n : (int)((0x65742130u >> (4 * n)) & 7u);
}

// One piece: 16 rows of a request and a run of its tiles.
struct Piece {
    int plane, b, rt;           // rank * Hk + head; request; row tile
    int tile0, tiles;           // first tile of this piece (in tiles of the context), how many
    int begin, all;             // first tile of the whole row tile, and its count
    int len, count, first;      // context, new tokens, row of the first new token
};

struct Work {
    const uint32_t *upto;       // [B + 1] prefix sums of the requests' units, per plane
    const SfarAttnArgs &a;
    // tiles that some row of the request attends to (at least one: rows of nothing are written too)
    __device__ __forceinline__ void range(int len, int count, int &begin, int &all) const
    {
        const int pos = max(0, len - count);
        begin = (a.window ? max(0, pos - a.window + 1) : 0) / kTile;
        all = max(1, (len + kTile - 1) / kTile - begin);
    }
    __device__ __forceinline__ Piece at(long long u, long long end) const
    {
        Piece p;
        const uint32_t S = upto[a.B];
        p.plane = (int)(u / S);
        const uint32_t v = (uint32_t)(u - (long long)p.plane * S);
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (upto[mid] <= v)
                lo = mid;
            else
                hi = mid;
        }
        p.b = lo;
        sfar_attn_request(a, lo, p.len, p.count, p.first);
        range(p.len, p.count, p.begin, p.all);
        const uint32_t w = v - upto[lo];
        p.rt = (int)(w / (uint32_t)p.all);
        const int k = (int)(w - (uint32_t)p.rt * (uint32_t)p.all);
        p.tile0 = p.begin + k;
        p.tiles = (int)min((long long)(p.all - k), end - u);
        return p;
    }
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 2) k_kv_attn(const __grid_constant__ SfarAttnArgs a)
{
    using L = Lay<D>;
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ __align__(8) unsigned long long bars[2 * kStages + 4];
    __shared__ Meta meta[kStages];
    __shared__ float s_ml[3][kConsumers][kRows];   // running maximum, sum, weight reference
    __shared__ uint32_t s_warp[kThreads / 32];
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (tc::smem(dyn) + 1023u) & ~1023u;
    unsigned char *mem = dyn + (base - tc::smem(dyn));
    const uint32_t ring = base, qbuf = base + kStages * L::kStage + L::kJoin;
    float *join = reinterpret_cast<float *>(mem + kStages * L::kStage);
    uint32_t *upto = reinterpret_cast<uint32_t *>(mem + L::kBytes);
    const uint32_t full = tc::smem(bars), empty = full + 8 * kStages, qfull = empty + 8 * kStages, qempty = qfull + 16;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::bar_init(full + 8 * s, 1);
            tc::bar_init(empty + 8 * s, kConsumers);
        }
        for (int s = 0; s < 2; ++s) {
            tc::bar_init(qfull + 8 * s, 32);
            tc::bar_init(qempty + 8 * s, kConsumers);
        }
        tc::bar_fence_init();
        tc::fence_async();
        upto[0] = 0;
    }
    pdl_wait();
    const unsigned long long limit = ld_relaxed_u64(&a.ctl->timeout_ns);

    // prefix sums of the requests' units: row tiles x tiles
    const Work work{upto, a};
    uint32_t carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        uint32_t v = 0;
        if (b < a.B) {
            int len, count, first, begin, all;
            sfar_attn_request(a, b, len, count, first);
            work.range(len, count, begin, all);
            v = (uint32_t)(((long long)count * a.G + kRows - 1) / kRows) * (uint32_t)all;
            if (blockIdx.x == 0)
                sfar_attn_check(a, b, len, count, first);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(SFAR_FULL, v, d);
            if (lane >= d)
                v += o;
        }
        if (lane == 31)
            s_warp[warp] = v;
        __syncthreads();
        uint32_t before = carry, sum = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp)
                before += s_warp[w];
            sum += s_warp[w];
        }
        if (b < a.B)
            upto[b + 1] = before + v;
        carry += sum;
        __syncthreads();
    }

    sfar_attn_padding<D>(a);

    const long long U = (long long)carry * a.R * a.Hk;
    const long long N = min((long long)gridDim.x, U);
    if (blockIdx.x >= N)
        return;
    const long long u0 = blockIdx.x * U / N, u1 = (blockIdx.x + 1) * U / N;

    if (warp == kConsumers) {
        // ------------------------------------------------------------- producer
        const uint64_t once = tc::evict_first();
        tc::Ring<kStages> st;
        tc::Ring<2> qs;
        bool gave_up = false;
        uint32_t issued = 0;
        const int per = (1 << a.shift) < kTile ? 1 << a.shift : kTile;     // tokens of one copy
        const int boxes = kTile / per;
        for (long long u = u0; u < u1 && !gave_up;) {
            const Piece p = work.at(u, u1);
            const int r = p.plane / a.Hk, hk = p.plane % a.Hk;
            if (!tc::bar_wait(qempty + 8 * qs.slot, qs.phase ^ 1u, limit)) {
                gave_up = true;
                break;
            }
            for (int i = lane; i < kRows * D / 8; i += 32) {
                const int rho = i / (D / 8), c = i % (D / 8), row = p.rt * kRows + rho;
                const int tok = row / a.G;
                const uint16_t *src = a.q[r];
                uint32_t bytes = 0;
                if (tok < p.count) {
                    src += (long long)(p.first + tok) * a.qts + (long long)(hk * a.G + row % a.G) * a.qhs + c * 8;
                    bytes = 16;
                }
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(qbuf + qs.slot * L::kQ + i * 16), "l"(src), "r"(bytes)
                             : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(qfull + 8 * qs.slot) : "memory");
            qs.next();
            const int *row = a.table + (size_t)p.b * a.W;
            for (int k = 0; k < p.tiles; ++k) {
                const int j0 = (p.tile0 + k) * kTile;
                // lane i: copy i of the tile
                const int j = j0 + lane * per;
                const bool live = lane < boxes && j < p.len;
                int page = live ? row[j >> a.shift] : 0;
                const bool bad = live && (unsigned)page >= (unsigned)a.pages;
                if (bad)
                    sfar_kv_fault(a.ctl, p.b, SFAR_KV_BAD_PAGE);
                const bool go = live && !bad;
                const int slab = page * a.Hk + hk;
                float ks = 0.f, vs = 0.f;
                if (go) {
                    ks = a.ks[r][slab];
                    vs = a.vs[r][slab];
                }
                if (!tc::bar_wait(empty + 8 * st.slot, st.phase ^ 1u, limit)) {
                    gave_up = true;
                    break;
                }
                const uint32_t bar = full + 8 * st.slot, dst = ring + st.slot * L::kStage + lane * per * D;
                if (go) {
                    tc::load_3d(dst, &a.kmap[r], 0, j & ((1 << a.shift) - 1), slab, bar, once);
                    tc::load_3d(dst + kTile * D, &a.vmap[r], 0, j & ((1 << a.shift) - 1), slab, bar, once);
                }
                const unsigned any = __ballot_sync(SFAR_FULL, go);
                const int of = lane * 16 / per;                             // the copy that 16 tokens lie in
                const float k16 = __shfl_sync(SFAR_FULL, ks, of & 31), v16 = __shfl_sync(SFAR_FULL, vs, of & 31);
                const unsigned dead = __ballot_sync(SFAR_FULL, lane < kTile / 16 && !(any >> (of & 31) & 1u));
                Meta &m = meta[st.slot];
                if (lane < kTile / 16) {
                    m.ks[lane] = k16;
                    m.vs[lane] = v16;
                }
                if (lane == 0)
                    m.bad = (int)dead;
                __syncwarp();
                if (lane == 0)
                    tc::bar_expect(bar, (uint32_t)__popc(any) * 2u * per * D);
                st.next();
                ++issued;
            }
            u += p.tiles;
        }
        if (gave_up && lane == 0) {
            sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
            // the copies in flight land before the shared memory is released
            const uint32_t back = issued < (uint32_t)kStages ? issued : (uint32_t)kStages;
            for (uint32_t i = issued - back; i < issued; ++i)
                tc::bar_wait(full + 8 * (i % kStages), (i / kStages) & 1u, limit);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }

    // ---------------------------------------------------------------- consumers
    constexpr int kK = D / 16;                     // steps of 16 along the head
    const int g = lane >> 2, t = lane & 3;
    tc::Ring<kStages> st;
    tc::Ring<2> qs;
    bool dead = false;                             // a wait gave up: go on without waiting, so that the warps stay together
    for (long long u = u0; u < u1;) {
        const Piece p = work.at(u, u1);
        const int r = p.plane / a.Hk, hk = p.plane % a.Hk;
        const int rows = min(kRows, p.count * a.G - p.rt * kRows);
        // the query rows g and g + 8, brought into binary16's range
        uint32_t q[kK][4];
        float f[2];
        int lo[2], hi[2];
        dead = dead || !tc::bar_wait(qfull + 8 * qs.slot, qs.phase, limit);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rho = g + 8 * i;
            uint4 v[D / 32];
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                v[c] = lds128(qbuf + qs.slot * L::kQ + rho * D * 2 + t * (D / 2) + c * 16);
                m = sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(m, v[c].x), v[c].y), v[c].z), v[c].w);
            }
            m = sfar_max_half(m);
            m = max(m, __shfl_xor_sync(SFAR_FULL, m, 1));
            m = max(m, __shfl_xor_sync(SFAR_FULL, m, 2));
            const int e = max((int)(m >> 7) - 127, -112);       // largest magnitude below 2^(e + 1)
            const float up = sfar_exp2i(14 - e);
            f[i] = a.scale * 1.4426950408889634f * sfar_exp2i(max(e - 14, -126));
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int x = 0; x < 4; ++x)       // values 8 c + 2 x, + 1 of the lane's D / 4
                    q[2 * c + (x >> 1)][2 * (x & 1) + i] = half2_of(bf16_lo(w[x]) * up, bf16_hi(w[x]) * up);
            }
            const int pos = p.len - p.count + (p.rt * kRows + rho) / a.G;
            hi[i] = rho < rows ? pos + 1 : INT_MAX;
            lo[i] = rho < rows && a.window ? max(0, pos - a.window + 1) : 0;
        }
        __syncwarp();
        if (lane == 0)
            tc::bar_arrive(qempty + 8 * qs.slot);
        qs.next();
        // tiles that every row sees whole
        const int pos0 = p.len - p.count + p.rt * kRows / a.G, pos1 = p.len - p.count + (p.rt * kRows + rows - 1) / a.G;
        const int all_from = a.window ? max(0, pos1 - a.window + 1) : 0, all_to = pos0 + 1;

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        // log2 references: of the scores (sum), of the weights (o)
        float top[2] = {-INFINITY, -INFINITY}, wtop[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
        for (int k = 0; k < p.tiles; ++k) {
            const int j0 = (p.tile0 + k) * kTile;
            dead = dead || !tc::bar_wait(full + 8 * st.slot, st.phase, limit);
            const uint32_t kt = ring + st.slot * L::kStage, vt = kt + kTile * D;
            const Meta &m = meta[st.slot];
            const bool edge = j0 < all_from || j0 + kTile > all_to || m.bad;
            const int c0 = warp * 16;              // this warp's tokens of the tile
            float s[2][4] = {};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int tok = c0 + 8 * n + token_of<D>(g);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint4 w4 = lds128(kt + at_chunk<D>(tok, t * (D / 64) + c));
                    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mma_f16(s[n], q[4 * c + x], cvt_f16x2_e4m3(w[x]), cvt_f16x2_e4m3(w[x] >> 16));
                }
            }
            const float ks = m.ks[warp], vs = m.vs[warp];
            const bool gone = (m.bad >> warp) & 1;
            // scores in units of log2; columns 2 t, 2 t + 1 of either fragment
            float x[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[n][e] = s[n][e] * (f[e >> 1] * ks);
            if (edge) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + c0 + 8 * n + token_of<D>(2 * t + (e & 1));
                        if (gone || j >= p.len || j < lo[e >> 1] || j >= hi[e >> 1])
                            x[n][e] = -INFINITY;
                    }
            }
            const float lvs = lg2(fabsf(vs));
            float now[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                now[i] = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
                now[i] = fmaxf(now[i], __shfl_xor_sync(SFAR_FULL, now[i], 1));
                now[i] = fmaxf(now[i], __shfl_xor_sync(SFAR_FULL, now[i], 2));
            }
            const bool move = now[0] > top[0] + kAttnLift || now[1] > top[1] + kAttnLift || now[0] + lvs > wtop[0] + kAttnLift ||
                              now[1] + lvs > wtop[1] + kAttnLift;
            if (__any_sync(SFAR_FULL, move)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float next = fmaxf(top[i], now[i]), wnext = fmaxf(wtop[i], now[i] + lvs);
                    const float keep = wtop[i] == -INFINITY ? 0.f : ex2(wtop[i] - wnext);
                    sum[i] *= top[i] == -INFINITY ? 1.f : ex2(top[i] - next);
                    top[i] = next;
                    wtop[i] = wnext;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][2 * i] *= keep;
                        o[n][2 * i + 1] *= keep;
                    }
                }
            }
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float ref = top[i] == -INFINITY ? 0.f : top[i];
                const float by = copysignf(wtop[i] == -INFINITY ? 0.f : ex2(ref + lvs - wtop[i]), vs);
                float e4[4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        e4[2 * n + e] = ex2(x[n][2 * i + e] - ref);
                sum[i] += (e4[0] + e4[1]) + (e4[2] + e4[3]);
                w[i] = half2_of(e4[0] * by, e4[1] * by);
                w[2 + i] = half2_of(e4[2] * by, e4[3] * by);
            }
            // values: rows of the columns 2 t, 2 t + 1 (either fragment), 16 (8) bytes of the head at 16 g (8 g)
            constexpr int kW = D / 32;             // words of a lane's part of a row
            uint32_t v[4][kW];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int tok = c0 + 8 * (e >> 1) + token_of<D>(2 * t + (e & 1));
                if constexpr (D == 128) {
                    const uint4 y = lds128(vt + at_chunk<D>(tok, g));
                    v[e][0] = y.x;
                    v[e][1] = y.y;
                    v[e][2] = y.z;
                    v[e][3] = y.w;
                } else {
                    const uint2 y = lds64(vt + at_chunk<D>(tok, g >> 1) + (g & 1) * 8);
                    v[e][0] = y.x;
                    v[e][1] = y.y;
                }
            }
            bool nan = false;
            if (edge) {
                // a value that some row must not see is taken out; one that is NaN is put back below for the rows that see it
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j0 + c0 + 8 * (e >> 1) + token_of<D>(2 * t + (e & 1));
                    const bool off = gone || j >= p.len;
#pragma unroll
                    for (int i = 0; i < kW; ++i) {
                        if (off)
                            v[e][i] = 0;
                        const uint32_t is = __vcmpeq4(v[e][i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        nan = nan || is;
                        v[e][i] &= ~is;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                const uint32_t a01 = __byte_perm(v[0][i], v[1][i], 0x5140), a23 = __byte_perm(v[0][i], v[1][i], 0x7362);
                const uint32_t b01 = __byte_perm(v[2][i], v[3][i], 0x5140), b23 = __byte_perm(v[2][i], v[3][i], 0x7362);
                mma_f16(o[4 * i], w, cvt_f16x2_e4m3(a01), cvt_f16x2_e4m3(b01));
                mma_f16(o[4 * i + 1], w, cvt_f16x2_e4m3(a01 >> 16), cvt_f16x2_e4m3(b01 >> 16));
                mma_f16(o[4 * i + 2], w, cvt_f16x2_e4m3(a23), cvt_f16x2_e4m3(b23));
                mma_f16(o[4 * i + 3], w, cvt_f16x2_e4m3(a23 >> 16), cvt_f16x2_e4m3(b23 >> 16));
            }
            if (edge && __any_sync(SFAR_FULL, nan)) {
                // o[n][2 i + e]: row g + 8 i, element (D / 8) (2 t + e) + n of the head
                for (int n = 0; n < 16 && !gone; ++n) {
                    const int j = j0 + c0 + n;
#pragma unroll
                    for (int d = 0; d < D / 8; ++d)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int at = (D / 8) * (2 * t + e) + d;
                            uint32_t byte;
                            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(vt + at_chunk<D>(c0 + n, at >> 4) + (at & 15)));
                            if ((byte & 0x7f) == 0x7f && j < p.len) {
                                if (j >= lo[0] && j < hi[0])
                                    o[d][e] = NAN;
                                if (j >= lo[1] && j < hi[1])
                                    o[d][2 + e] = NAN;
                            }
                        }
                }
            }
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(empty + 8 * st.slot);
            st.next();
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[i] += __shfl_xor_sync(SFAR_FULL, sum[i], 1);
            sum[i] += __shfl_xor_sync(SFAR_FULL, sum[i], 2);
        }
        // join the warps' states
        consumers_sync();                          // the last piece's has been read
        if (t == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s_ml[0][warp][g + 8 * i] = top[i];
                s_ml[1][warp][g + 8 * i] = sum[i];
                s_ml[2][warp][g + 8 * i] = wtop[i];
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int n = 0; n < D / 8; n += 4) {
                    float *dst = join + (warp * kRows + g + 8 * i) * L::kRow + t * (D / 4 + 4) + e * (D / 8) + n;
                    *reinterpret_cast<float4 *>(dst) =
                        make_float4(o[n][2 * i + e], o[n + 1][2 * i + e], o[n + 2][2 * i + e], o[n + 3][2 * i + e]);
                }
        consumers_sync();
        constexpr int kE = D / 8;                  // elements of one row per thread: 8 threads a row
        const int row = tid >> 3, col = (tid & 7) * kE;
        SfarAttnState<kE> all;
        for (int w = 0; w < kConsumers; ++w)
            all.reference(s_ml[0][w][row], s_ml[2][w][row]);
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
            const float by = all.add(s_ml[0][w][row], s_ml[1][w][row], s_ml[2][w][row]);
            const float *src = join + (w * kRows + row) * L::kRow + col / (D / 4) * (D / 4 + 4) + col % (D / 4);
#pragma unroll
            for (int e = 0; e < kE; e += 4)
                all.add4(e, by, *reinterpret_cast<const float4 *>(src + e));
        }
        bool write = true;
        if (p.tiles < p.all) {
            // a part: leave it in the workspace; the last of the row tile's CTAs joins them in order
            const long long from = u - (p.tile0 - p.begin), to = from + p.all;
            const long long c0 = ((from + 1) * N - 1) / U, c1 = (to * N - 1) / U;
            const int mine = p.tile0 == p.begin ? 1 : 0;
            auto slot = [&](long long c, int which) { return a.part + ((size_t)c * 2 + which) * (kRows * (D + 4)); };
            float *dst = slot(blockIdx.x, mine);
            if (row < rows) {
#pragma unroll
                for (int e = 0; e < kE; e += 4)
                    __stcg(reinterpret_cast<float4 *>(dst + row * D + col + e),
                           make_float4(all.o[e], all.o[e + 1], all.o[e + 2], all.o[e + 3]));
                if (col == 0)
                    __stcg(reinterpret_cast<float4 *>(dst + kRows * D + row * 4), make_float4(all.top, all.sum, all.wtop, 0.f));
            }
            __threadfence();
            consumers_sync();
            if (tid == 0) {
                const int done = atomicAdd(a.arrived + c0, 1);
                s_last = done == (int)(c1 - c0);
                if (s_last)
                    a.arrived[c0] = 0;             // for the next call
            }
            consumers_sync();
            write = s_last;
            if (write && row < rows) {
                __threadfence();
                all = SfarAttnState<kE>();
#pragma unroll 8
                for (long long c = c0; c <= c1; ++c) {
                    const float4 m = __ldcg(reinterpret_cast<const float4 *>(slot(c, c == c0) + kRows * D + row * 4));
                    all.reference(m.x, m.z);
                }
#pragma unroll 4
                for (long long c = c0; c <= c1; ++c) {
                    const float *src = slot(c, c == c0);
                    const float4 m = __ldcg(reinterpret_cast<const float4 *>(src + kRows * D + row * 4));
                    float4 v[kE / 4];
#pragma unroll
                    for (int e = 0; e < kE; e += 4)
                        v[e / 4] = __ldcg(reinterpret_cast<const float4 *>(src + row * D + col + e));
                    const float by = all.add(m.x, m.y, m.z);
#pragma unroll
                    for (int e = 0; e < kE; e += 4)
                        all.add4(e, by, v[e / 4]);
                }
            }
        }
        if (write && row < rows) {
            const int n = p.rt * kRows + row;
            const float inv = all.factor();
            uint16_t *dst = a.out[r] + (long long)(p.first + n / a.G) * a.ots + (long long)(hk * a.G + n % a.G) * a.ohs + col;
#pragma unroll
            for (int e = 0; e < kE; e += 8)
                st_v4(dst + e, make_uint4(tc::bf16x2(all.o[e] * inv, all.o[e + 1] * inv), tc::bf16x2(all.o[e + 2] * inv, all.o[e + 3] * inv),
                                          tc::bf16x2(all.o[e + 4] * inv, all.o[e + 5] * inv), tc::bf16x2(all.o[e + 6] * inv, all.o[e + 7] * inv)));
        }
        u += p.tiles;
    }
    if (dead && lane == 0)
        sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
}

const void *sfar_kernel_kv_attn(int head_dim, int *threads, int *smem)
{
    *threads = kThreads;
    *smem = (head_dim == 64 ? Lay<64>::kBytes : Lay<128>::kBytes) + 1024;
    return head_dim == 64 ? (const void *)k_kv_attn<64> : (const void *)k_kv_attn<128>;
}
