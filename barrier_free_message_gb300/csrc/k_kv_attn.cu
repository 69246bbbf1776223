// k_kv_attn.cu -- attention of the step's tokens over the paged 8-bit cache
// (include/sfar_kv.h), for few query rows per request: decode steps.
//
// The G query heads that share a key head and a request's new tokens are the
// rows of one matrix, taken 8 or 16 at a time.  One pass over the keys with the
// running maximum and sum of the softmax: per tile of 64 cached tokens
// S = Q K^T, p = exp2(S - max), O = O * correction + p V.  HBM-bound: every
// cached byte is read once, 2 D bytes per token and key head, against 64 flops
// per byte at 16 rows -- far below what mma.sync does, so the tile stays in the
// layout of the warp-wide instruction and nothing waits on a CTA.  The
// products are formed transposed, S^T = K Q^T and O^T = V^T p^T: tokens and
// head elements take the instruction's 16 rows, the query rows its 8 columns,
// so that 8 rows (the common G) waste nothing.
//
// Numbers: e4m3 is exact in binary16, so keys and values are widened on the
// way into the registers and never rounded.  A query row is brought into
// binary16's range by a power of two (bf16's 8 bits are exact there; only
// elements 2^-29 below the row's largest lose bits) that goes back into the
// score's factor, with the page's scale.  Scores, maxima, sums and the
// accumulator are binary32.  A value's weight, p times its page's scale, is
// rounded to binary16 for the second product (2^-11, where the bf16 result has
// 2^-8); it is taken relative to a running reference of its own, so that the
// scales' size does not matter.  A row's references move only when its scores
// pass them by 2^7.9, so that the accumulator is seldom rescaled.  The weights'
// stands 2^8 lower and uses binary16's range: weights are at most 2^15.9, and
// lose bits only below 2^-22 of the row's largest.
//
// Work: the tiles of all (rank, key head, request, 8 or 16 rows) form one line that
// is cut into equal pieces, one per CTA, wherever the cuts fall: a batch of
// unequal contexts and a single long one load the GPU alike, and the host
// needs no length.  Rows whose tiles lie in several CTAs are joined by the
// last of them to finish, in the order of the pieces (the result does not
// depend on which that is), from partial results in the handle's workspace.
//
// A CTA: one producer warp (page numbers, TMA copies of tiles into a ring of
// stages with the swizzle that the fragment loads want, page scales, query
// rows), four consumer warps of 16 tokens of each tile with running states of
// their own, joined through shared memory once per piece.  Three CTAs per SM
// with 8 rows, two with 16 (the registers of the accumulator): the others'
// tiles hide a CTA's first page lookups and its joins.
//
// Measured: 8 ranks, one key head of 128, 8 query heads: 64 requests of 6003 to
// 10400 tokens, 1.08 GB in 162 us, 6.7 TB/s or 0.98 of a copy's rate; 16
// requests of 301 to 4096, 72 MB in 22 us, of which about 8 pass outside the
// stream of tiles (launch, prefix sums and first page lookups, partial results
// and their join, unequal ends).  4 ranks of two key heads with 5 query heads
// each, one context of 131071 tokens: 269 MB in 49 us, 5.5 TB/s.  99 tokens of
// one request: 5.9 us, the latency of the chain; 2112 row tiles of 5 tokens 24.
// 8 rows fit 128 registers; 16 rows of 128 elements spill 44 bytes at 168.
#include "sfar_e4m3.cuh"
#include "sfar_attn.cuh"
#include "sfar_tc.cuh"

namespace {

constexpr int kTile = SFAR_ATTN_TILE;              // cached tokens per stage
constexpr int kConsumers = 4, kThreads = 32 * (kConsumers + 1);
// A weight is exp2(score - top) times exp2(top + log2 scale - wtop).  Tokens of value scale 0 count for `top` alone, so
// where they are the row's largest the second factor has no bound while the first underflows; a page's weights are taken
// for 0 where it passes this, their share of the row's sum being below 2^-100.  Up to nonzero scales 2^100 apart it stays
// below.
constexpr float kFar = 120.f;

// Shared memory of a CTA, after the prefix sums.
template <int D, int RH> struct Lay {
    static constexpr int kRows = 8 * RH, kStages = RH == 1 ? 3 : 4;
    static constexpr int kStage = 2 * kTile * D;
    static constexpr int kRow = D + 4;             // floats of a row in the join buffer, padded against bank conflicts
    static constexpr int kJoin = kConsumers * kRows * kRow * 4;
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kBytes = kStages * kStage + kJoin + 2 * kQ;
};
struct Meta {                                      // of a stage
    float ks[kTile / 16], vs[kTile / 16];          // scales of each 16 tokens' page
    int bad;                                       // bit i: tokens 16 i .. are on no page of the pool
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, const uint32_t (&b)[2])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
// an 8 x 8 matrix of 16-bit values, a row to four lanes, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Byte of (token, 16-byte chunk) in a tile as TMA wrote it: 128-byte rows with
// the 128-byte swizzle, 64-byte rows with the 64-byte one.
template <int D> __device__ __forceinline__ uint32_t at_chunk(int token, int chunk)
{
    return D == 128 ? token * 128 + ((chunk ^ (token & 7)) << 4) : token * 64 + ((chunk ^ ((token >> 1) & 3)) << 4);
}
// The token (of 8) that stands at place n of a fragment's 8.  For 64-byte rows
// an order in which neither the key loads (places n, n + 1) nor the value loads
// (places 0 2 4 6, then 1 3 5 7) meet in a bank.
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

template <int kRows> struct Work {
    const uint32_t *upto;       // [B + 1] prefix sums of the requests' units, per plane
    const SfarAttnArgs &a;
    // tiles that some row of the request attends to (at least one: rows of nothing are written too)
    __device__ __forceinline__ void range(int len, int count, int &begin, int &all) const
    {
        begin = sfar_attn_from(a, len - count) / kTile;
        all = max(1, (len + kTile - 1) / kTile - begin);
    }
    __device__ __forceinline__ Piece at(long long u, long long end) const
    {
        Piece p;
        const uint32_t S = upto[a.B];
        p.plane = (int)sfar_div(u, S);
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

template <int D, int RH>
__global__ void __launch_bounds__(kThreads, RH == 1 ? 3 : 2) k_kv_attn(const __grid_constant__ SfarAttnArgs a)
{
    using L = Lay<D, RH>;
    constexpr int kRows = L::kRows, kStages = L::kStages;
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ __align__(8) unsigned long long bars[2 * kStages + 4];
    __shared__ Meta meta[kStages];
    __shared__ Piece s_next[2];                    // with the query rows' buffers: what the producer has begun with
    __shared__ Piece s_piece[kConsumers];          // each warp's, out of its registers
    __shared__ float s_ml[3][kConsumers][kRows];   // running maximum, sum, weight reference
    __shared__ uint32_t s_warp[kThreads / 32];
    __shared__ int s_last, s_nan[2][2];            // by the piece's parity: first and last token whose value holds a NaN
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (tc::smem(dyn) + 1023u) & ~1023u;
    unsigned char *mem = dyn + (base - tc::smem(dyn));
    const uint32_t ring = base, qbuf = base + kStages * L::kStage + L::kJoin;
    float *joint = reinterpret_cast<float *>(mem + kStages * L::kStage);
    uint32_t *upto = reinterpret_cast<uint32_t *>(mem + L::kBytes);
    const uint32_t full = tc::smem(bars), empty = full + 8 * kStages, qfull = empty + 8 * kStages, qempty = qfull + 16;

    if (warp == kConsumers && lane < 2 * a.R)
        tc::prefetch_map(lane & 1 ? &a.vmap[lane >> 1] : &a.kmap[lane >> 1]);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::bar_init(full + 8 * s, 1);
            tc::bar_init(empty + 8 * s, kConsumers);
        }
        for (int s = 0; s < 2; ++s) {
            tc::bar_init(qfull + 8 * s, 33);
            tc::bar_init(qempty + 8 * s, kConsumers);
        }
        tc::bar_fence_init();
        tc::fence_async();
        upto[0] = 0;
        s_nan[0][0] = INT_MAX;
        s_nan[0][1] = -1;
    }
    pdl_wait();
    const unsigned long long limit = ld_relaxed_u64(&a.ctl->timeout_ns);

    // prefix sums of the requests' units: row tiles x tiles
    const Work<kRows> work{upto, a};
    uint32_t carry = 0;
    int row_tiles = 0;                             // this thread's requests'
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        uint32_t v = 0;
        if (b < a.B) {
            int len, count, first, begin, all;
            sfar_attn_request(a, b, len, count, first);
            work.range(len, count, begin, all);
            const int n = (int)(((long long)count * a.G + kRows - 1) / kRows);
            v = (uint32_t)n * (uint32_t)all;
            row_tiles = min(row_tiles + n, 1 << 26);       // above any step's; 32 such sums fit 32 bits
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

    // The line is cut into as many pieces as there are CTAs, but short row tiles are left whole, or in cuts of four tiles:
    // joining two parts costs what six tiles do (a context of 99 tokens: 8.2 us in two parts, 5.7 in one).
    row_tiles = __reduce_add_sync(SFAR_FULL, row_tiles);
    if (lane == 0)
        s_warp[warp] = (uint32_t)row_tiles;
    __syncthreads();
    long long whole = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
        whole += s_warp[w];
    const long long U = sfar_attn_many(a, whole) ? 0 : (long long)carry * a.R * a.Hk;
    const long long N = min(min((long long)gridDim.x, U), max(whole * a.R * a.Hk, U / 4));
    if (blockIdx.x >= N) {
        sfar_attn_padding<D>(a, tid, kThreads);
        return;
    }
    const long long u0 = sfar_div(blockIdx.x * U, N), u1 = sfar_div((blockIdx.x + 1) * U, N);

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
            // the piece's query rows, once its first copies are on their way
            auto fetch = [&]() {
                if (!tc::bar_wait(qempty + 8 * qs.slot, qs.phase ^ 1u, limit)) {
                    gave_up = true;
                    return;
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
                if (lane == 0) {
                    s_next[qs.slot] = p;
                    tc::bar_arrive(qfull + 8 * qs.slot);
                }
                qs.next();
            };
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
                if (k == 0)
                    fetch();
                const unsigned any = __ballot_sync(SFAR_FULL, go);
                const int of = lane * 16 / per;                             // the copy that 16 tokens lie in
                const float k16 = __shfl_sync(SFAR_FULL, ks, of & 31), v16 = __shfl_sync(SFAR_FULL, vs, of & 31);
                const unsigned dead = __ballot_sync(SFAR_FULL, lane < kTile / 16 && !(any >> (of & 31) & 1u));
                Meta &m = meta[st.slot];
                if (lane < kTile / 16) {
                    m.ks[lane] = k16;
                    m.vs[lane] = fabsf(v16) <= kNoScale ? 0.f : v16;
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
    int piece = 0;
    for (long long u = u0; u < u1;) {
        dead = dead || !tc::bar_wait(qfull + 8 * qs.slot, qs.phase, limit);
        __syncwarp();
        if (__any_sync(SFAR_FULL, dead)) {
            dead = true;
            const Piece q = work.at(u, u1);
            if (lane == 0)
                s_piece[warp] = q;
        } else if (lane < sizeof(Piece) / 4) {
            reinterpret_cast<int *>(&s_piece[warp])[lane] = reinterpret_cast<const int *>(&s_next[qs.slot])[lane];
        }
        __syncwarp();
        const Piece &p = s_piece[warp];
        const int r = p.plane / a.Hk, hk = p.plane % a.Hk;
        const int rows = min(kRows, p.count * a.G - p.rt * kRows);
        // The query rows, brought into binary16's range: of each 8, lane (g, t) holds a quarter of row g, and answers for
        // rows 2 t and 2 t + 1 of the scores.
        uint32_t q[RH][kK][2];
        float f[RH][2];
        int lo[RH][2], hi[RH][2];
        const unsigned char *qrow = mem + kStages * L::kStage + L::kJoin + qs.slot * L::kQ;
#pragma unroll
        for (int i = 0; i < RH; ++i) {
            uint4 v[D / 32];
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                v[c] = *reinterpret_cast<const uint4 *>(qrow + (8 * i + g) * D * 2 + t * (D / 2) + c * 16);
                m = sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(m, v[c].x), v[c].y), v[c].z), v[c].w);
            }
            m = sfar_max_half(m);
            m = max(m, __shfl_xor_sync(SFAR_FULL, m, 1));
            m = max(m, __shfl_xor_sync(SFAR_FULL, m, 2));
            const int e = max((int)(m >> 7) - 127, -112);       // largest magnitude below 2^(e + 1)
            const float up = m >= 0x7f80u ? 0.f : sfar_exp2i(14 - e);        // an infinity becomes NaN: scores of -inf would count as masked
            const float mine = a.scale * 1.4426950408889634f * sfar_exp2i(max(e - 14, -126));
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int x = 0; x < 4; ++x)       // values 8 c + 2 x, + 1 of the lane's D / 4
                    q[i][2 * c + (x >> 1)][x & 1] = half2_of(bf16_lo(w[x]) * up, bf16_hi(w[x]) * up);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int rho = 8 * i + 2 * t + y, pos = p.len - p.count + (p.rt * kRows + rho) / a.G;
                f[i][y] = __shfl_sync(SFAR_FULL, mine, 4 * (2 * t + y));
                hi[i][y] = rho < rows ? pos + 1 : INT_MAX;
                lo[i][y] = rho < rows ? sfar_attn_from(a, pos) : 0;
            }
        }
        __syncwarp();
        if (lane == 0)
            tc::bar_arrive(qempty + 8 * qs.slot);
        qs.next();
        // tiles that every row sees whole
        const int pos0 = p.len - p.count + p.rt * kRows / a.G, pos1 = p.len - p.count + (p.rt * kRows + rows - 1) / a.G;
        const int all_from = sfar_attn_from(a, pos1), all_to = pos0 + 1;

        float o[RH][D / 16][4] = {};               // o[i][n][2 h + y]: row 8 i + 2 t + y, element (D / 8) g + 2 n + h
        // log2 references: of the scores (sum), of the weights (o)
        float top[RH][2], wtop[RH][2], sum[RH][2];
#pragma unroll
        for (int i = 0; i < 2 * RH; ++i) {
            top[i >> 1][i & 1] = wtop[i >> 1][i & 1] = -INFINITY;
            sum[i >> 1][i & 1] = 0.f;
        }
        const int j00 = p.tile0 * kTile, j1 = j00 + p.tiles * kTile;
        for (int j0 = j00; j0 < j1; j0 += kTile) {
            dead = dead || !tc::bar_wait(full + 8 * st.slot, st.phase, limit);
            const unsigned char *kt = mem + st.slot * L::kStage, *vt = kt + kTile * D;
            const Meta &m = meta[st.slot];
            const bool edge = j0 < all_from || j0 + kTile > all_to || m.bad;
            const int c0 = warp * 16;              // this warp's tokens of the tile
            // scores, transposed: x[i][2 h + y] of token g (+ 8 h) and row 8 i + 2 t + y
            float x[RH][4] = {};
            {
                const unsigned char *k0 = kt, *k1 = kt;
                uint4 ka[D / 64], kb[D / 64];
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    ka[c] = *reinterpret_cast<const uint4 *>(k0 + at_chunk<D>(c0 + token_of<D>(g), t * (D / 64) + c));
                    kb[c] = *reinterpret_cast<const uint4 *>(k1 + at_chunk<D>(c0 + 8 + token_of<D>(g), t * (D / 64) + c));
                }
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint32_t w[4] = {ka[c].x, ka[c].y, ka[c].z, ka[c].w}, z[4] = {kb[c].x, kb[c].y, kb[c].z, kb[c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a0 = cvt_f16x2_e4m3(w[e]), a1 = cvt_f16x2_e4m3(z[e]), a2 = cvt_f16x2_e4m3(w[e] >> 16),
                                       a3 = cvt_f16x2_e4m3(z[e] >> 16);
#pragma unroll
                        for (int i = 0; i < RH; ++i)
                            mma_f16(x[i], a0, a1, a2, a3, q[i][4 * c + e]);
                    }
                }
            }
            const float ks = m.ks[warp], vs = m.vs[warp];
            const bool gone = (m.bad >> warp) & 1;
            const float lvs = lg2(fabsf(vs));
            bool move = false;
#pragma unroll
            for (int i = 0; i < RH; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float by = f[i][y] * ks;   // to units of log2
                    x[i][y] *= by;
                    x[i][2 + y] *= by;
                    if (edge) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int j = j0 + c0 + 8 * h + token_of<D>(g);
                            if (gone || j >= p.len || j < lo[i][y] || j >= hi[i][y])
                                x[i][2 * h + y] = -INFINITY;
                        }
                    }
                    const float now = fmaxf(x[i][y], x[i][2 + y]);
                    move = move || now > top[i][y] + kAttnLift || now + lvs > wtop[i][y] + (kAttnLift + kAttnDeep);
                }
            if (__any_sync(SFAR_FULL, move)) {
#pragma unroll
                for (int i = 0; i < RH; ++i)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float now = fmaxf(x[i][y], x[i][2 + y]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            now = fmaxf(now, __shfl_xor_sync(SFAR_FULL, now, d));
                        // a row's references go by its own scores alone
                        const float next = now > top[i][y] + kAttnLift ? now : top[i][y];
                        const float wnext = now + lvs > wtop[i][y] + (kAttnLift + kAttnDeep) ? now + lvs - kAttnDeep : wtop[i][y];
                        const float keep = wtop[i][y] == -INFINITY ? 1.f : ex2(wtop[i][y] - wnext);      // o is 0 then, or NaN
                        sum[i][y] *= top[i][y] == -INFINITY ? 1.f : ex2(top[i][y] - next);
                        top[i][y] = next;
                        wtop[i][y] = wnext;
#pragma unroll
                        for (int n = 0; n < D / 16; ++n) {
                            o[i][n][y] *= keep;
                            o[i][n][2 + y] *= keep;
                        }
                    }
            }
            uint32_t w[RH][2];
#pragma unroll
            for (int i = 0; i < RH; ++i) {
                float e4[4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float ref = top[i][y] == -INFINITY ? 0.f : top[i][y];
                    const float up = ref + lvs - wtop[i][y];          // inf or NaN while no token has a value scale
                    const float by = copysignf(up <= kFar ? ex2(up) : 0.f, vs);
                    const float e0 = ex2(x[i][y] - ref), e1 = ex2(x[i][2 + y] - ref);
                    sum[i][y] += e0 + e1;
                    e4[y] = e0 * by;
                    e4[2 + y] = e1 * by;
                }
                w[i][0] = transpose8(half2_of(e4[0], e4[1]));
                w[i][1] = transpose8(half2_of(e4[2], e4[3]));
            }
            // values: rows of the columns 2 t, 2 t + 1 (either fragment), 16 (8) bytes of the head at 16 g (8 g)
            constexpr int kW = D / 32;             // words of a lane's part of a row
            uint32_t v[4][kW];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int tok = c0 + 8 * (e >> 1) + token_of<D>(2 * t + (e & 1));
                if constexpr (D == 128) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(vt + at_chunk<D>(tok, g));
                    v[e][0] = y.x;
                    v[e][1] = y.y;
                    v[e][2] = y.z;
                    v[e][3] = y.w;
                } else {
                    const uint2 y = *reinterpret_cast<const uint2 *>(vt + at_chunk<D>(tok, g >> 1) + (g & 1) * 8);
                    v[e][0] = y.x;
                    v[e][1] = y.y;
                }
            }
            if (edge) {
                // places that hold no token are zeros; a NaN, which would reach every row, is taken out, and put back
                // when the piece is joined
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j0 + c0 + 8 * (e >> 1) + token_of<D>(2 * t + (e & 1));
                    uint32_t any = 0;
#pragma unroll
                    for (int i = 0; i < kW; ++i) {
                        if (gone || j >= p.len)
                            v[e][i] = 0;
                        const uint32_t is = __vcmpeq4(v[e][i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        any |= is;
                        v[e][i] &= ~is;
                    }
                    if (any) {
                        atomicMin(&s_nan[piece & 1][0], j);
                        atomicMax(&s_nan[piece & 1][1], j);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                const uint32_t a01 = __byte_perm(v[0][i], v[1][i], 0x5140), a23 = __byte_perm(v[0][i], v[1][i], 0x7362);
                const uint32_t b01 = __byte_perm(v[2][i], v[3][i], 0x5140), b23 = __byte_perm(v[2][i], v[3][i], 0x7362);
                const uint32_t va[8] = {cvt_f16x2_e4m3(a01), cvt_f16x2_e4m3(a01 >> 16), cvt_f16x2_e4m3(b01), cvt_f16x2_e4m3(b01 >> 16),
                                        cvt_f16x2_e4m3(a23), cvt_f16x2_e4m3(a23 >> 16), cvt_f16x2_e4m3(b23), cvt_f16x2_e4m3(b23 >> 16)};
#pragma unroll
                for (int r8 = 0; r8 < RH; ++r8) {
                    mma_f16(o[r8][2 * i], va[0], va[1], va[2], va[3], w[r8]);
                    mma_f16(o[r8][2 * i + 1], va[4], va[5], va[6], va[7], w[r8]);
                }
            }
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(empty + 8 * st.slot);
            st.next();
        }
        // join the warps' states
        consumers_sync();                          // the last piece's has been read
        if (tid == 0) {
            s_nan[(piece + 1) & 1][0] = INT_MAX;
            s_nan[(piece + 1) & 1][1] = -1;
        }
#pragma unroll
        for (int i = 0; i < RH; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float all = sum[i][y];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    all += __shfl_xor_sync(SFAR_FULL, all, d);
                const int rho = 8 * i + 2 * t + y;
                if (g == 0) {
                    s_ml[0][warp][rho] = top[i][y];
                    s_ml[1][warp][rho] = all;
                    s_ml[2][warp][rho] = wtop[i][y];
                }
                float *dst = joint + (warp * kRows + rho) * L::kRow + g * (D / 8);
#pragma unroll
                for (int n = 0; n < D / 16; n += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * n) = make_float4(o[i][n][y], o[i][n][2 + y], o[i][n + 1][y], o[i][n + 1][2 + y]);
            }
        consumers_sync();
        constexpr int kE = RH * D / 16, kT = D / kE;       // elements of one row per thread, threads of a row
        const int row = tid / kT, col = tid % kT * kE;
        SfarAttnState<kE> all;
        for (int w = 0; w < kConsumers; ++w)
            all.reference(s_ml[0][w][row], s_ml[2][w][row]);
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
            const float by = all.add(s_ml[0][w][row], s_ml[1][w][row], s_ml[2][w][row]);
            const float *src = joint + (w * kRows + row) * L::kRow + col;
#pragma unroll
            for (int e = 0; e < kE; e += 4)
                all.add4(e, by, *reinterpret_cast<const float4 *>(src + e));
        }
        const int *nan = s_nan[piece++ & 1];
        if (nan[1] >= 0 && row < rows) {
            const int n = p.rt * kRows + row, pos = p.len - p.count + n / a.G;
            const int from = max(max(nan[0], p.tile0 * kTile), sfar_attn_from(a, pos));
            const int to = min(min(nan[1], pos), (p.tile0 + p.tiles) * kTile - 1);
            for (int j = from; j <= to; ++j) {
                const int page = a.table[(size_t)p.b * a.W + (j >> a.shift)];
                if ((unsigned)page >= (unsigned)a.pages)
                    continue;
                const uint8_t *vp = a.v[r] + ((((long long)page * a.Hk + hk) << a.shift) + (j & ((1 << a.shift) - 1))) * D + col;
#pragma unroll
                for (int e = 0; e < kE; ++e)
                    if ((vp[e] & 0x7f) == 0x7f)
                        all.o[e] = NAN;
            }
        }
        bool write = true;
        if (p.tiles < p.all) {
            // a part: leave it in the workspace, for the last of the row tile's CTAs
            const long long from = u - (p.tile0 - p.begin), to = from + p.all;
            const int c0 = (int)sfar_div((from + 1) * N - 1, U), c1 = (int)sfar_div(to * N - 1, U);
            SfarJoin join(a, 0, c0, c1, blockIdx.x);
            auto slot = [&](int c) { return a.part + ((size_t)c * 2 + (c == c0)) * (kRows * (D + 4)); };
            float *dst = slot(blockIdx.x);
            for (;;) {
                __syncwarp();                      // a row's threads have read what its first one now overwrites
                if (row < rows) {
#pragma unroll
                    for (int e = 0; e < kE; e += 4)
                        __stcg(reinterpret_cast<float4 *>(dst + row * D + col + e),
                               make_float4(all.o[e], all.o[e + 1], all.o[e + 2], all.o[e + 3]));
                    if (col == 0)
                        __stcg(reinterpret_cast<float4 *>(dst + kRows * D + row * 4), make_float4(all.top, all.sum, all.wtop, 0.f));
                }
                consumers_sync();
                if (tid == 0)
                    s_last = join.last();
                consumers_sync();
                write = s_last;
                if (!write)
                    break;
                all = SfarAttnState<kE>();
                // one pass, a batch of parts in flight (the code is as short as its loads allow: it runs once, from a
                // cold instruction cache)
                constexpr int kBatch = 32 / kE;
                const int last = row < rows ? join.hi : join.lo - 1;
#pragma unroll 1
                for (int c = join.lo; c <= last; c += kBatch * join.step) {
                    float4 m[kBatch], v[kBatch][kE / 4];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        m[i] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
                        const int from = c + i * join.step;
                        const float *src = slot(from);
                        if (from <= last)
                            m[i] = __ldcg(reinterpret_cast<const float4 *>(src + kRows * D + row * 4));
#pragma unroll
                        for (int e = 0; e < kE / 4; ++e) {
                            v[i][e] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (from <= last)
                                v[i][e] = __ldcg(reinterpret_cast<const float4 *>(src + row * D + col + 4 * e));
                        }
                    }
                    SfarAttnState<kE> next;
                    next.reference(all.top, all.wtop);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        next.reference(m[i].x, m[i].z);
                    const float keep = next.add(all.top, all.sum, all.wtop);
#pragma unroll
                    for (int e = 0; e < kE; ++e)
                        next.o[e] = all.o[e] * keep;
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const float by = next.add(m[i].x, m[i].y, m[i].z);
#pragma unroll
                        for (int e = 0; e < kE / 4; ++e)
                            next.add4(4 * e, by, v[i][e]);
                    }
                    all = next;
                }
                dst = slot(join.lo);
                if (!join.next(a, 0))
                    break;
            }
        }
        if (write && row < rows) {
            const int n = p.rt * kRows + row;
            const float inv = all.factor();
            uint16_t *dst = a.out[r] + (long long)(p.first + n / a.G) * a.ots + (long long)(hk * a.G + n % a.G) * a.ohs + col;
#pragma unroll
            for (int e = 0; e < kE; e += 4)
                st_v2u32(dst + e, tc::bf16x2(all.o[e] * inv, all.o[e + 1] * inv), tc::bf16x2(all.o[e + 2] * inv, all.o[e + 3] * inv));
        }
        u += p.tiles;
    }
    sfar_attn_padding<D>(a, tid, 32 * kConsumers);
    if (dead && lane == 0)
        sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
}

// rows: 8 or 16 at a time
const void *sfar_kernel_kv_attn(int head_dim, int rows, int *threads, int *smem)
{
#define SFAR_ATTN(D, RH) (*smem = Lay<D, RH>::kBytes + 1024, (const void *)k_kv_attn<D, RH>)
    *threads = kThreads;
    if (rows == 8)
        return head_dim == 64 ? SFAR_ATTN(64, 1) : SFAR_ATTN(128, 1);
    return head_dim == 64 ? SFAR_ATTN(64, 2) : SFAR_ATTN(128, 2);
#undef SFAR_ATTN
}
