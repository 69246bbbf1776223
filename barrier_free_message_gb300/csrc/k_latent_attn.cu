// k_latent_attn.cu -- attention of the step's tokens over the paged latent
// cache, absorbed form (include/sfar_latent.h).
//
// A request's new tokens times all query heads are the rows of one matrix,
// taken 16, 32 or 64 at a time; a cached row serves them all, as key (all its
// numbers) and as value (the latent).  One pass with the running maximum and
// sum of the softmax; per tile of 64 cached tokens, on the tensor cores,
//   S^T = C Q^T   (tokens x rows, contraction over latent + key)
//   O^T += L^T P^T (latent x rows, contraction over the tokens).
// Transposed, because the few rows then are the short side: an MMA takes 64
// tokens or 128 elements of the latent, and both products read the tile from
// shared memory as TMA wrote it, once as the K-major and once as the M-major
// operand.
// HBM-bound: 2 (latent + key) bytes a token against 2 NR (2 latent + key)
// flops, 32 flops a byte at 16 rows.
//
// Softmax: a warp holds 16 tokens' scores, spread as an accumulator's fragment
// (a thread 2 tokens of a quarter of the rows).  A row's reference
// moves only when a score passes it by 2^7.9 (a vote of the CTA's softmax
// threads, no maxima otherwise), and the accumulator is rescaled in tensor
// memory only then.  What a row does not attend to is masked by its place: a
// score of -inf is not that.  Weights go to shared memory as bf16, the type that an
// MMA with these values takes; sums are of the unrounded ones.
//
// Shared memory holds two tiles and more: a ring of pairs of 64-element boxes
// (16 KB) and one of key boxes (8 KB).  A pair is free again when its part of
// the second product is done, so the next tiles stream in while this one is
// multiplied.
//
// Work: as in k_kv_attn.cu the tiles of all (rank, request, row tile) form one
// line that is cut into equal pieces, one per CTA; row tiles cut apart are
// joined by the last of their CTAs, in order.  Prefix sums of 32 requests at a
// time are kept, so that shared memory is the tiles'.
// Warps 0-3: softmax; 4: copies and pieces; 5: the MMAs; 6: query rows, and the
// zeros past the last request.
//
// Measured, latent 512, key 64: 8 ranks, 32 requests of 301 to 6100 tokens, 20
// heads: 964 MB in 165 us, 5.8 TB/s or 0.86 of a copy's rate; 64 requests of 2000,
// 16 heads: 6.0 TB/s; 131071 tokens, 4 ranks, 20 rows: 604 MB in 117 us, 10 of
// them before the first tile and in joins.  Per tile at 32 rows 3400 clocks:
// 1300 of scores, 1260 of softmax and handing over, 600 of products (shared
// memory's rate: both read the whole tile), against 3130 that its bytes take
// at the copy's rate.  64 rows: 4500 to 5200 clocks a tile.
// Tried: the next tile's scores beside this one's softmax (2 to 13% slower, 4%
// faster at 64 rows: the ring holds two tiles and a half); 8 softmax warps at 64
// rows (17% slower); two CTAs of 16 rows to an SM (8% slower); results written
// as pairs exchanged between lanes (10% slower for short contexts).
#include "sfar_attn.cuh"
#include "sfar_latent_args.h"

namespace {

constexpr int kTile = SFAR_LATENT_TILE, kGroup = SFAR_LATENT_GROUP;
constexpr int kSoft = 4, kCopyWarp = kSoft, kMmaWarp = kSoft + 1, kQueryWarp = kSoft + 2, kThreads = 32 * (kQueryWarp + 1);
constexpr int kBox = kTile * 128, kPair = 2 * kBox;                // bytes of 64 elements of every token, of 128
constexpr float kLeast = -3.4028234663852886e38f;                  // the least finite number
constexpr int kMeta = 8, kPieces = 4, kParts = 16, kKept = 64, kWhole = 8;     // kMeta: above the tiles in flight; kParts: joined at once, at most

template <int L, int NR> struct Lay {
    static constexpr int kBlocks = L / 128, kChunks = L / 64 + 1;
    // slots of the rings: what fits
    static constexpr int kPairs = L == 256 ? NR == 64 ? 8 : 9 : NR == 64 ? 7 : 10, kKeys = L == 256 || NR == 16 ? 3 : 2;
    static constexpr int kQ = kChunks * NR * 128, kP = NR * 128;
    static constexpr int oKey = kPairs * kPair, oQ = oKey + kKeys * kBox, oP = oQ + kQ;
    static constexpr int kBytes = oP + kP;
    static constexpr int kNeed = NR + kBlocks * NR, kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;    // tensor memory
    static constexpr int kPart = NR * (L + 2);                     // floats of a partial result
};

// One piece: NR rows of a request and a run of its tiles.
struct Piece {
    int r, b, rt;               // rank; request; row tile
    int tile0, tiles;           // first tile, how many are on the line
    int run;                    // of these, the ones that some row attends to
    int all;                    // tiles of the whole row tile
    int len, count, first;      // context, new tokens, row of the first new token
    long long at;               // place of the piece's first tile on the line
};

struct Request {
    int len, count, first;
};
template <int NR, class A> struct Work {
    const uint32_t *upto;       // [groups + 1] prefix sums of the units of 32 requests, per rank
    const Request *kept;        // the first kKept requests, read once
    const A &a;
    __device__ __forceinline__ int tiles(int len) const { return max(1, (len + kTile - 1) / kTile); }
    __device__ __forceinline__ int row_tiles(int count) const { return (int)(((long long)count * a.Hq + NR - 1) / NR); }
    // by a whole warp
    __device__ __forceinline__ Piece at(long long u, long long end) const
    {
        const int lane = threadIdx.x & 31, groups = (a.B + kGroup - 1) / kGroup;
        Piece p;
        p.at = u;
        const uint32_t S = upto[groups];
        p.r = (int)sfar_div(u, S);
        uint32_t v = (uint32_t)(u - (long long)p.r * S);
        int lo = 0, hi = groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (upto[mid] <= v)
                lo = mid;
            else
                hi = mid;
        }
        v -= upto[lo];
        const int b = lo * kGroup + lane;
        int len = 0, count = 0, first = 0;
        uint32_t sum = 0;
        if (b < a.B) {
            if (b < kKept) {
                len = kept[b].len, count = kept[b].count, first = kept[b].first;
            } else {
                sfar_attn_request(a, b, len, count, first);
            }
            sum = (uint32_t)row_tiles(count) * (uint32_t)tiles(len);
        }
        const uint32_t mine = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(SFAR_FULL, sum, d);
            if (lane >= d)
                sum += o;
        }
        const unsigned past = __ballot_sync(SFAR_FULL, sum > v);
        const int l = past ? __ffs(past) - 1 : 0;
        p.b = lo * kGroup + l;
        p.len = __shfl_sync(SFAR_FULL, len, l);
        p.count = __shfl_sync(SFAR_FULL, count, l);
        p.first = __shfl_sync(SFAR_FULL, first, l);
        const uint32_t w = v - __shfl_sync(SFAR_FULL, sum - mine, l);
        p.all = tiles(p.len);
        p.rt = (int)(w / (uint32_t)p.all);
        p.tile0 = (int)(w - (uint32_t)p.rt * (uint32_t)p.all);
        p.tiles = p.all <= kWhole ? p.all - p.tile0 : (int)min((long long)(p.all - p.tile0), end - u);
        const long long last = min((long long)p.count * a.Hq, ((long long)p.rt + 1) * NR) - 1;       // the row tile's last row
        const int to = p.len - p.count + (int)(last / a.Hq) + 1;                                     // tokens it attends to
        p.run = max(0, min(p.tiles, (max(0, to) + kTile - 1) / kTile - p.tile0));
        return p;
    }
};

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}
// Four 8 x 8 matrices of 16-bit values, in fragments, transposed to rows of 16 bytes: lanes 8 i .. 8 i + 7 give the i-th's.
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// whether one of the two bf16 is an infinity or NaN
__device__ __forceinline__ bool odd2(uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; }

// the larger one, NaN if one is
__device__ __forceinline__ float at_least(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// What a row's accumulator is multiplied by: 0 if it attends to nothing, NaN if all its scores are -inf.
__device__ __forceinline__ float factor(float ref, float sum) { return ref == kLeast ? NAN : sum == 0.f ? 0.f : 1.f / sum; }

// The rows whose accumulator holds an infinity or NaN, by the softmax threads: NaN for their sums, and for their results if
// these have been written.  Puts the flag that brought them here back.
template <int L, int NR> __device__ __noinline__ void odd_rows(uint32_t tO, int rows, float *sum, uint16_t *const *out, int *flag)
{
    for (int again = 0; again < (out ? 2 : 1); ++again) {
        for (int n0 = 0; n0 < rows; n0 += 8)
            for (int c = 0; c < L / 128; ++c) {
                uint32_t o[8];
                tc::ld8(o, tO + c * NR + n0);
                tc::wait_ld(o);
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    if (n0 + n < rows) {
                        if (again == 0 && (o[n] & 0x7f800000u) == 0x7f800000u)
                            sum[n0 + n] = NAN;
                        if (again && isnan(sum[n0 + n]))
                            out[n0 + n][c * 128 + threadIdx.x] = 0x7fff;
                    }
            }
        soft_sync();
        if (threadIdx.x == 0)
            *flag = 0;                             // all have read it; set no sooner than after another barrier
    }
}

// Zeros for the rows past the last request, by a warp of each CTA.
template <int L> __device__ __noinline__ void padding(const SfarLatentAttnArgs &a, int lane)
{
    if (a.starts[a.B] < a.T)
        sfar_attn_padding<L>(a, lane, 32);
}

// Adds up `parts` partial results, the first at p0, the second at p1 and the others `step` floats on from it, each times
// its row's weight w[part][row], by the 128 threads of the softmax: into the first one, or, where out is given, times by[row]
// to the rows of the result.  A thread has kBatch parts of kY rows in flight: time passes by round trips (1.2 us), so few
// parts are taken with more rows.
template <int L, int NR, int kBatch, int kY>
__device__ __forceinline__ void add_parts(float *p0, const float *p1, size_t step, int parts, int rows, const float *w, uint16_t *const *out,
                                          const float *by)
{
    constexpr int kPer = L / 4, kStep = 32 * kSoft / kPer;         // threads of a row, rows at once
    const int d = threadIdx.x % kPer * 4;
#pragma unroll 1
    for (int n0 = threadIdx.x / kPer; n0 < rows; n0 += kY * kStep) {
        float4 o[kY];
        int at[kY];                                // rows past the last: the last again
#pragma unroll
        for (int y = 0; y < kY; ++y) {
            o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            at[y] = min(n0 + y * kStep, rows - 1);
        }
#pragma unroll 1
        for (int c0 = 0; c0 < parts; c0 += kBatch) {
            float4 v[kBatch][kY];
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                const int part = min(c0 + c, parts - 1);           // parts past the last: the last again, not added
                const float *src = (part == 0 ? p0 : p1 + (size_t)(part - 1) * step) + d;
#pragma unroll
                for (int y = 0; y < kY; ++y)
                    v[c][y] = __ldcg(reinterpret_cast<const float4 *>(src + at[y] * L));
            }
#pragma unroll
            for (int c = 0; c < kBatch; ++c)
                if (c0 + c < parts)
#pragma unroll
                    for (int y = 0; y < kY; ++y) {
                        const float f = w[(c0 + c) * NR + at[y]];
                        o[y].x += f * v[c][y].x;
                        o[y].y += f * v[c][y].y;
                        o[y].z += f * v[c][y].z;
                        o[y].w += f * v[c][y].w;
                    }
        }
#pragma unroll
        for (int y = 0; y < kY; ++y) {
            const int n = n0 + y * kStep;
            if (n >= rows)
                break;
            if (out) {
                const float f = by[n];
                st_v2u32(out[n] + d, tc::bf16x2(o[y].x * f, o[y].y * f), tc::bf16x2(o[y].z * f, o[y].w * f));
            } else {
                __stcg(reinterpret_cast<float4 *>(p0 + n * L + d), o[y]);
            }
        }
    }
}
// out of line, so that the kernel's loops keep their registers
template <int L, int NR>
__device__ __noinline__ void add_parts(float *p0, const float *p1, size_t step, int parts, int rows, const float *w, uint16_t *const *out,
                                       const float *by)
{
    if (parts <= 2)
        add_parts<L, NR, 2, 12>(p0, p1, step, parts, rows, w, out, by);
    else if (parts <= 4)
        add_parts<L, NR, 4, 7>(p0, p1, step, parts, rows, w, out, by);
    else
        add_parts<L, NR, 8, 4>(p0, p1, step, parts, rows, w, out, by);
}

}  // namespace

template <int L, int NR> __global__ void __launch_bounds__(kThreads, 1) k_latent_attn(const __grid_constant__ SfarLatentAttnArgs a)
{
    using Y = Lay<L, NR>;
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ __align__(8) unsigned long long bars[2 * Y::kPairs + 2 * Y::kKeys + 2 * kPieces + 6];
    __shared__ Piece s_piece[kPieces];             // what the copying warp has begun with; no tiles: the end
    __shared__ uint32_t s_live[kMeta];             // of a tile: which 16 places hold a token on a page of the pool
    __shared__ uint32_t upto[SFAR_KV_MAX_REQUESTS / kGroup + 1];
    __shared__ Request s_kept[kKept];
    __shared__ uint32_t s_warp[kThreads / 32], s_tmem;
    __shared__ int s_hi[NR], s_last, s_odd;
    __shared__ float s_max[kSoft][NR], s_sum[NR], s_ref[NR], s_keep[NR], s_inv[NR], s_w[kParts][NR], s_m[kParts][NR];
    __shared__ uint16_t *s_out[NR];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t mem = (tc::smem(dyn) + 1023u) & ~1023u;
    unsigned char *gen = dyn + (mem - tc::smem(dyn));
    const uint32_t full = tc::smem(bars), empty = full + 8 * Y::kPairs, kfull = empty + 8 * Y::kPairs, kempty = kfull + 8 * Y::kKeys,
                   pfull = kempty + 8 * Y::kKeys, pempty = pfull + 8 * kPieces, qbar = pempty + 8 * kPieces, sbar = qbar + 8, wbar = qbar + 16,
                   obar = qbar + 24, qempty = qbar + 32, drain = qbar + 40;

    if (warp == kCopyWarp && lane < a.R)
        tc::prefetch_map(&a.map[lane]);
    if (warp == kQueryWarp && lane < a.R && a.q_flat)
        tc::prefetch_map(&a.qmap[lane]);
    if (tid == 0) {
        for (uint32_t b = full; b <= drain; b += 8)
            tc::bar_init(b, b >= pempty && b < qbar ? kSoft + 2 : b == qbar ? 32 : b == wbar ? kSoft : 1);
        tc::bar_fence_init();
        tc::fence_async();
        upto[0] = 0;
        s_odd = 0;
    }
    if (warp == kMmaWarp)
        tc::tmem_alloc<1>(tc::smem(&s_tmem), Y::kCols);
    pdl_wait();
    const unsigned long long limit = ld_relaxed_u64(&a.ctl->timeout_ns);

    // prefix sums of the requests' units: row tiles x tiles, 32 requests to a warp
    const Work<NR, SfarLatentAttnArgs> work{upto, s_kept, a};
    uint32_t carry = 0;
    int row_tiles = 0;                             // of this thread's requests
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        uint32_t v = 0;
        if (b < a.B) {
            int len, count, first;
            sfar_attn_request(a, b, len, count, first);
            if (b < kKept)
                s_kept[b] = Request{len, count, first};
            const int n = work.row_tiles(count);
            v = (uint32_t)n * (uint32_t)work.tiles(len);
            row_tiles = min(row_tiles + n, 1 << 26);       // above any step's; 32 such sums fit 32 bits
            if (blockIdx.x == 0)
                sfar_attn_check(a, b, len, count, first);
        }
        v = __reduce_add_sync(SFAR_FULL, v);
        if (lane == 0)
            s_warp[warp] = v;
        __syncthreads();
        uint32_t before = carry;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            carry += s_warp[w];
            if (w <= warp)
                before += s_warp[w];
        }
        if (lane == 0 && b < a.B)
            upto[b / kGroup + 1] = before;
        __syncthreads();
    }
    row_tiles = __reduce_add_sync(SFAR_FULL, row_tiles);
    if (lane == 0)
        s_warp[warp] = (uint32_t)row_tiles;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    long long whole = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
        whole += s_warp[w];
    // Row tiles of up to 8 tiles are left whole (34 requests of 127 tokens, 22 heads, 8 ranks: 28 us cut in equal pieces, 19 so:
    // joining two parts costs what four tiles do), longer ones in cuts of no less than four.
    const long long U = sfar_attn_many(a, whole) ? 0 : (long long)carry * a.R;
    const long long N = min(min((long long)gridDim.x, U), max(whole * a.R, U / 4));
    const long long u0 = blockIdx.x < N ? sfar_div(blockIdx.x * U, N) : 0, u1 = blockIdx.x < N ? sfar_div((blockIdx.x + 1) * U, N) : 0;

    if (warp < kSoft) {
        // -------------------------------------------------------------- softmax
        bool dead = false;                         // a wait gave up: go on without waiting
        const uint32_t lanes = (uint32_t)warp * 32u << 16, tS = tmem + lanes, tO = tmem + NR + lanes;
        // of a tile, token 16 warp + g + 8 h of rows 8 i + 2 t + y is x[4 i + 2 h + y]; of a block of the latent, element tid
        const int g = lane >> 2, t = lane & 3;
        constexpr int kI = NR / 8;
        const float f = a.scale * 1.4426950408889634f;
        // where a lane's row of the transposed weights goes: P[row][64 tokens], 128-byte swizzle; matrices (i, h) of two i at once
        const uint32_t pw = mem + Y::oP + ((lane >> 4) * 8 + (lane & 7)) * 128 + (((2 * warp + (lane >> 3 & 1)) ^ (lane & 7)) << 4);
        tc::Ring<kPieces> ps;
        tc::Ring<Y::kPairs> st;                    // the first pair of the tile
        uint32_t sphase = 0, ophase = 0, tile = 0;
        // The next piece, by all softmax warps alike; false: the end, or a wait that gave up.  It is read where the copying
        // warp has put it, and given back when it has been written out.
        auto take = [&](int &at) {
            dead = dead || !tc::bar_wait(pfull + 8 * ps.slot, ps.phase, limit);
            if (soft_any(dead)) {
                dead = true;
                return false;
            }
            at = (int)ps.slot;
            ps.next();
            return s_piece[at].tiles != 0;
        };
        int now_at = 0;
        while (take(now_at)) {
            const Piece &p = s_piece[now_at];
            const int row0 = p.rt * NR, rows = (int)min((long long)NR, (long long)p.count * a.Hq - row0);
            if (tid < NR) {
                const int n = row0 + min(tid, rows - 1), i = n / a.Hq, h = n - i * a.Hq;
                s_hi[tid] = p.len - p.count + i + 1;
                s_out[tid] = a.out[p.r] + (long long)(p.first + i) * a.ots + h * a.ohs;
            }
            soft_sync();                           // s_hi, s_out
            const int all_to = s_hi[0];            // every row sees the tokens before it
            float ref[2 * kI], sum[2 * kI];        // of rows 8 i + 2 t + y
#pragma unroll
            for (int n = 0; n < 2 * kI; ++n) {
                ref[n] = -INFINITY;
                sum[n] = 0.f;
            }
            const int run = p.run, j00 = p.tile0 * kTile, len = p.len;
            for (int k = 0; k < run; ++k, ++tile) {
                const int j0 = j00 + k * kTile, j = j0 + 16 * warp + g;
                dead = dead || !tc::bar_wait(sbar, sphase, limit) || !tc::bar_wait(full + 8 * st.slot, st.phase, limit);
                sphase ^= 1u;
                tc::fence_after();
                uint32_t raw[4 * kI];
                tc::ld_rows(raw, tS);
                tc::wait_ld(raw);
                const uint32_t live = s_live[tile % kMeta];
                const bool edge = j0 + kTile > all_to || live != 0xfu, none = warp && !(live >> warp & 1u);
                bool there[2] = {true, true}, odd[2] = {false, false};
                if (edge) {
                    // A place that holds no token becomes zeros, whatever lies there (16 without one are left out of the
                    // product, but for the first); so does a token with an infinity or NaN that not every row sees, and the
                    // rows that do see it get a NaN for its weight.  Two threads to a token of the warp's 16, a box of every
                    // pair each.
                    const int mine = 16 * warp + (lane >> 1);
                    const bool on = live >> warp & 1u, here = on && j0 + mine < len;
                    bool bad = false;
                    tc::Ring<Y::kPairs> it = st;
                    for (int c = 0; c < Y::kBlocks; ++c, it.next()) {
                        dead = dead || !tc::bar_wait(full + 8 * it.slot, it.phase, limit);
                        if (here && j0 + mine >= all_to) {
                            const unsigned char *at = gen + it.slot * kPair + (lane & 1) * kBox + mine * 128;
                            for (int i = 0; i < 8; ++i) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(at + ((i ^ (mine & 7)) << 4));
                                bad = bad || odd2(v.x) || odd2(v.y) || odd2(v.z) || odd2(v.w);
                            }
                        }
                    }
                    const uint32_t bads = __ballot_sync(SFAR_FULL, bad);
                    it = st;
                    for (int c = 0; c < Y::kBlocks; ++c, it.next())
                        if (!none && (!here || (bads >> (lane & 30) & 3u))) {
                            unsigned char *at = gen + it.slot * kPair + (lane & 1) * kBox + mine * 128;
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<uint4 *>(at + ((i ^ (mine & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        there[h] = on && j + 8 * h < len;
                        odd[h] = bads >> (2 * (g + 8 * h)) & 3u;
                    }
                }
                for (int c = 0; c < Y::kBlocks; ++c)
                    st.next();
                // Scores in units of log2; -inf: not attended to.  A score of -inf that is attended to has weight 0, too, but a
                // row that has such scores alone is NaN: they count as the least finite number for its reference.
                float x[4 * kI];
                bool move = false;
                const float least = edge ? -INFINITY : kLeast;
#pragma unroll
                for (int n = 0; n < 4 * kI; ++n)
                    x[n] = __uint_as_float(raw[n]) * f;
                if (edge) {
#pragma unroll
                    for (int i = 0; i < kI; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int hi = s_hi[8 * i + 2 * t + y];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float &v = x[4 * i + 2 * h + y];
                                v = !there[h] || j + 8 * h >= hi ? -INFINITY : at_least(v, kLeast);
                            }
                        }
                }
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        move |= fmaxf(fmaxf(x[4 * i + y], x[4 * i + 2 + y]), least) - ref[2 * i + y] > kAttnLift;
                if (soft_any(move)) {
#pragma unroll
                    for (int i = 0; i < kI; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float m = fmaxf(fmaxf(x[4 * i + y], x[4 * i + 2 + y]), least);
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1)
                                m = fmaxf(m, __shfl_xor_sync(SFAR_FULL, m, d));
                            if (g == 0)
                                s_max[warp][8 * i + 2 * t + y] = m;
                        }
                    soft_sync();
#pragma unroll
                    for (int i = 0; i < kI; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int n = 8 * i + 2 * t + y, e = 2 * i + y;
                            const float now = fmaxf(fmaxf(s_max[0][n], s_max[1][n]), fmaxf(s_max[2][n], s_max[3][n]));
                            const float next = now - ref[e] > kAttnLift ? now : ref[e];
                            const float keep = ref[e] == -INFINITY ? 1.f : ex2(ref[e] - next);     // all is 0 then, or NaN
                            ref[e] = next;
                            sum[e] *= keep;
                            if (warp == 0 && g == 0)
                                s_keep[n] = keep;
                        }
                    soft_sync();                   // s_max has been read, s_keep is there until the next move's first barrier
                    if (k) {
#pragma unroll 1
                        for (int n = 0; n < Y::kBlocks * NR; n += 16) {
                            uint32_t o[16];
                            tc::ld16(o, tO + n);
                            tc::wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * s_keep[n % NR + e]);
                            tc::st16(tO + n, o);
                        }
                        tc::wait_st();
                    }
                }
                uint32_t w[2 * kI];                // weights of rows 8 i + 2 t and + 1: w[2 i + h]
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float e[2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float v = x[4 * i + 2 * h + y];
                            e[y] = ex2(v - ref[2 * i + y]);
                            if (edge) {
                                e[y] = v == -INFINITY ? 0.f : e[y];
                                if (odd[h] && j + 8 * h < s_hi[8 * i + 2 * t + y])
                                    e[y] = NAN;
                            }
                            sum[2 * i + y] += e[y];
                        }
                        w[2 * i + h] = tc::bf16x2(e[0], e[1]);
                    }
#pragma unroll
                for (int i = 0; i < kI; i += 2)
                    store_transposed(pw + i * 1024, w[2 * i], w[2 * i + 1], w[2 * i + 2], w[2 * i + 3]);
                tc::fence_async();
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(wbar);
            }
            // the rows' sums
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float v = sum[2 * i + y];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1)
                        v += __shfl_xor_sync(SFAR_FULL, v, d);
                    if (g == 0) {
                        s_max[warp][8 * i + 2 * t + y] = v;
                        if (warp == 0)
                            s_ref[8 * i + 2 * t + y] = ref[2 * i + y];
                    }
                }
            soft_sync();
            if (tid < NR) {
                const float v = (s_max[0][tid] + s_max[1][tid]) + (s_max[2][tid] + s_max[3][tid]);
                s_sum[tid] = v;
                s_inv[tid] = factor(s_ref[tid], v);
            }
            soft_sync();
            if (p.run) {
                dead = dead || !tc::bar_wait(obar, ophase, limit);
                ophase ^= 1u;
                tc::fence_after();
            }
            // A row that attends to a latent that is not finite is NaN.  Where the token's weight is 0, only the accumulator's
            // element says so.
            uint64_t odd[Y::kBlocks] = {};         // NaN: some element is not finite, maybe of a row past the request's
            // The accumulator, element tid of each 128 of the latent, a row at a time.  begin(n): what is read once for a row.
            auto each = [&](auto begin, auto what) {
#pragma unroll 1
                for (int n0 = 0; n0 < rows; n0 += 8) {
                    decltype(begin(0)) of[8];
#pragma unroll
                    for (int n = 0; n < 8; ++n)
                        of[n] = begin(n0 + n);
                    uint32_t o[Y::kBlocks][8];
#pragma unroll
                    for (int c = 0; c < Y::kBlocks; ++c)
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            o[c][n] = 0;
                    if (run) {
#pragma unroll
                        for (int c = 0; c < Y::kBlocks; ++c)
                            tc::ld8(o[c], tO + c * NR + n0);
#pragma unroll
                        for (int c = 0; c < Y::kBlocks; ++c)
                            tc::wait_ld(o[c]);
                    }
#pragma unroll
                    for (int n = 0; n < 8; n += 2)
#pragma unroll
                        for (int c = 0; c < Y::kBlocks; ++c)
                            odd[c] = tc::fma2(tc::pack2u(o[c][n], o[c][n + 1]), 0ull, odd[c]);
#pragma unroll
                    for (int n = 0; n < 8; ++n)
                        if (n0 + n < rows) {
#pragma unroll
                            for (int c = 0; c < Y::kBlocks; ++c) {
                                what(of[n], n0 + n, c * 128 + tid, __uint_as_float(o[c][n]));
                            }
                        }
                }
            };
            // a barrier, too (a flag in shared memory beside one takes less than a vote)
            auto any_odd = [&] {
                float all = 0.f;
#pragma unroll
                for (int c = 0; c < Y::kBlocks; ++c)
                    all += tc::unpack2(odd[c]).x + tc::unpack2(odd[c]).y;
                if (all != 0.f)
                    s_odd = 1;
                soft_sync();
                return s_odd != 0;
            };
            if (p.tiles == p.all) {
                struct Row {
                    uint16_t *out;
                    float by;
                };
                each([&](int n) { return Row{s_out[n], s_inv[n]}; },
                     [&](const Row &r, int, int d, float v) { r.out[d] = (uint16_t)tc::bf16x2(v * r.by, 0.f); });
                if (any_odd())                     // the tables in shared memory have been read
                    odd_rows<L, NR>(tO, rows, s_sum, s_out, &s_odd);
            } else {
                // a part: leave it in the workspace, for the last of the row tile's CTAs
                const long long from = p.at - p.tile0, to = from + p.all;
                const int c0 = (int)sfar_div((from + 1) * N - 1, U), c1 = (int)sfar_div(to * N - 1, U);
                SfarJoin join(a, 0, c0, c1, blockIdx.x, kParts);
                auto slot = [&](int c) { return a.part + ((size_t)c * 2 + (c == c0)) * Y::kPart; };
                float *dst = slot(blockIdx.x);
                each([](int) { return 0; }, [&](int, int n, int d, float v) { __stcg(dst + n * L + d, v); });
                auto leave = [&] {
                    if (tid < rows)
                        __stcg(reinterpret_cast<float2 *>(dst + NR * L) + tid, make_float2(s_ref[tid], s_sum[tid]));
                };
                leave();
                if (any_odd()) {
                    odd_rows<L, NR>(tO, rows, s_sum, nullptr, &s_odd);
                    leave();
                    soft_sync();
                }
                for (;;) {
                    if (tid == 0)
                        s_last = join.last();
                    soft_sync();
                    if (!s_last)
                        break;
                    const int parts = (join.hi - join.lo) / join.step + 1;
                    // references and sums of all parts at once, then what each part's rows are multiplied by
                    for (int i = tid; i < parts * NR; i += 32 * kSoft) {
                        const int c = i / NR, n = i % NR;
                        const float2 m = n < rows ? __ldcg(reinterpret_cast<const float2 *>(slot(join.lo + c * join.step) + NR * L) + n)
                                                  : make_float2(-INFINITY, 0.f);
                        s_w[c][n] = m.x;
                        s_m[c][n] = m.y;
                    }
                    soft_sync();
                    float top = -INFINITY, total = 0.f;
                    if (tid < NR) {
                        for (int c = 0; c < parts; ++c)
                            top = fmaxf(top, s_w[c][tid]);
                        for (int c = 0; c < parts; ++c) {
                            const float m = s_w[c][tid], w = m == -INFINITY ? 0.f : ex2(m - top);
                            s_w[c][tid] = w;
                            total += m == -INFINITY ? s_m[c][tid] : w * s_m[c][tid];        // its sum is 0 then, or NaN
                        }
                        s_inv[tid] = factor(top, total);
                    }
                    soft_sync();
                    float *group = slot(join.lo);
                    const bool more = join.up != 0;
                    add_parts<L, NR>(slot(join.lo), slot(join.lo + join.step), (size_t)join.step * 2 * Y::kPart, parts, rows, &s_w[0][0],
                                     more ? nullptr : s_out, s_inv);
                    if (more && tid < rows)
                        __stcg(reinterpret_cast<float2 *>(group + NR * L) + tid, make_float2(top, total));
                    if (!join.next(a, 0))
                        break;
                    soft_sync();
                }
                soft_sync();                       // the tables in shared memory have been read
            }
            tc::fence_before();                    // before the MMAs that the next weights allow
            if (lane == 0)
                tc::bar_arrive(pempty + 8 * now_at);
        }
        if (dead && lane == 0)
            sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
    } else if (warp == kCopyWarp) {
        // --------------------------------------------------------------- copies
        const uint64_t once = tc::evict_first(), often = tc::evict_last();
        // by all lanes alike
        auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(SFAR_FULL, tc::bar_wait(bar, parity, limit)); };
        tc::Ring<Y::kPairs> st;
        tc::Ring<Y::kKeys> ks;
        tc::Ring<kPieces> ps;
        bool dead = false;
        uint32_t pairs = 0, keys = 0, tile = 0;    // issued
        const int per = min(1 << a.shift, kTile), boxes = kTile / per;     // tokens of one copy, copies of a tile's 64 elements
        for (long long u = u0; !dead;) {
            Piece p;
            p.tiles = 0;
            const bool end = u >= u1;
            if (!end) {
                p = work.at(u, u1);
                if (p.tile0 && p.all <= kWhole) {
                    u += p.tiles;                  // a short row tile is the CTA's that has its first tile
                    continue;
                }
            }
            if (!wait(pempty + 8 * ps.slot, ps.phase ^ 1u)) {
                dead = true;
                break;
            }
            if (lane == 0) {
                s_piece[ps.slot] = p;
                tc::bar_arrive(pfull + 8 * ps.slot);
            }
            ps.next();
            if (end)
                break;
            u += p.tiles;
            const int *row = a.table + (size_t)p.b * a.W;
            const CUtensorMap *map = &a.map[p.r];
            const uint64_t pol = (long long)p.count * a.Hq <= NR ? once : often;     // other row tiles read it again
            // lane i: the page of copy i, of 32 copies from token `base` on
            auto pages = [&](int base) {
                const unsigned j = (unsigned)base + (unsigned)(lane * per);      // may pass 2^31
                int page = 0;
                if (j < (unsigned)p.len && j < (unsigned)(p.tile0 + p.run) * (unsigned)kTile)
                    page = row[j >> a.shift];
                return page;
            };
            const int stretch = 32 * per;
            int base = p.tile0 * kTile, page = pages(base), next = pages(base + stretch);
            for (int k = 0; k < p.run && !dead; ++k) {
                const int j0 = (p.tile0 + k) * kTile;
                if (j0 - base >= stretch) {
                    base += stretch;
                    page = next;
                    next = pages(base + stretch);
                }
                // lane i: copy i % 4 of the tile, of the first or second 64 elements of a pair
                const int box = lane & 3, at = (j0 - base) / per + box, j = j0 + box * per;
                const int mine = __shfl_sync(SFAR_FULL, page, at & 31), y = j & ((1 << a.shift) - 1);
                const bool live = box < boxes && j < p.len, bad = live && (unsigned)mine >= (unsigned)a.pages, go = live && !bad;
                if (bad && lane < 4)
                    sfar_kv_fault(a.ctl, p.b, SFAR_KV_BAD_PAGE);
                const unsigned any = __ballot_sync(SFAR_FULL, go) & 0xfu;
                const unsigned held = __ballot_sync(SFAR_FULL, lane < 4 && (any >> (lane * 16 / per) & 1u) && j0 + lane * 16 < p.len);
                if (lane == 0)
                    s_live[tile % kMeta] = held;
                __syncwarp();
                ++tile;
                const uint32_t bytes = (uint32_t)__popc(any) * per * 128;
                for (int c = 0; c < Y::kBlocks; ++c) {
                    if (!wait(empty + 8 * st.slot, st.phase ^ 1u)) {
                        dead = true;
                        break;
                    }
                    const uint32_t bar = full + 8 * st.slot;
                    if (go && lane < 8)
                        tc::load_3d(mem + st.slot * kPair + (lane >> 2) * kBox + box * per * 128, map, c * 128 + (lane >> 2) * 64, y, mine, bar, pol);
                    __syncwarp();
                    if (lane == 0)
                        tc::bar_expect(bar, 2 * bytes);
                    ++pairs;
                    st.next();
                }
                if (dead)
                    break;
                if (!wait(kempty + 8 * ks.slot, ks.phase ^ 1u)) {
                    dead = true;
                    break;
                }
                const uint32_t bar = kfull + 8 * ks.slot;
                if (go && lane < 4)
                    tc::load_3d(mem + Y::oKey + ks.slot * kBox + box * per * 128, map, L, y, mine, bar, pol);
                __syncwarp();
                if (lane == 0)
                    tc::bar_expect(bar, bytes);
                ++keys;
                ks.next();
            }
        }
        if (dead && lane == 0) {
            sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
            // the copies in flight land before the shared memory is released
            for (uint32_t i = pairs - min(pairs, (uint32_t)Y::kPairs); i < pairs; ++i)
                tc::bar_wait(full + 8 * (i % Y::kPairs), (i / Y::kPairs) & 1u, limit);
            for (uint32_t i = keys - min(keys, (uint32_t)Y::kKeys); i < keys; ++i)
                tc::bar_wait(kfull + 8 * (i % Y::kKeys), (i / Y::kKeys) & 1u, limit);
        }
    } else if (warp == kQueryWarp) {
        // -------------------------------------------------------------- queries
        // A piece's query rows: [chunk][row][64 elements], 128-byte swizzle; zeros past the rows and past a short key.
        const uint64_t once = tc::evict_first();
        tc::Ring<kPieces> ps;
        uint32_t phase = 1, asked = 0;
        bool dead = false;
        for (;;) {
            dead = !__all_sync(SFAR_FULL, tc::bar_wait(pfull + 8 * ps.slot, ps.phase, limit));
            if (dead || s_piece[ps.slot].tiles == 0)
                break;
            const Piece &p = s_piece[ps.slot];
            if (p.run) {
                // the last piece's scores have been formed
                dead = !__all_sync(SFAR_FULL, tc::bar_wait(qempty, phase, limit));
                phase ^= 1u;
                if (dead)
                    break;
                const int row0 = p.rt * NR;
                ++asked;
                if (a.q_flat) {
                    // rows one stride apart: a copy to 64 elements of all (those past the request's are others', and not written out)
                    if (lane == 0)
                        tc::bar_expect_only(qbar, Y::kQ);
                    __syncwarp();
                    if (lane < Y::kChunks)
                        tc::load_2d(mem + Y::oQ + lane * (NR * 128), &a.qmap[p.r], 64 * lane, p.first * a.Hq + row0, qbar, once);
                } else {
                    constexpr int kVecs = Y::kChunks * 8, kEach = NR < 32 ? NR : 32;
                    const int rows = (int)min((long long)NR, (long long)p.count * a.Hq - row0);
                    for (int m = 0; m < NR; m += kEach) {
                        // lane i: where row m + i comes from
                        const int row = row0 + min(m + lane, rows - 1), i = row / a.Hq;
                        const uint16_t *src = a.q[p.r] + (long long)(p.first + i) * a.qts + (long long)(row - i * a.Hq) * a.qhs;
#pragma unroll 4
                        for (int e = lane; e < kEach * kVecs; e += 32) {
                            const int y = e / kVecs, c = e - y * kVecs, n = m + y;
                            const uint16_t *from = reinterpret_cast<const uint16_t *>(__shfl_sync(SFAR_FULL, (unsigned long long)src, y));
                            const bool in = n < rows && c * 8 < L + a.rope;
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(mem + Y::oQ + (c >> 3) * (NR * 128) + n * 128 +
                                                                                              (((c & 7) ^ (n & 7)) << 4)),
                                         "l"(in ? from + c * 8 : from), "r"(in ? 16u : 0u)
                                         : "memory");
                        }
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    tc::fence_async();
                }
                tc::bar_arrive(qbar);
            }
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(pempty + 8 * ps.slot);
            ps.next();
        }
        if (dead && lane == 0) {
            sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
            if (asked)                             // the copies in flight land before the shared memory is released
                tc::bar_wait(qbar, (asked - 1) & 1u, limit);
        }
        padding<L>(a, lane);
    } else {
        // ----------------------------------------------------------------- MMAs
        constexpr uint32_t idS = tc::idesc_bf16(64, NR), idO = tc::idesc_bf16(128, NR) | tc::kTransposeA;
        const uint64_t dq = tc::desc_k128(mem + Y::oQ), dp = tc::desc_k128(mem + Y::oP), dk = tc::desc_k128(mem), dv = tc::desc_n128(mem, kBox),
                       dr = tc::desc_k128(mem + Y::oKey);
        tc::Ring<Y::kPairs> st;
        tc::Ring<Y::kKeys> ks;
        tc::Ring<kPieces> ps;
        uint32_t qphase = 0, wphase = 0, tile = 0;
        bool dead = false;
        if (tc::elect_one()) {                     // all by one lane
            int run = 0, tiles = 0;
            auto take = [&]() {
                dead = !tc::bar_wait(pfull + 8 * ps.slot, ps.phase, limit);
                if (!dead) {
                    run = s_piece[ps.slot].run;
                    tiles = s_piece[ps.slot].tiles;
                    tc::bar_arrive(pempty + 8 * ps.slot);
                    ps.next();
                }
            };
            take();
            while (!dead && tiles) {
                if (run == 0) {
                    take();
                    continue;
                }
                dead = !tc::bar_wait(qbar, qphase, limit);
                qphase ^= 1u;
                const int now = run;
                for (int k = 0; k < now && !dead; ++k) {
                    tc::Ring<Y::kPairs> it = st;
#pragma unroll
                    for (int c = 0; c < Y::kBlocks; ++c, it.next()) {
                        dead = dead || !tc::bar_wait(full + 8 * it.slot, it.phase, limit);
                        if (dead)
                            break;
                        tc::fence_after();
                        const uint64_t d = dk + it.slot * (kPair >> 4);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            tc::mma_f16_ss(tmem, d + (i >> 2) * (kBox >> 4) + 2 * (i & 3), dq + (2 * c + (i >> 2)) * (NR * 128 >> 4) + 2 * (i & 3), idS,
                                           c + i > 0);
                    }
                    dead = dead || !tc::bar_wait(kfull + 8 * ks.slot, ks.phase, limit);
                    if (dead)
                        break;
                    for (int i = 0; i < a.rope / 16; ++i)
                        tc::mma_f16_ss(tmem, dr + ks.slot * (kBox >> 4) + 2 * i, dq + (L / 64) * (NR * 128 >> 4) + 2 * i, idS, true);
                    tc::commit(kempty + 8 * ks.slot);
                    tc::commit(sbar);
                    ks.next();
                    if (k == now - 1) {
                        tc::commit(qempty);
                        take();                    // the next piece, beside the softmax
                    }
                    dead = dead || !tc::bar_wait(wbar, wphase, limit);
                    wphase ^= 1u;
                    if (dead)
                        break;
                    tc::fence_after();
                    const uint32_t live = s_live[tile++ % kMeta] | 1u;
#pragma unroll
                    for (int c = 0; c < Y::kBlocks; ++c, st.next()) {
#pragma unroll
                        for (int i = 0; i < kTile / 16; ++i)
                            if (live >> i & 1u)
                                tc::mma_f16_ss(tmem + NR + c * NR, dv + st.slot * (kPair >> 4) + 128 * i, dp + 2 * i, idO, k + i > 0);
                        tc::commit(empty + 8 * st.slot);
                    }
                }
                if (!dead)
                    tc::commit(obar);
            }
        }
        __syncwarp();
        dead = __any_sync(SFAR_FULL, dead);
        if (tc::elect_one()) {
            if (dead)
                sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
            // every MMA and every arrival it causes is done before the CTA leaves
            tc::commit(drain);
            tc::bar_wait(drain, 0, limit);
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp)
        tc::tmem_free<1>(tmem, Y::kCols);
}

const void *sfar_kernel_latent_attn(int latent, int rows, int *threads, int *smem)
{
#define SFAR_LATENT(L, NR) (*smem = Lay<L, NR>::kBytes + 1024, (const void *)k_latent_attn<L, NR>)
    *threads = kThreads;
    if (rows == 16)
        return latent == 256 ? SFAR_LATENT(256, 16) : SFAR_LATENT(512, 16);
    if (rows == 32)
        return latent == 256 ? SFAR_LATENT(256, 32) : SFAR_LATENT(512, 32);
    return latent == 256 ? SFAR_LATENT(256, 64) : SFAR_LATENT(512, 64);
#undef SFAR_LATENT
}
