// k_kv_prompt.cu -- attention of the step's tokens over the paged 8-bit cache
// (include/sfar_kv.h), for many query rows per request: chunks of prompts.
//
// The same rows, softmax and references as k_kv_attn.cu, on the tensor cores:
// per 128 rows and 128 cached tokens S = Q K^T and O += W V, both accumulated
// in tensor memory.  Compute-bound: 4 D flops per visible (row, token).
//
// Operands.  Keys are used as they lie in the cache, e4m3; the query row,
// scaled by a power of two to a largest magnitude in [128, 256), is split into
// two e4m3 numbers: the leading 4 of bf16's 8 significant bits, and the other
// 4.  The split is exact for elements down to 2^-9 of the row's largest and
// off by at most 2^-17 of that below; two e4m3 products cost what one binary16
// product would, and the keys need no conversion.  Values are widened to
// binary16 (exact) by two warps, once for the 256 rows that share them; the
// weights are rounded to binary16 and are the operand in tensor memory, in the
// place of the scores they come from.  One running reference serves weights
// and sum, the weights' (score times value scale), and the sum is of weight /
// value scale: nothing is lost while the value scales of one request are
// within 2^100 of one another.  Tokens of value scale 0 have no weight; their
// exponentials have a reference and a sum of their own, joined at the end.  The
// accumulator is rescaled, in tensor memory, only when a reference moves.
//
// A CTA takes 256 rows as two tiles of 128, each with eight softmax warps (two
// threads per row, a half of its columns each: the row's maximum needs one
// exchange and no shuffles).  The tensor core alternates: while it runs
// O_B += W_B V and S_B = Q_B K' of one tile, the other's softmax works.
// Warps 0-15: softmax; 16, 17: values widened; 18: copies, page scales and
// queries; 19: the MMAs.
//
// Work: as in k_kv_attn.cu the tiles of all (rank, key head, request, 256
// rows) form one line, cut into one equal piece per SM; row tiles cut apart
// are joined by the last of their CTAs, in order.
//
// Measured, 8 ranks of 8 query heads and one key head of 128, three chunks of
// 700 to 1024 new tokens at the ends of contexts of 1100 to 4099: 203 us, 1080
// TFLOP/s, 0.55 of a bf16 product's rate; the tensor core is busy 0.50 of the
// time.  A tile's chain is what bounds it: about 2000 clocks from scores to
// weights (maxima 400, the warps' agreement on the reference 300, exponentials
// 930, masks and stores the rest) against 1088 of products, which two tiles in
// flight only just cover.  One thread per row took 288 us, scores kept in
// registers over the agreement spilled and took 771 (what is left spills 8 to 12
// bytes of 96 registers a thread).
#include "sfar_e4m3.cuh"
#include "sfar_attn.cuh"
#include "sfar_tc.cuh"

namespace {

constexpr int kTile = 128;                         // cached tokens per step
constexpr int kRows = SFAR_PROMPT_ROWS;            // query rows per CTA: two tiles of 128
constexpr int kSoft = 16;                          // softmax warps
constexpr int kWiden = 2, kCopyWarp = kSoft + kWiden, kMmaWarp = kCopyWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kOver = 6;                           // what a row tile costs beside its tiles, in tiles
constexpr float kSumUp = 20.f, kSumDown = 0x1p-20f;    // the sum is kept 2^20 down: so it holds scales from 2^-100 to 2^100
constexpr int kKStages = 3, kVStages = 2, kHStages = 2, kMeta = 4, kPieces = 8;

template <int D> struct Lay {
    static constexpr int kK = kTile * D, kH = kTile * D * 2, kQ = 128 * D;
    static constexpr int oK = 0, oV = oK + kKStages * kK, oH = oV + kVStages * kK, oQ = oH + kHStages * kH;
    static constexpr int kBytes = oQ + 4 * kQ;     // queries: two tiles, nearest and rest
};
struct Meta {                                      // of a step
    // each 16 tokens: key scale, log2 of the value scale (-inf for 0), kSumDown over the value scale (0 for 0)
    float ks[kTile / 16], lvs[kTile / 16], ivs[kTile / 16];
    // bit i: tokens 16 i .. are on no page of the pool; 8: a key scale is negative; 16 + i: tokens' value scale is 0 (they
    // have no weight and are summed apart); 24 + i: it is negative (its magnitude is put, and -v for the values)
    uint32_t odd;
    int pad[3];
};
enum Bar {                                         // barriers, by index
    kKFull = 0,
    kKEmpty = kKFull + kKStages,
    kVFull = kKEmpty + kKStages,
    kVEmpty = kVFull + kVStages,
    kHFull = kVEmpty + kVStages,
    kHEmpty = kHFull + kHStages,
    kMFull = kHEmpty + kHStages,
    kSFull = kMFull + kMeta,
    kPFull = kSFull + 2,
    kOFull = kPFull + 2,
    kOEmpty = kOFull + 2,
    kQFull = kOEmpty + 2,
    kPiece = kQFull + 2,
    kPieceFree = kPiece + kPieces,
    kDrain = kPieceFree + kPieces,
    kBars = kDrain + 1
};

// One piece: 256 rows of a request and a run of its tiles.
struct Piece {
    long long at;               // its first place on the line
    int plane, b, rt;           // rank * Hk + head; request; row tile
    int tile0, tiles;           // first tile of this piece (in tiles of the context), how many (may be none)
    int units;                  // places on the line: tiles, and the row tile's kOver if they are this piece's
    int begin, all;             // first tile of the whole row tile, and its count
    int len, count, first;      // context, new tokens, row of the first new token
};

struct Work {
    const uint32_t *upto;       // [B + 1] prefix sums of the requests' units, per plane
    const SfarAttnArgs &a;
    // tiles that some row of a row tile attends to (at least one: rows of nothing are written too)
    __device__ __forceinline__ void range(int len, int count, int rt, int &begin, int &all) const
    {
        const int i0 = rt * kRows / a.G, i1 = min(count - 1, (rt * kRows + kRows - 1) / a.G);
        const int pos0 = len - count + i0, pos1 = len - count + i1;
        begin = sfar_attn_from(a, pos0) / kTile;
        all = max(1, (max(0, pos1 + 1) + kTile - 1) / kTile - begin);
    }
    __device__ __forceinline__ int row_tiles(int count) const { return (int)(((long long)count * a.G + kRows - 1) / kRows); }
    // by a whole warp
    __device__ __forceinline__ Piece at(long long u, long long end) const
    {
        const int lane = threadIdx.x & 31;
        Piece p;
        p.at = u;
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
        uint32_t w = v - upto[lo];
        // the row tile that unit w lies in: 32 at a time
        const int n = row_tiles(p.count);
        for (int rt0 = 0;; rt0 += 32) {
            int begin = 0, all = 0;
            if (rt0 + lane < n)
                range(p.len, p.count, rt0 + lane, begin, all);
            uint32_t sum = rt0 + lane < n ? (uint32_t)all + kOver : 0u;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t o = __shfl_up_sync(SFAR_FULL, sum, d);
                if (lane >= d)
                    sum += o;
            }
            const unsigned past = __ballot_sync(SFAR_FULL, sum > w);
            if (past || rt0 + 32 >= n) {
                const int l = past ? __ffs(past) - 1 : 0;
                p.rt = rt0 + l;
                p.begin = __shfl_sync(SFAR_FULL, begin, l);
                p.all = __shfl_sync(SFAR_FULL, all, l);
                const int k = (int)(w - (__shfl_sync(SFAR_FULL, sum, l) - (uint32_t)(p.all + kOver)));
                p.tile0 = p.begin + k;
                p.units = (int)min((long long)(p.all + kOver - k), end - u);
                p.tiles = max(0, min(p.units, p.all - k));
                return p;
            }
            w -= __shfl_sync(SFAR_FULL, sum, 31);
        }
    }
    // the next piece with tiles from place u on, and u past it; false: none before `end`
    __device__ __forceinline__ bool take(long long &u, long long end, Piece &p) const
    {
        while (u < end) {
            p = at(u, end);
            u += p.units;
            if (p.tiles > 0)
                return true;
        }
        return false;
    }
};

// 0xff for each byte that is a NaN of e4m3
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }
// Sixteen e4m3 as binary16 to two 16-byte chunks of a swizzled row, whose places differ in bit 4.
__device__ __forceinline__ void widen(unsigned char *to, const uint4 &v)
{
    *reinterpret_cast<uint4 *>(to) = make_uint4(cvt_f16x2_e4m3(v.x), cvt_f16x2_e4m3(v.x >> 16), cvt_f16x2_e4m3(v.y), cvt_f16x2_e4m3(v.y >> 16));
    *reinterpret_cast<uint4 *>((uintptr_t)to ^ 16) =
        make_uint4(cvt_f16x2_e4m3(v.z), cvt_f16x2_e4m3(v.z >> 16), cvt_f16x2_e4m3(v.w), cvt_f16x2_e4m3(v.w >> 16));
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// the largest of 16 values, NaN left out unless all are
__device__ __forceinline__ float max16(const uint32_t *v)
{
    float m[5];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        m[i] = max3(__uint_as_float(v[3 * i]), __uint_as_float(v[3 * i + 1]), __uint_as_float(v[3 * i + 2]));
    return fmaxf(max3(m[0], m[1], m[2]), max3(m[3], m[4], __uint_as_float(v[15])));
}
// What takes a product with keys of scale ks to units of log2, without its sign.  Never 0, so that a masked product of -inf
// stays that; products are below 2^25, so 2^-60 stands for any smaller one.
__device__ __forceinline__ float score_scale(float f, float ks) { return fmaxf(f * fabsf(ks), 0x1p-60f); }
// The eight warps of a tile's softmax; the two warps that share 32 rows.
__device__ __forceinline__ void tile_sync(int x) { asm volatile("bar.sync %0, 256;" ::"r"(1 + x) : "memory"); }
__device__ __forceinline__ bool tile_any(int x, bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(1 + x), "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(3 + pair) : "memory"); }
__device__ __forceinline__ bool pair_any(int pair, bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(3 + pair), "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv_prompt(const __grid_constant__ SfarAttnArgs a)
{
    using L = Lay<D>;
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ __align__(8) unsigned long long bars[kBars];
    __shared__ __align__(16) Meta meta[kMeta];
    __shared__ uint32_t s_warp[kThreads / 32], s_tmem;
    __shared__ Piece s_piece[kPieces];             // what the copying warp has begun with; no tiles: the end
    __shared__ float s_row[3][2][2][128];          // [what][tile][half]: what the two threads of a row tell each other
    __shared__ int s_last[2], s_nan[4][2];         // by the piece, modulo 4: first and last context token whose value holds a NaN
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t mem = (tc::smem(dyn) + 1023u) & ~1023u;
    unsigned char *gen = dyn + (mem - tc::smem(dyn));
    uint32_t *upto = reinterpret_cast<uint32_t *>(gen + L::kBytes);
    const uint32_t b0 = tc::smem(bars);
    auto bar = [&](int i) { return b0 + 8u * (uint32_t)i; };

    if (warp == kCopyWarp && lane < 2 * a.R)
        tc::prefetch_map(lane & 1 ? &a.vmap[lane >> 1] : &a.kmap[lane >> 1]);
    if (tid < kBars) {
        const int i = tid;
        const bool widen = (i >= kVEmpty && i < kVEmpty + kVStages) || (i >= kHFull && i < kHFull + kHStages);
        const bool eight = (i >= kPFull && i < kPFull + 2) || (i >= kOEmpty && i < kPiece);
        tc::bar_init(bar(i), eight ? kSoft / 2 : widen ? kWiden : i >= kPieceFree && i < kDrain ? kSoft + kWiden + 1 : 1);
        tc::bar_fence_init();
        tc::fence_async();
    }
    if (tid < 4) {
        s_nan[tid][0] = INT_MAX;
        s_nan[tid][1] = -1;
    }
    if (tid == 0)
        upto[0] = 0;
    if (warp == kMmaWarp)
        tc::tmem_alloc<1>(tc::smem(&s_tmem), 512);
    pdl_wait();
    const unsigned long long limit = ld_relaxed_u64(&a.ctl->timeout_ns);

    // prefix sums of the requests' units
    const Work work{upto, a};
    uint32_t carry = 0;
    int row_tiles = 0;                             // of this warp's requests
    for (int r0 = 0; r0 < a.B; r0 += kThreads / 32) {
        // a warp per request
        const int b = r0 + warp;
        uint32_t v = 0;
        if (b < a.B) {
            int len, count, first;
            sfar_attn_request(a, b, len, count, first);
            const int n = work.row_tiles(count);
            row_tiles = min(row_tiles + n, 1 << 26);       // above any step's
            for (int rt = lane; rt < n; rt += 32) {
                int begin, all;
                work.range(len, count, rt, begin, all);
                v += (uint32_t)(all + kOver);
            }
            v = __reduce_add_sync(SFAR_FULL, v);
            if (blockIdx.x == 0 && lane == 0)
                sfar_attn_check(a, b, len, count, first);
        }
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
            upto[b + 1] = before;
        __syncthreads();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;

    // As in k_kv_attn.cu, short row tiles are left whole where there are few: those of more than 6 tiles are cut into
    // pieces of no less than 4 (one request of 38 tokens x 8 heads and 1233 cached ones 37 us whole, 25 in such pieces; one
    // of 268 cached 16 and 22).
    if (lane == 0)
        s_warp[warp] = (uint32_t)row_tiles;
    __syncthreads();
    long long whole = 0;
    for (int w = 0; w < kThreads / 32; ++w)
        whole += s_warp[w];
    const long long U = sfar_attn_many(a, whole) ? 0 : (long long)carry * a.R * a.Hk;
    const long long row_all = whole * a.R * a.Hk;
    const long long N = min(min((long long)gridDim.x, U), U > 2 * kOver * row_all ? max(row_all, U / 4) : row_all);
    const long long u0 = blockIdx.x < N ? sfar_div(blockIdx.x * U, N) : 0, u1 = blockIdx.x < N ? sfar_div((blockIdx.x + 1) * U, N) : 0;

    if (warp < kSoft) {
        // -------------------------------------------------------------- softmax
        bool dead = false;                         // a wait gave up: go on without waiting
        // two threads to a row of scores, and of the accumulator: the first half of the columns and the second
        const int x = warp >> 3, half = warp >> 2 & 1, pair = x * 4 + (warp & 3);
        const int lrow = (warp & 3) * 32 + lane, rho = x * 128 + lrow;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t tS = tmem + x * 256 + 64 * half + lanes, tO = tmem + x * 256 + 128 + D / 2 * half + lanes;
        auto told = [&](int what) -> float & { return s_row[what][x][half][lrow]; };
        auto other = [&](int what) { return s_row[what][x][half ^ 1][lrow]; };
        unsigned char *qs = gen + L::oQ + x * 2 * L::kQ;             // this tile's queries: as they are, then split
        tc::Ring<kMeta> ms;
        uint32_t sphase = 0, ophase = 0;
        int piece = 0;
        // a piece's query rows into shared memory, as they are: 256 (D = 128) or 128 bytes to a row
        auto fetch = [&](const Piece &p) {
            const int r = p.plane / a.Hk, hk = p.plane % a.Hk, rows = min(kRows, p.count * a.G - p.rt * kRows);
            // lane i < 16: where the warp's row i comes from
            const int mine = x * 128 + (warp & 7) * 16 + (lane & 15), n = p.rt * kRows + mine;
            const uint16_t *src = a.q[r];
            if (mine < rows)
                src += (long long)(p.first + n / a.G) * a.qts + (long long)(hk * a.G + n % a.G) * a.qhs;
            constexpr int kC = D / 8;
#pragma unroll 4
            for (int i = 0; i < 16 * kC; i += 32) {
                const int row = (i + lane) / kC, c = (i + lane) % kC;
                const uint16_t *from = reinterpret_cast<const uint16_t *>(__shfl_sync(SFAR_FULL, (unsigned long long)src, row));
                const int at = (warp & 7) * 16 + row;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem(qs) + at * 2 * D + ((c ^ (at & (kC - 1))) << 4)),
                             "l"(from + c * 8), "r"(x * 128 + at < rows ? 16u : 0u)
                             : "memory");
            }
        };
        // Its rows, split, K-major with the swizzle of their length: the leading 4 bits of every element and the other
        // 4.  Returns what takes a product of this thread's row to a score in units of log2.
        auto split = [&]() {
            constexpr int kC = D / 16;             // 16-byte chunks of this thread's half of a row
            uint4 v[kC];
            asm volatile("cp.async.wait_all;" ::: "memory");
            tile_sync(x);
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                v[c] = *reinterpret_cast<const uint4 *>(qs + lrow * 2 * D + (((half * kC + c) ^ (lrow & (2 * kC - 1))) << 4));
                m = sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(m, v[c].x), v[c].y), v[c].z), v[c].w);
            }
            m = sfar_max_half(m);
            told(0) = __uint_as_float(m);
            tile_sync(x);                          // every row has been read: the split ones go into its place
            m = max(m, __float_as_uint(other(0)));
            const bool special = m >= 0x7f80u;
            const int e = special ? 127 : max((int)(m >> 7) - 127, -112);
            const float up = sfar_exp2i(7 - e);
#pragma unroll
            for (int c = 0; c < kC; c += 2) {
                const uint32_t w[8] = {v[c].x, v[c].y, v[c].z, v[c].w, v[c + 1].x, v[c + 1].y, v[c + 1].z, v[c + 1].w};
                uint32_t ph[8], pl[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const float x0 = bf16_lo(w[y]) * up, x1 = bf16_hi(w[y]) * up;
                    const float h0 = __uint_as_float(__float_as_uint(x0) & 0xfff00000u), h1 = __uint_as_float(__float_as_uint(x1) & 0xfff00000u);
                    ph[y] = cvt_e4m3x2(h0, h1);
                    pl[y] = cvt_e4m3x2(x0 - h0, x1 - h1);
                }
                if (special) {                     // infinities would saturate: NaN
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        if ((w[y] & 0x7f80u) == 0x7f80u)
                            ph[y] |= 0x7fu;
                        if ((w[y] & 0x7f800000u) == 0x7f800000u)
                            ph[y] |= 0x7f00u;
                    }
                }
                const int at = (half * kC + c) / 2, chunk = D == 128 ? at ^ (lrow & 7) : at ^ ((lrow >> 1) & 3);
                unsigned char *dst = qs + lrow * D + chunk * 16;
                *reinterpret_cast<uint4 *>(dst) = make_uint4(ph[0] | ph[1] << 16, ph[2] | ph[3] << 16, ph[4] | ph[5] << 16, ph[6] | ph[7] << 16);
                *reinterpret_cast<uint4 *>(dst + L::kQ) = make_uint4(pl[0] | pl[1] << 16, pl[2] | pl[3] << 16, pl[4] | pl[5] << 16, pl[6] | pl[7] << 16);
            }
            tc::fence_async();
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(bar(kQFull + x));
            return a.scale * 1.4426950408889634f * sfar_exp2i(max(e - 7, -126));
        };
        // The next piece, by all warps of the tile alike (or by none: after a wait that gave up).  It is read where the
        // copying warp has put it, and given back when it has been written out.
        tc::Ring<kPieces> ps;
        auto take = [&](int &at) {
            dead = dead || !tc::bar_wait(bar(kPiece + ps.slot), ps.phase, limit);
            const bool none = tile_any(x, dead);
            at = (int)ps.slot;
            ps.next();
            return !none && s_piece[at].tiles > 0;
        };
        auto rows_of = [&](const Piece &p) { return min(kRows, p.count * a.G - p.rt * kRows) - x * 128; };   // of this tile
        int now_at, next_at;
        bool have = take(now_at);
        float f = 0.f;
        if (have && rows_of(s_piece[now_at]) > 0) {
            fetch(s_piece[now_at]);
            f = split();
        }
        while (have) {
            const Piece &p = s_piece[now_at];
            const bool mine = rows_of(p) > 0;      // the tile has rows
            const int n = p.rt * kRows + rho;      // row of the request
            const bool row = lrow < rows_of(p);
            const int tok = n / a.G;
            const int pos = p.len - p.count + tok;
            const int hi = row ? min(p.len, pos + 1) : INT_MAX, lo = row ? sfar_attn_from(a, pos) : 0;
            // tiles that every row of this warp sees whole
            const int all_from = __reduce_max_sync(SFAR_FULL, lo), all_to = min(p.len, __reduce_min_sync(SFAR_FULL, hi));
            // log2 reference of the row's weights; sum: of this half's weight / value scale
            float wtop = -INFINITY, sum = 0.f;
            float zt = -INFINITY, zs = 0.f;        // reference and sum of this half's tokens of value scale 0
            const int tiles = p.tiles, j00 = p.tile0 * kTile + 64 * half;
            for (int k = 0; mine && k < tiles; ++k) {
                const int j0 = j00 + k * kTile;
                dead = dead || !tc::bar_wait(bar(kMFull + ms.slot), ms.phase, limit);
                const Meta &m = meta[ms.slot];
                const float4 ks = *reinterpret_cast<const float4 *>(m.ks + 4 * half), lv = *reinterpret_cast<const float4 *>(m.lvs + 4 * half),
                             iv = *reinterpret_cast<const float4 *>(m.ivs + 4 * half);
                const float c[4] = {score_scale(f, ks.x), score_scale(f, ks.y), score_scale(f, ks.z), score_scale(f, ks.w)};
                const float lvs[4] = {lv.x, lv.y, lv.z, lv.w}, ivs[4] = {iv.x, iv.y, iv.z, iv.w};
                const uint32_t odd = m.odd;
                const uint32_t none = odd >> (4 * half) & 15u;
                const bool edge = j0 < all_from || j0 + 64 > all_to || none || (odd & 0xff0100u);
                dead = dead || !tc::bar_wait(bar(kSFull + x), sphase, limit);
                sphase ^= 1u;
                tc::fence_after();
                if (k == tiles - 1) {
                    // the last scores of the piece are complete: the next one's queries may come in
                    have = take(next_at);
                    if (have && rows_of(s_piece[next_at]) > 0)
                        fetch(s_piece[next_at]);
                }
                if (edge) {
                    // -inf where the row does not see the token (products, not scores, so that what is seen is rounded as in a
                    // tile without masks)
#pragma unroll 1
                    for (int i = 0; i < 64; i += 16) {
                        uint32_t v[16];
                        tc::ld16(v, tS + i);
                        tc::wait_ld(v);
                        const int from = none >> (i >> 4) & 1 ? 64 : lo - j0 - i, to = min(hi, p.len) - j0 - i;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            v[e] = e >= from && e < to ? v[e] : __float_as_uint(-INFINITY);
                        tc::st16(tS + i, v);
                    }
                    tc::wait_st();
                    if (odd & 0xff0100u) {
                        // rare, and in a loop of its own: the other sign where a key scale is negative, sums where a value scale is 0
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            const float scale = m.ks[4 * half + i];
                            const bool zero = odd >> (16 + 4 * half + i) & 1;
                            if (!zero && !(scale < 0.f))
                                continue;
                            uint32_t v[16];
                            tc::ld16(v, tS + 16 * i);
                            tc::wait_ld(v);
                            if (scale < 0.f) {
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    v[e] ^= v[e] == __float_as_uint(-INFINITY) ? 0u : 0x80000000u;
                                tc::st16(tS + 16 * i, v);
                            }
                            if (zero) {
                                const float by = score_scale(f, scale), next = fmaxf(zt, max16(v) * by), ref = next == -INFINITY ? 0.f : next;
                                zs *= zt == -INFINITY ? 1.f : ex2(zt - next);
                                zt = next;
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    zs += ex2(fmaf(__uint_as_float(v[e]), by, -ref));
                            }
                        }
                        tc::wait_st();
                    }
                }
                float now;
                {
                    uint32_t s[32];
                    tc::ld32(s, tS);
                    tc::wait_ld(s);
                    now = fmaxf(fmaf(max16(s), c[0], lvs[0]), fmaf(max16(s + 16), c[1], lvs[1]));
                    tc::ld32(s, tS + 32);
                    tc::wait_ld(s);
                    now = fmaxf(now, fmaxf(fmaf(max16(s), c[2], lvs[2]), fmaf(max16(s + 16), c[3], lvs[3])));
                }
                uint32_t s[2][16];                 // scores are read twice rather than held: registers that spill cost more
                tc::ld16(s[0], tS);
                if (pair_any(pair, now > wtop + (kAttnLift + kAttnDeep))) {
                    told(1) = now;
                    pair_sync(pair);
                    // a row's reference goes by its own scores alone
                    const float most = fmaxf(now, other(1)), next = most > wtop + (kAttnLift + kAttnDeep) ? most - kAttnDeep : wtop;
                    const float keep = wtop == -INFINITY ? 1.f : ex2(wtop - next);   // o is 0 then, or NaN
                    sum *= keep;
                    wtop = next;
                    if (k > 0) {
                        // the scores' barrier says that the products before are complete
#pragma unroll 1
                        for (int i = 0; i < D / 2; i += 16) {
                            uint32_t o[16];
                            tc::ld16(o, tO + i);
                            tc::wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                            tc::st16(tO + i, o);
                        }
                    }
                }
                const float ref = wtop == -INFINITY ? 0.f : wtop;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    tc::wait_ld(s[i & 1]);
                    if (i < 3)
                        tc::ld16(s[(i + 1) & 1], tS + 16 * (i + 1));
                    uint32_t w[8];
                    const float off = lvs[i] - ref;
                    float add0 = 0.f, add1 = 0.f;
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float a0 = ex2(fmaf(__uint_as_float(s[i & 1][e]), c[i], off)), a1 = ex2(fmaf(__uint_as_float(s[i & 1][e + 1]), c[i], off));
                        add0 += a0;
                        add1 += a1;
                        w[e / 2] = half2_of(a0, a1);
                    }
                    sum = fmaf(add0 + add1, ivs[i], sum);
                    tc::st8(tS + 8 * i, w);        // over scores that have been read
                }
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(bar(kPFull + x));
                ms.next();
            }
            if (!mine) {
                for (int k = 0; k < tiles; ++k)
                    ms.next();
                have = take(next_at);
                if (have && rows_of(s_piece[next_at]) > 0)
                    fetch(s_piece[next_at]);
            }
            // both sums at one reference
            float top = fmaxf(wtop + kSumUp, zt);
            sum = (wtop == -INFINITY ? sum : ex2(wtop + kSumUp - top) * sum) + (zt == -INFINITY ? zs : ex2(zt - top) * zs);
            // the next queries first, so that their first scores are formed while this piece is written out
            float fnext = 0.f;
            if (have && rows_of(s_piece[next_at]) > 0)
                fnext = split();
            // --------------------------------------------------------- epilogue
            if (mine) {
                pair_sync(pair);                   // the last move's exchange has been read
                told(1) = top;
                told(2) = sum;
                pair_sync(pair);
                const float at = fmaxf(top, other(1));
                sum = (top == -INFINITY ? sum : ex2(top - at) * sum) + (other(1) == -INFINITY ? other(2) : ex2(other(1) - at) * other(2));
                top = at;
                dead = dead || !tc::bar_wait(bar(kOFull + x), ophase, limit);
                ophase ^= 1u;
                tc::fence_after();
            }
            const bool part = p.tiles < p.all;
            const long long from = p.at - (p.tile0 - p.begin), to = from + p.all;
            const int c0 = part ? (int)sfar_div((from + 1) * N - 1, U) : 0, c1 = part ? (int)sfar_div(to * N - 1, U) : 0;
            // [element / 4][row] and the reference last, so that neighbouring rows are neighbours
            auto slot = [&](int cta) {
                return reinterpret_cast<float4 *>(a.part) + ((size_t)cta * 2 + (cta == c0)) * (kRows * (D / 4 + 1)) + rho;
            };
            float4 *dst = slot(blockIdx.x);
            const float inv = sum == 0.f ? 0.f : (wtop == -INFINITY ? 1.f : ex2(wtop - top)) / sum;       // 0: the row attends to nothing
            const int r = p.plane / a.Hk, hk = p.plane % a.Hk;
            uint16_t *out = a.out[r] + (long long)(p.first + tok) * a.ots + (long long)(hk * a.G + n - tok * a.G) * a.ohs;
            const int *nan = s_nan[piece++ & 3];
            const int d0 = half * (D / 2);
            if (mine) {
#pragma unroll 1
                for (int i = 0; i < D / 2; i += 16) {
                    uint32_t o[16];
                    tc::ld16(o, tO + i);
                    tc::wait_ld(o);
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] = __uint_as_float(o[e]);
                    if (nan[1] >= 0 && row && !dead) {
                        // values that were NaN and taken out: put back for the rows that see them
                        const int from_j = max(max(lo, nan[0]), p.tile0 * kTile), to_j = min(min(hi, nan[1] + 1), (p.tile0 + p.tiles) * kTile);
                        for (int j = from_j; j < to_j; ++j) {
                            const int page = a.table[(size_t)p.b * a.W + (j >> a.shift)];
                            if ((unsigned)page >= (unsigned)a.pages)
                                continue;
                            const uint8_t *vp = a.v[r] + (((long long)page * a.Hk + hk << a.shift) + (j & ((1 << a.shift) - 1))) * D + d0 + i;
                            for (int e = 0; e < 16; ++e)
                                if ((vp[e] & 0x7f) == 0x7f)
                                    for (int z = 0; z < 16; ++z)
                                        if (z == e)
                                            v[z] = NAN;
                        }
                    }
                    if (!row)
                        continue;
                    if (part) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            __stcg(dst + (d0 + i + e) / 4 * kRows, make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
                    } else {
                        uint32_t b[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            b[e] = tc::bf16x2(v[2 * e] * inv, v[2 * e + 1] * inv);
                        tc::st32(out + d0 + i, b);
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(bar(kOEmpty + x));
                if (part && row && half == 0)
                    __stcg(dst + D / 4 * kRows, make_float4(top, sum, wtop, 0.f));
            }
            if (mine && part) {
                // the last of the row tile's CTAs joins its parts; the two tiles of rows separately
                SfarJoin join(a, x, c0, c1, blockIdx.x);
                for (;;) {
                    tile_sync(x);
                    if ((tid & 255) == 0)
                        s_last[x] = join.last();
                    tile_sync(x);
                    if (!s_last[x])
                        break;
                    // sums first, then the accumulator, 16 columns at a time
                    SfarAttnState<4> st;
                    const int last = row ? join.hi : join.lo - 1;
#pragma unroll 4
                    for (int c = join.lo; c <= last; c += join.step) {
                        const float4 t = __ldcg(slot(c) + D / 4 * kRows);
                        SfarAttnState<4> next;
                        next.reference(st.top, st.wtop);
                        next.reference(t.x, t.z);
                        next.add(st.top, st.sum, st.wtop);
                        next.add(t.x, t.y, t.z);
                        st = next;
                    }
                    const float by = st.factor();
                    const int lo_part = join.lo, step = join.step;
                    const bool more = join.next(a, x);
                    dst = slot(lo_part);
#pragma unroll 1
                    for (int i = d0; row && i < d0 + D / 2; i += 16) {
                        float v[16] = {};
#pragma unroll 2
                        for (int c = lo_part; c <= last; c += step) {
                            const float4 *src = slot(c);
                            const float4 t = __ldcg(src + D / 4 * kRows);
                            float4 y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = __ldcg(src + (i / 4 + e) * kRows);
                            const float w = t.z == -INFINITY ? 1.f : ex2(t.z - st.wtop);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                v[4 * e] += w * y[e].x;
                                v[4 * e + 1] += w * y[e].y;
                                v[4 * e + 2] += w * y[e].z;
                                v[4 * e + 3] += w * y[e].w;
                            }
                        }
                        if (more) {
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                __stcg(dst + (i + e) / 4 * kRows, make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
                        } else {
                            uint32_t b[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                b[e] = tc::bf16x2(v[2 * e] * by, v[2 * e + 1] * by);
                            tc::st32(out + i, b);
                        }
                    }
                    if (!more)
                        break;
                    tile_sync(x);                  // both threads of a row have read the group's references
                    if (row && half == 0)
                        __stcg(dst + D / 4 * kRows, make_float4(st.top, st.sum, st.wtop, 0.f));
                }
            }
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(bar(kPieceFree + now_at));
            now_at = next_at;
            f = fnext;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (dead && lane == 0)
            sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
    } else {
        if (warp < kCopyWarp) {
            // --------------------------------------- values: e4m3 -> binary16
            tc::Ring<kVStages> vs;
            tc::Ring<kHStages> hs;
            tc::Ring<kMeta> ms;
            const int ct = tid - 32 * kSoft;
            // this thread's 16-byte chunk c of tokens ct / kC, + 32 kWiden / kC, ...: the swizzle's bits of a token repeat
            constexpr int kC = D / 16, kSteps = kTile * kC / (32 * kWiden), kFrom = 32 * kWiden * 16, kTo = 32 * kWiden / kC * 128;
            static_assert((32 * kWiden / kC) % 8 == 0 && kSteps % 4 == 0, "a step keeps the swizzle");
            // Eight neighbouring lanes take four chunks of two tokens: their stores meet in no bank (eight chunks of one
            // token, as they lie, would go to four pairs of equal banks).
            const int tok0 = D == 128 ? 2 * (ct >> 4) + (ct >> 2 & 1) : ct >> 2, c = D == 128 ? 4 * (ct >> 3 & 1) + (ct & 3) : ct & 3;
            const int from = tok0 * D + ((D == 128 ? c ^ (tok0 & 7) : c ^ ((tok0 >> 1) & 3)) << 4);
            // 64 elements (128 bytes) of a token to a row, swizzled; the second 64 in a block of their own
            const int to = (c >> 2) * (kTile * 128) + tok0 * 128 + (((2 * (c & 3)) ^ (tok0 & 7)) << 4);
            bool dead = false;
            uint32_t qphase = 0, ophase = 0;
            int before = 0, piece = 0;             // rows of the piece before
            tc::Ring<kPieces> ps;
            for (;; ps.next()) {
                dead = __any_sync(SFAR_FULL, dead || !tc::bar_wait(bar(kPiece + ps.slot), ps.phase, limit));
                if (dead)
                    break;
                const Piece p = s_piece[ps.slot];
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(bar(kPieceFree + ps.slot));
                if (p.tiles == 0)
                    break;
                // The first rows' queries are in place: they have read the marks of the piece before the last.  Those
                // are cleared for the piece after the next.
                dead = dead || !tc::bar_wait(bar(kQFull), qphase, limit);
                qphase ^= 1u;
                int *nan = s_nan[piece & 3];
                if (ct == 0) {
                    s_nan[(piece + 2) & 3][0] = INT_MAX;
                    s_nan[(piece + 2) & 3][1] = -1;
                }
                ++piece;
                // tiles that every row of the piece sees whole
                const int pos0 = p.len - p.count + p.rt * kRows / a.G;
                const int pos1 = p.len - p.count + min(p.count - 1, (p.rt * kRows + kRows - 1) / a.G);
                const int all_from = sfar_attn_from(a, pos1), all_to = min(p.len, pos0 + 1);
                for (int k = 0; k < p.tiles; ++k) {
                    const int j0 = (p.tile0 + k) * kTile;
                    dead = dead || !tc::bar_wait(bar(kMFull + ms.slot), ms.phase, limit);
                    const uint32_t odd = meta[ms.slot].odd & 0xff0000ffu;
                    dead = dead || !tc::bar_wait(bar(kVFull + vs.slot), vs.phase, limit) ||
                           !tc::bar_wait(bar(kHEmpty + hs.slot), hs.phase ^ 1u, limit);
                    const unsigned char *src = gen + L::oV + vs.slot * L::kK + from;
                    unsigned char *dst = gen + L::oH + hs.slot * L::kH + to;
                    if (j0 >= all_from && j0 + kTile <= all_to && !odd) {
#pragma unroll 1
                        for (int n = 0; n < kSteps; n += 4) {
                            uint4 v[4];
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                v[b] = *reinterpret_cast<const uint4 *>(src + (n + b) * kFrom);
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                widen(dst + (n + b) * kTo, v[b]);
                        }
                    } else {
                        // some row does not see some token: places that hold none are zeros, and a NaN, which
                        // would reach every row, is taken out here and put back at the end
#pragma unroll 1
                        for (int n = 0; n < kSteps; n += 2) {
                            uint4 v[2];
#pragma unroll
                            for (int b = 0; b < 2; ++b)
                                v[b] = *reinterpret_cast<const uint4 *>(src + (n + b) * kFrom);
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                const int tok = tok0 + (n + b) * (32 * kWiden / kC), g = tok >> 4;
                                const uint32_t keep = j0 + tok >= p.len || (odd >> g & 1) ? 0u : ~0u;
                                const uint32_t sign = odd >> (24 + g) & 1 ? 0x80808080u : 0u;
                                uint32_t *w = &v[b].x, any = 0;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t is = nan_bytes(w[e]) & keep;
                                    any |= is;
                                    w[e] = (w[e] ^ sign) & keep & ~is;
                                }
                                if (any) {
                                    atomicMin(&nan[0], j0 + tok);
                                    atomicMax(&nan[1], j0 + tok);
                                }
                                widen(dst + (n + b) * kTo, v[b]);
                            }
                        }
                    }
                    if (k == p.tiles - 1) {
                        // so have the second rows of the piece before, if it had any, at the latest now
                        if (before > 128) {
                            dead = dead || !tc::bar_wait(bar(kOEmpty + 1), ophase, limit);
                            ophase ^= 1u;
                        }
                        before = min(kRows, p.count * a.G - p.rt * kRows);
                    }
                    tc::fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        tc::bar_arrive(bar(kHFull + hs.slot));
                        tc::bar_arrive(bar(kVEmpty + vs.slot));
                    }
                    vs.next();
                    hs.next();
                    ms.next();
                }
            }
            sfar_attn_padding<D>(a, ct, 32 * kWiden);
        } else if (warp == kCopyWarp) {
            // ------------------------------------------------------------ copies
            tc::Ring<kKStages> kr;
            tc::Ring<kVStages> vr;
            tc::Ring<kMeta> ms;
            uint32_t issued = 0;
            bool dead = false;
            const uint64_t often = tc::evict_last();
            const int per = min(1 << a.shift, SFAR_ATTN_TILE), boxes = kTile / per;   // tokens of one copy
            Piece p;
            tc::Ring<kPieces> ps;
            for (long long u = u0; !dead; ps.next()) {
                const bool have = work.take(u, u1, p);
                if (!tc::bar_wait(bar(kPieceFree + ps.slot), ps.phase ^ 1u, limit)) {
                    dead = true;
                    break;
                }
                if (!have)
                    p.tiles = 0;
                if (lane == 0) {
                    s_piece[ps.slot] = p;
                    tc::bar_arrive(bar(kPiece + ps.slot));
                }
                if (!have)
                    break;
                const int r = p.plane / a.Hk, hk = p.plane % a.Hk;
                const int *row = a.table + (size_t)p.b * a.W;
                for (int k = 0; k < p.tiles; ++k) {
                    const int j = (p.tile0 + k) * kTile + lane * per;    // lane i: copy i of the tile
                    const bool live = lane < boxes && j < p.len;
                    const int page = live ? row[j >> a.shift] : 0;
                    const bool bad = live && (unsigned)page >= (unsigned)a.pages;
                    if (bad)
                        sfar_kv_fault(a.ctl, p.b, SFAR_KV_BAD_PAGE);
                    const bool go = live && !bad;
                    const int slab = page * a.Hk + hk, y = j & ((1 << a.shift) - 1);
                    float ks = 0.f, vs = 0.f;
                    if (go) {
                        ks = a.ks[r][slab];
                        vs = a.vs[r][slab];
                    }
                    const unsigned any = __ballot_sync(SFAR_FULL, go);
                    const uint32_t bytes = (uint32_t)__popc(any) * per * D;
                    if (!tc::bar_wait(bar(kKEmpty + kr.slot), kr.phase ^ 1u, limit)) {
                        dead = true;
                        break;
                    }
                    if (go)
                        tc::load_3d(mem + L::oK + kr.slot * L::kK + lane * per * D, &a.kmap[r], 0, y, slab, bar(kKFull + kr.slot), often);
                    __syncwarp();
                    const int of = lane * 16 / per;                      // the copy that 16 tokens lie in
                    const float k16 = __shfl_sync(SFAR_FULL, ks, of & 31), v16 = __shfl_sync(SFAR_FULL, vs, of & 31);
                    const bool sixteen = lane < kTile / 16, there = any >> (of & 31) & 1u;
                    const uint32_t none = __ballot_sync(SFAR_FULL, sixteen && !there), minus = __ballot_sync(SFAR_FULL, sixteen && v16 < 0.f);
                    const bool nil = fabsf(v16) <= kNoScale;
                    const uint32_t zero = __ballot_sync(SFAR_FULL, sixteen && there && nil);
                    const bool negative = __any_sync(SFAR_FULL, ks < 0.f);
                    Meta &m = meta[ms.slot];
                    if (sixteen) {
                        m.ks[lane] = k16;
                        m.lvs[lane] = nil ? -INFINITY : lg2(fabsf(v16));
                        m.ivs[lane] = nil ? 0.f : kSumDown * (1.f / fabsf(v16));
                    }
                    if (lane == 0)
                        m.odd = none | (negative ? 256u : 0u) | zero << 16 | minus << 24;
                    __syncwarp();
                    if (lane == 0) {
                        tc::bar_arrive(bar(kMFull + ms.slot));
                        tc::bar_expect(bar(kKFull + kr.slot), bytes);
                    }
                    ++issued;
                    if (!tc::bar_wait(bar(kVEmpty + vr.slot), vr.phase ^ 1u, limit)) {
                        dead = true;
                        break;
                    }
                    if (go)
                        tc::load_3d(mem + L::oV + vr.slot * L::kK + lane * per * D, &a.vmap[r], 0, y, slab, bar(kVFull + vr.slot), often);
                    __syncwarp();
                    if (lane == 0)
                        tc::bar_expect(bar(kVFull + vr.slot), bytes);
                    kr.next();
                    vr.next();
                    ms.next();
                }
            }
            if (dead && lane == 0) {
                sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
                // the copies in flight land before the shared memory is released
                for (uint32_t i = issued - min(issued, (uint32_t)kKStages); i < issued; ++i)
                    tc::bar_wait(bar(kKFull + i % kKStages), (i / kKStages) & 1u, limit);
                for (uint32_t i = issued - min(issued, (uint32_t)kVStages); i < issued; ++i)
                    tc::bar_wait(bar(kVFull + i % kVStages), (i / kVStages) & 1u, limit);
            }
        } else {
            // -------------------------------------------------------------- MMAs
            constexpr uint32_t idS = tc::idesc_e4m3(128, kTile);
            // binary16 weights in tensor memory times values with the head contiguous (N-major)
            constexpr uint32_t idO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
            tc::Ring<kKStages> kr;
            tc::Ring<kHStages> hr;
            bool dead = false;
            uint32_t qphase[2] = {0, 0}, pphase[2] = {0, 0}, ofree[2] = {1, 1};
            const uint64_t dv0 = tc::desc_n128(mem + L::oH, kTile * 128), dk0 = tc::desc_k<D>(mem + L::oK), dq0 = tc::desc_k<D>(mem + L::oQ);
            tc::Ring<kPieces> ps;
            for (;; ps.next()) {
                dead = __any_sync(SFAR_FULL, dead || !tc::bar_wait(bar(kPiece + ps.slot), ps.phase, limit));
                if (dead)
                    break;
                const Piece p = s_piece[ps.slot];
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(bar(kPieceFree + ps.slot));
                if (p.tiles == 0)
                    break;
                const int tiles = min(kRows, p.count * a.G - p.rt * kRows) > 128 ? 2 : 1;
                if (tc::elect_one()) {             // the same lane every time: the rings stay in its registers
                    // the products of one tile of rows: W V of the step before, S of this one
                    auto values = [&](int x, bool add) {
                        const uint64_t dv = dv0 + hr.slot * (L::kH >> 4);
#pragma unroll
                        for (int i = 0; i < kTile / 16; ++i)
                            tc::mma_f16_ts(tmem + x * 256 + 128, tmem + x * 256 + (i < 4 ? 8 * i : 32 + 8 * i), dv + 128 * i, idO, add || i > 0);
                    };
                    auto scores = [&](int x) {
                        const uint64_t dk = dk0 + kr.slot * (L::kK >> 4), dq = dq0 + x * (2 * L::kQ >> 4);
#pragma unroll
                        for (int i = 0; i < D / 32; ++i)
                            tc::mma_f8<1>(tmem + x * 256, dq + 2 * i, dk + 2 * i, idS, i > 0);
#pragma unroll
                        for (int i = 0; i < D / 32; ++i)
                            tc::mma_f8<1>(tmem + x * 256, dq + (L::kQ >> 4) + 2 * i, dk + 2 * i, idS, true);
                        tc::commit(bar(kSFull + x));
                    };
                    auto wait = [&](int which, uint32_t &phase) {
                        const bool in = tc::bar_wait(bar(which), phase, limit);
                        phase ^= 1u;
                        return in;
                    };
                    dead = !tc::bar_wait(bar(kKFull + kr.slot), kr.phase, limit);
                    for (int x = 0; x < tiles && !dead; ++x) {
                        dead = !wait(kQFull + x, qphase[x]);
                        tc::fence_after();
                        if (!dead)
                            scores(x);
                    }
                    if (!dead) {
                        tc::commit(bar(kKEmpty + kr.slot));
                        kr.next();
                    }
                    // The loop that the tensor core waits for: as few instructions between a tile's weights and its
                    // products as there can be.
                    for (int k = 1; k < p.tiles && !dead; ++k) {
                        dead = !tc::bar_wait(bar(kHFull + hr.slot), hr.phase, limit) || !tc::bar_wait(bar(kKFull + kr.slot), kr.phase, limit) ||
                               (k == 1 && !wait(kOEmpty, ofree[0])) || !wait(kPFull, pphase[0]);
                        if (dead)
                            break;
                        tc::fence_after();
                        values(0, k > 1);
                        scores(0);
                        if (tiles == 2) {
                            dead = (k == 1 && !wait(kOEmpty + 1, ofree[1])) || !wait(kPFull + 1, pphase[1]);
                            if (dead)
                                break;
                            tc::fence_after();
                            values(1, k > 1);
                            scores(1);
                        }
                        tc::commit(bar(kHEmpty + hr.slot));
                        tc::commit(bar(kKEmpty + kr.slot));
                        hr.next();
                        kr.next();
                    }
                    dead = dead || !tc::bar_wait(bar(kHFull + hr.slot), hr.phase, limit);
                    for (int x = 0; x < tiles && !dead; ++x) {
                        dead = (p.tiles == 1 && !wait(kOEmpty + x, ofree[x])) || !wait(kPFull + x, pphase[x]);
                        if (dead)
                            break;
                        tc::fence_after();
                        values(x, p.tiles > 1);
                        tc::commit(bar(kOFull + x));
                    }
                    if (!dead) {
                        tc::commit(bar(kHEmpty + hr.slot));
                        hr.next();
                    }
                }
                dead = __any_sync(SFAR_FULL, dead);
            }
            if (tc::elect_one()) {
                if (dead)
                    sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
                // every MMA and every arrival it causes is done before the CTA leaves
                tc::commit(bar(kDrain));
                tc::bar_wait(bar(kDrain), 0, limit);
            }
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp)
        tc::tmem_free<1>(tmem, 512);
}

const void *sfar_kernel_kv_prompt(int head_dim, int *threads, int *smem)
{
    *threads = kThreads;
    *smem = (head_dim == 64 ? Lay<64>::kBytes : Lay<128>::kBytes) + 1024;
    return head_dim == 64 ? (const void *)k_kv_prompt<64> : (const void *)k_kv_prompt<128>;
}
