// k_latent_prompt.cu -- attention of prompts over expanded keys and values,
// the rotated part of the keys shared by the heads (include/sfar_latent.h).
//
// Per 128 new tokens of one head and 128 context tokens, on the tensor cores,
// both accumulated in tensor memory:
//   S = Q K^T + Qr Kr^T, O += P V.
// Compute-bound: 2 (2 D + rope) flops per visible pair; D = 128, rope = 64:
// 1280 clocks of products a tile, against 512 of exponentials.
//
// A CTA takes 256 rows as two tiles, so that while one tile's softmax works
// the tensor core has the other's products; keys and values are then read once
// for both.  Two threads own a row, half of its columns each: 16 softmax
// warps keep their scores in registers.  The two warps of 32 rows vote at every
// tile, by a barrier of their own and before any exponential, whether a
// reference moves (kAttnLift), tell each other maxima if one does and sums at
// the end (one thread to a row, 8 warps: 431 us where this took 362).  Weights
// go back to tensor memory as bf16, in the place of the scores; the accumulator
// is rescaled, there, only when a row's reference moves.
//
// Keys (three boxes of 64 elements x 128 tokens, 16 KB) and values (two) pass
// through one ring of 8 boxes in the order of their use; a box is given back
// by the last product that reads it.  Values that some rows of the piece do not
// see are looked at by two warps of their own, in the time of the softmax:
// infinities and NaN become zeros for the products, and the rows that do see
// them add them to their results.
//
// Work: row tiles are taken from a counter, one (rank, head) of a request after
// another, of its row tiles the one with the longest context first: they share
// keys and values in L2.  Fewer than CTAs are cut along the context and joined,
// in the parts' order.
// Warps 0-7, 8-15: the tiles' softmax; then copies and pieces, the MMAs, and two
// that look at values.
//
// Measured: 8 ranks, 12 heads, 3 prompts of 0.7 to 1 thousand tokens over
// contexts of 1.1 to 4.1 thousand, D = 128, rope = 64: 371 to 378 us, 1090 to
// 1110 TFLOP/s of visible pairs, 0.58 of the measured rate; tensor pipes active
// 52%.  With two tiles the last four warps' 64 registers do not hold all that
// they need: 216 bytes of stack a thread (232 with D = 64), none with one tile.
// What bounds it is a tile's chain, scores -> softmax -> product, of which
// two run beside one another (tensor memory holds no third), while shared
// memory gives a product of 128 x 128 its operands in just the 64 clocks that
// it takes.  Not L2: with half the bytes of keys and values it took 2% less.
// Slower: weights handed over in two halves, so that the second product starts
// earlier (378 us); loops of products not unrolled (513); copies announced to L2
// ahead (418).
#include "sfar_attn.cuh"
#include "sfar_latent_args.h"

namespace {

constexpr int kTile = 128, kGroup = SFAR_LATENT_GROUP, kBox = kTile * 128;     // bytes of 64 elements of 128 tokens
constexpr int kPieces = 4, kLeast = 4, kKept = 64;
constexpr int kRegsSoft = 104, kRegsRest = 64;     // with two tiles, 16 warps and 4: together the launch's 20 x 96

template <int D, int TILES> struct Lay {
    static constexpr int kV = D / 64, kK = kV + 1;                 // boxes of a step's values, keys
    static constexpr int kQ = TILES * kK * kBox;
    static constexpr int kSlots = TILES == 2 && D == 128 ? 8 : 10;
    static constexpr int kBytes = kQ + kSlots * kBox;
    static constexpr int kSoftWarps = 8 * TILES, kCopyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kThreads = 32 * (kSoftWarps + 4);
};

// 128 or 256 rows of one head of a request.
struct Piece {
    int r, h, b, rt;            // rank, head, request, row tile; b < 0: the end
    int len, count, first, kfirst;      // context, new tokens, rows of the first new and of the first context token
    int steps[2];               // of this piece, the tiles of the context that each tile of rows attends to
    int from;                   // the first tile of the piece
    int part, c0, c1;           // this part of the row tile, its first and its last
};

// The two warps that share 32 rows.
__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory"); }
__device__ __forceinline__ bool pair_any(int pair, bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(1 + pair), "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}
// All the softmax warps.
template <int TILES> __device__ __forceinline__ void all_sync() { asm volatile("bar.sync 9, %0;" ::"n"(256 * TILES) : "memory"); }
template <int TILES> __device__ __forceinline__ bool all_any(bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 9, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)v), "n"(256 * TILES)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ uint32_t times0(uint32_t w, uint32_t sum)
{
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(sum));
    return r;
}
__device__ __forceinline__ bool odd2(uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; }
// the same with zeros in place of infinities and NaN
__device__ __forceinline__ uint32_t finite2(uint32_t w)
{
    return w & ((w & 0x7f80u) == 0x7f80u ? 0xffff0000u : ~0u) & ((w & 0x7f800000u) == 0x7f800000u ? 0xffffu : ~0u);
}
// What a row's scores are multiplied by in its weights 2^(f s - ref), taken with one rounding, that of ref = f top: all of the
// row's have it in common, but beyond 2^32 it moves them out of binary32.  There f top is shrunk to 2^30, where it moves them by
// 2^64 and neighbouring numbers are 64 apart, so that the largest score has all the weight, as it has in full size.
__device__ __forceinline__ float row_factor(float top, float f) { return fabsf(top) * f > 0x1p30f ? 0x1p30f / fabsf(top) : f; }
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

struct Request {
    int len, count, first, kfirst;
};
// Request b's rows, none if its offsets are out of order or beyond the tensors.
__device__ __forceinline__ bool request(const SfarLatentPromptArgs &a, int b, Request &q)
{
    q.first = a.starts[b];
    q.kfirst = a.kstarts[b];
    const int e = a.starts[b + 1], ke = a.kstarts[b + 1];
    const bool ok = q.first >= 0 && e >= q.first && e <= a.T && q.kfirst >= 0 && ke >= q.kfirst && ke <= a.S;
    q.count = ok ? e - q.first : 0;
    q.len = ok ? ke - q.kfirst : 0;
    return ok;
}

// Every row of the piece sees the tokens before all_see; its first whole_steps steps have no others.
__device__ __forceinline__ int all_see(const Piece &p, int rows) { return min(p.len, p.len - p.count + p.rt * rows + 1); }
__device__ __forceinline__ int whole_steps(const Piece &p, int rows) { return max(0, max(0, all_see(p, rows)) / kTile - p.from); }

// the lowest n bits, n > 0
__device__ __forceinline__ uint32_t low_bits(int n) { return n < 32 ? (1u << n) - 1 : ~0u; }
// Infinities and NaN of values that the products had zeros for, into `dim` elements of a row's result, or of its part (`rows`
// floats from one to the next).  odd: a bit for each of the `tokens` that the row attends to of those from v on, set if it has
// such a value.
__device__ __noinline__ void add_odd(const uint32_t *odd, int tokens, const uint16_t *v, long long vts, int dim, uint16_t *out, float *part, int rows)
{
    for (int d = 0; d < dim; d += 8) {
        float sum[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum[e] = -0.f;                         // adds nothing, to -0 either
        bool open = true;                          // some element is not NaN yet
        for (int at = 0; open && at < tokens; at += 32)
            for (uint32_t m = odd[at >> 5] & low_bits(tokens - at); open && m; m &= m - 1) {
                const uint4 x = ld_nc_v4(v + (at + __ffs(m) - 1) * vts + d);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                open = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t one = e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16;
                    if ((one & 0x7f800000u) == 0x7f800000u)
                        sum[e] += __uint_as_float(one);
                    open = open || !isnan(sum[e]);
                }
            }
        if (part) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (sum[e] != 0.f)
                    __stcg(part + (d + e) * rows, __ldcg(part + (d + e) * rows) + sum[e]);
        } else {
            uint4 x = *reinterpret_cast<const uint4 *>(out + d);
            auto plus = [](uint32_t &w, float l, float h) { w = tc::bf16x2(__uint_as_float(w << 16) + l, __uint_as_float(w & 0xffff0000u) + h); };
            plus(x.x, sum[0], sum[1]);
            plus(x.y, sum[2], sum[3]);
            plus(x.z, sum[4], sum[5]);
            plus(x.w, sum[6], sum[7]);
            st_v4(out + d, x);
        }
    }
}

template <int D> __device__ __noinline__ void padding(const SfarLatentPromptArgs &a, int lane)
{
    if (a.starts[a.B] < a.T)
        sfar_attn_padding<D>(a, lane, 32);
}

// What a row's accumulator is multiplied by.  A sum is 0 if a row attends to nothing, then so is its result, or if all its
// scores are -inf: NaN.
__device__ __forceinline__ float factor(float sum, bool sees) { return sum == 0.f ? sees ? NAN : 0.f : 1.f / sum; }

// Joins `parts` parts, the first at p0, the others `step` floats on from it each: 8 elements of a row to a thread, rows next to
// one another as they lie in a part, kItems of them with kBatch parts each in flight (time passes by round trips).  Into the
// result, or into the first part; then a thread's first item's reference and sum are given back.  The first `blind` rows
// attend to nothing.
template <int D, int TILES, int kBatch, int kItems>
__device__ __forceinline__ float2 join_parts(float *p0, uint32_t step, int parts, int rows, int blind, uint16_t *out, long long ots)
{
    constexpr int kRows = 128 * TILES, kThreads = 256 * TILES;
    float2 kept = make_float2(-INFINITY, 0.f);
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < rows * (D / 8); i0 += kItems * kThreads) {
        uint32_t at[kItems], n[kItems];            // items past the last: the last again
        float top[kItems], total[kItems], o[kItems][8];
#pragma unroll
        for (int y = 0; y < kItems; ++y) {
            const int i = min(i0 + y * kThreads, rows * (D / 8) - 1);
            n[y] = (uint32_t)i % (uint32_t)rows;
            at[y] = 8u * (uint32_t)i - 7u * n[y];  // of the item's first element, 8 (i / rows), in a part
            top[y] = -INFINITY;
            total[y] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[y][e] = 0.f;
        }
#pragma unroll 1
        for (int c0 = 0; c0 < parts; c0 += kBatch) {
            float2 m[kItems][kBatch];
            float v[kItems][kBatch][8];
#pragma unroll
            for (int y = 0; y < kItems; ++y)
#pragma unroll
                for (int c = 0; c < kBatch; ++c) {
                    const uint32_t from = min(c0 + c, parts - 1) * step;           // parts past the last: the last again, not added
                    m[y][c] = __ldcg(reinterpret_cast<const float2 *>(p0 + (from + kRows * D + 2 * n[y])));
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[y][c][e] = __ldcg(p0 + (from + at[y] + e * rows));
                }
#pragma unroll
            for (int y = 0; y < kItems; ++y)
#pragma unroll
                for (int c = 0; c < kBatch; ++c)
                    if (c0 + c < parts) {
                        const float now = fmaxf(top[y], m[y][c].x);
                        const float keep = top[y] == now ? 1.f : ex2(top[y] - now), w = m[y][c].x == -INFINITY ? 0.f : ex2(m[y][c].x - now);
                        top[y] = now;
                        // a part that has seen nothing: its sum is 0, or NaN
                        total[y] = total[y] * keep + (m[y][c].x == -INFINITY ? m[y][c].y : w * m[y][c].y);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[y][e] = o[y][e] * keep + w * v[y][c][e];
                    }
        }
#pragma unroll
        for (int y = 0; y < kItems; ++y) {
            if (i0 + y * kThreads >= rows * (D / 8))
                break;
            if (out) {
                const float by = factor(total[y], (int)n[y] >= blind);
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = tc::bf16x2(o[y][2 * e] * by, o[y][2 * e + 1] * by);
                st_v4(out + n[y] * ots + (at[y] - n[y]) / (uint32_t)rows, make_uint4(w[0], w[1], w[2], w[3]));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    __stcg(p0 + (at[y] + e * rows), o[y][e]);
            }
        }
        if (i0 == (int)threadIdx.x)
            kept = make_float2(top[0], total[0]);
    }
    return kept;
}
// All softmax threads, after their parts: joins the row tile's parts if this CTA is the last of them.
template <int D, int TILES> __device__ __noinline__ void join(const SfarLatentPromptArgs &a, const Piece &p, int *s_last)
{
    constexpr int kRows = 128 * TILES, kPart = kRows * (D + 2);
    const int rows = min(kRows, p.count - p.rt * kRows);
    SfarJoin j(a, 0, p.c0, p.c1, p.part);
    for (;;) {
        all_sync<TILES>();
        if (threadIdx.x == 0)
            *s_last = j.last();
        all_sync<TILES>();
        if (!*s_last)
            return;
        const int parts = (j.hi - j.lo) / j.step + 1;
        const bool more = j.up != 0;
        float *const p0 = a.part + (size_t)j.lo * kPart;
        uint16_t *const out = more ? nullptr : a.out[p.r] + (long long)(p.first + p.rt * kRows) * a.ots + (long long)p.h * a.ohs;
        const uint32_t step = (uint32_t)(j.step * kPart);
        const int blind = p.count - p.len - p.rt * kRows;
        const float2 m = parts <= 2 ? join_parts<D, TILES, 2, 2>(p0, step, parts, rows, blind, out, a.ots)
                                    : join_parts<D, TILES, 4, 1>(p0, step, parts, rows, blind, out, a.ots);
        if (more) {
            all_sync<TILES>();                     // the first part's references have been read
            if ((int)threadIdx.x < rows)
                __stcg(reinterpret_cast<float2 *>(p0 + kRows * D) + threadIdx.x, m);
        }
        if (!j.next(a, 0))
            return;
    }
}

}  // namespace

template <int D, int TILES>
__global__ void __launch_bounds__(Lay<D, TILES>::kThreads, 1) k_latent_prompt(const __grid_constant__ SfarLatentPromptArgs a)
{
    using Y = Lay<D, TILES>;
    constexpr int kRows = 128 * TILES, kPart = kRows * (D + 2), kThreads = Y::kThreads, kSoftWarps = Y::kSoftWarps,
                  kCopyWarp = Y::kCopyWarp, kMmaWarp = Y::kMmaWarp;
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ __align__(8) unsigned long long bars[2 * Y::kSlots + 2 * kPieces + 13];
    __shared__ Piece s_piece[kPieces];
    __shared__ __align__(16) uint32_t s_odd[kPieces][Y::kV][(TILES + 1) * kTile / 32];     // tokens with values that are not finite, of each box
    __shared__ __align__(16) uint32_t upto[SFAR_KV_MAX_REQUESTS / kGroup + 4];
    Request *const kept = reinterpret_cast<Request *>(upto + 4);    // of up to kKept requests (two sums), read once
    __shared__ uint32_t s_warp[kThreads / 32], s_tmem;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t mem = (tc::smem(dyn) + 1023u) & ~1023u, ring = mem + Y::kQ;
    unsigned char *gen = dyn + (mem - tc::smem(dyn));
    const uint32_t full = tc::smem(bars), empty = full + 8 * Y::kSlots, pfull = empty + 8 * Y::kSlots, pempty = pfull + 8 * kPieces,
                   qfull = pempty + 8 * kPieces, qempty = qfull + 16, sbar = qempty + 16, wbar = sbar + 16, obar = wbar + 16, look = obar + 16,
                   clean = look + 8, drain = clean + 8;

    if (warp == kCopyWarp && lane < a.R) {
        tc::prefetch_map(&a.qmap[lane]);
        tc::prefetch_map(&a.kmap[lane]);
        tc::prefetch_map(&a.vmap[lane]);
        tc::prefetch_map(&a.krmap[lane]);
    }
    if (tid == 0) {
        for (uint32_t b = full; b <= drain; b += 8)
            tc::bar_init(b, b >= pempty && b < qfull ? kSoftWarps + 1 + Y::kV : b >= wbar && b < obar ? 8 : b == clean ? Y::kV : 1);
        tc::bar_fence_init();
        tc::fence_async();
        upto[0] = 0;
    }
    for (int i = tid; i < kPieces * Y::kV * (TILES + 1) * kTile / 32; i += kThreads)
        (&s_odd[0][0][0])[i] = 0;
    if (warp == kMmaWarp)
        tc::tmem_alloc<1>(tc::smem(&s_tmem), 256 * TILES);
    pdl_wait();
    const unsigned long long limit = ld_relaxed_u64(&a.ctl->timeout_ns);

    // prefix sums of the requests' row tiles, 32 requests to a warp
    uint32_t carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        uint32_t v = 0;
        if (b < a.B) {
            Request q;
            if (!request(a, b, q) && blockIdx.x == 0)
                sfar_kv_fault(a.ctl, b, SFAR_KV_BAD_TOKENS);
            if (a.B <= kKept)
                kept[b] = q;
            v = min((uint32_t)(q.count + kRows - 1) / kRows, 1u << 26);     // offsets in no order: 32 such sums fit 32 bits
        }
        v = __reduce_add_sync(SFAR_FULL, v);
        if (lane == 0)
            s_warp[warp] = v;
        __syncthreads();
        uint32_t before = carry;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            carry = min(carry + min(s_warp[w], 1u << 30), 1u << 30);
            if (w <= warp)
                before = carry;
        }
        if (lane == 0 && b < a.B)
            upto[b / kGroup + 1] = before;
        __syncthreads();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    const bool many = carry > (uint32_t)a.most;    // more than the step has: offsets in no order, nothing is computed
    if (many && blockIdx.x == 0 && tid == 0)
        sfar_kv_fault(a.ctl, a.B, SFAR_KV_BAD_TOKENS);
    // Fewer row tiles than CTAs are cut along the context, into at most two parts for each CTA and of no less than kLeast
    // tiles, twice that for more than 32 rows, whose parts are longer to write and read (one request, 4 heads, 1000 tokens: 31 us
    // so, 38 with kLeast; 4 new tokens after 16384 gain 3 us by it); the last of a row tile's parts to finish joins them, in
    // their order.
    const uint32_t whole = many ? 0 : carry * (uint32_t)(a.R * a.Hq);
    const uint32_t cuts = whole && whole < gridDim.x ? 2 * gridDim.x / whole : 1, items = whole * cuts;

    if (warp < kSoftWarps) {
        // -------------------------------------------------------------- softmax
        if constexpr (TILES == 2)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        bool dead = false;                         // a wait gave up: go on without waiting
        // two threads to a row of scores, and of the accumulator: the first half of the columns and the second
        const int x = warp >> 3, half = warp >> 2 & 1, pair = x * 4 + (warp & 3), lrow = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16, tS = tmem + x * 256 + 64 * half + lanes, tO = tmem + x * 256 + 128 + D / 2 * half + lanes;
        // What the two threads of a row tell each other, in a column of the scores that have been read (shared memory is full).
        auto swap = [&](float v) {
            tc::st1(tS + 63, __float_as_uint(v));
            tc::wait_st();
            tc::fence_before();
            pair_sync(pair);
            tc::fence_after();
            uint32_t r[1];
            tc::ld1(r, tS + 63 + (half ? -64 : 64));
            tc::wait_ld(r);
            return __uint_as_float(r[0]);
        };
        // never 0, so that a masked score of -inf stays that
        const float f = fmaxf(a.scale * 1.4426950408889634f, 1e-37f);
        tc::Ring<kPieces> ps;
        uint32_t sphase = 0, ophase = 0;
        for (;;) {
            dead = dead || !tc::bar_wait(pfull + 8 * ps.slot, ps.phase, limit);
            // Those that speak to one another leave together: two warps, or where row tiles are cut all of them (join()).
            dead = cuts > 1 ? all_any<TILES>(dead) : pair_any(pair, dead);
            if (dead)
                break;
            const Piece &p = s_piece[ps.slot];
            if (p.b < 0)
                break;
            const int i = p.rt * kRows + x * 128 + lrow, pos = p.len - p.count + i;
            const bool row = i < p.count;
            const int hi = (row ? pos + 1 : INT_MAX) - 64 * half;                   // of this thread's columns
            const int mine_to = p.len - p.count + p.rt * kRows + x * 128 + (warp & 3) * 32 + 1 - 64 * half;   // every row of this warp
            float ref = -INFINITY, sum = 0.f;      // of the row; of this half
            // Weights are 2^(by_score s - less).  A row that has seen nothing, or scores of -inf alone: any finite numbers, weights 0.
            float by_score = f, less = 0.f;
            const int steps = p.steps[x];
            for (int k = 0; k < steps; ++k) {
                const int j0 = (p.from + k) * kTile;
                dead = dead || !tc::bar_wait(sbar + 8 * x, sphase, limit);
                sphase ^= 1u;
                tc::fence_after();
                uint32_t s[2][32];
                tc::ld32(s[0], tS);
                tc::ld32(s[1], tS + 32);
                tc::wait_ld(s[0]);
                tc::wait_ld(s[1]);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (j0 + 32 * c + 32 > mine_to) {
                        const int n = hi - j0 - 32 * c;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (e >= n)
                                s[c][e] = 0xff800000u;
                    }
                float m[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    m[c] = max3(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]), __uint_as_float(s[c][2]));
#pragma unroll
                    for (int e = 3; e < 31; e += 2)
                        m[c] = max3(m[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                }
                float now = fmaxf(max3(m[0], m[1], __uint_as_float(s[0][31])), __uint_as_float(s[1][31]));
                if (pair_any(pair, now * f - ref > kAttnLift)) {
                    now = fmaxf(now, swap(now));
                    const float next = now * f - ref > kAttnLift ? now * f : ref;
                    const float keep = ref == -INFINITY ? 1.f : ex2(ref - next);           // all is 0 then, or NaN
                    if (next != ref) {
                        by_score = row_factor(now, f);
                        less = now * by_score + (next - next);                             // NaN for a score of +inf
                    }
                    ref = next;
                    sum *= keep;
                    if (k) {
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 16) {
                            uint32_t o[16];
                            tc::ld16(o, tO + c);
                            tc::wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                            tc::st16(tO + c, o);
                        }
                    }
                    tc::wait_st();
                    tc::fence_before();
                    pair_sync(pair);               // the other's has been read
                }
                const uint64_t f2 = tc::pack2(by_score, by_score), b2 = tc::pack2(-less, -less);
                uint64_t part = 0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 y = tc::unpack2(tc::fma2(tc::pack2u(s[c][e], s[c][e + 1]), f2, b2));
                        const float u = ex2(y.x), v = ex2(y.y);
                        part = tc::add2(part, tc::pack2(u, v));
                        w[e >> 1] = tc::bf16x2(u, v);
                    }
                    tc::st16(tS + 16 * c, w);
                }
                const float2 both = tc::unpack2(part);
                sum += both.x + both.y;
                if (k == steps - 1)
                    sum += swap(sum);              // of the row, from here on
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(wbar + 8 * x);
            }
            if (steps) {
                dead = dead || !tc::bar_wait(obar + 8 * x, ophase, limit);
                ophase ^= 1u;
                tc::fence_after();
            }
            const bool parts = p.c0 != p.c1;
            const float by = parts ? 1.f : factor(sum, pos >= 0);
            uint16_t *dst = a.out[p.r] + (long long)(p.first + min(i, p.count - 1)) * a.ots + (long long)p.h * a.ohs + D / 2 * half;
            const int rows = min(kRows, p.count - p.rt * kRows);       // of the row tile: a part's stride
            float *part = a.part + (size_t)p.part * kPart + D / 2 * half * rows + x * 128 + lrow;      // [element][row]
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
                uint32_t o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e] = 0;
                if (steps) {
                    tc::ld16(o, tO + c);
                    tc::wait_ld(o);
                }
                if (parts) {
                    if (row)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            __stcg(part + (c + e) * rows, __uint_as_float(o[e]));
                    continue;
                }
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = tc::bf16x2(__uint_as_float(o[2 * e]) * by, __uint_as_float(o[2 * e + 1]) * by);
                if (row)
                    tc::st32(dst + c, y);
            }
            if (row) {
                const int from = p.from + whole_steps(p, kRows);       // where the values have been looked at
                const int tokens = min(pos + 1, (p.from + steps) * kTile) - from * kTile;
                const uint32_t *odd = s_odd[ps.slot][D == 128 ? half : 0];
                uint32_t any = 0;                  // of steps that were not looked at, an earlier piece's
#pragma unroll
                for (int i = 0; i <= TILES; ++i) {
                    const uint4 w = reinterpret_cast<const uint4 *>(odd)[i];
                    any |= w.x | w.y | w.z | w.w;
                }
                if (any)
                    add_odd(odd, tokens, a.v[p.r] + (p.kfirst + (long long)from * kTile) * a.vts + (long long)p.h * a.vhs + D / 2 * half, a.vts,
                            D / 2, dst, parts ? part : nullptr, rows);
            }
            if (parts) {
                if (row && half == 0)
                    __stcg(reinterpret_cast<float2 *>(a.part + (size_t)p.part * kPart + kRows * D) + x * 128 + lrow, make_float2(ref, sum));
                join<D, TILES>(a, p, reinterpret_cast<int *>(s_warp));
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(pempty + 8 * ps.slot);
            ps.next();
        }
        if (dead && lane == 0)
            sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
    } else {
        if constexpr (TILES == 2)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == kCopyWarp) {
            // ------------------------------------------------------------ copies
            const uint64_t often = tc::evict_last(), once = tc::evict_first();
            auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(SFAR_FULL, tc::bar_wait(bar, parity, limit)); };
            tc::Ring<Y::kSlots> st;
            tc::Ring<kPieces> ps;
            bool dead = false;
            uint32_t boxes = 0, qphase[2] = {1, 1}, queries[2] = {0, 0};     // queries: asked for
            const int groups = (a.B + kGroup - 1) / kGroup;
            const uint32_t planes = (uint32_t)(a.R * a.Hq);
            // row tile number `taken`, by the whole warp
            auto piece = [&](uint32_t taken) {
                Piece p;
                p.b = -1;
                p.steps[0] = p.steps[1] = 0;
                if (taken >= items)
                    return p;
                const int part = (int)(taken % cuts);
                p.part = (int)taken;
                taken /= cuts;
                int lo = 0, hi = groups;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (upto[mid] * planes <= taken)
                        lo = mid;
                    else
                        hi = mid;
                }
                uint32_t v = taken - upto[lo] * planes;
                const int b = lo * kGroup + lane;
                Request q{0, 0, 0, 0};
                if (b < a.B) {
                    if (a.B <= kKept)
                        q = kept[b];
                    else
                        request(a, b, q);
                }
                const uint32_t n = (uint32_t)(q.count + kRows - 1) / kRows;
                uint32_t sum = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t o = __shfl_up_sync(SFAR_FULL, sum, d);
                    if (lane >= d)
                        sum += o;
                }
                const unsigned past = __ballot_sync(SFAR_FULL, sum * planes > v);
                const int l = past ? __ffs(past) - 1 : 0;
                p.b = lo * kGroup + l;
                p.len = __shfl_sync(SFAR_FULL, q.len, l);
                p.count = __shfl_sync(SFAR_FULL, q.count, l);
                p.first = __shfl_sync(SFAR_FULL, q.first, l);
                p.kfirst = __shfl_sync(SFAR_FULL, q.kfirst, l);
                const uint32_t tiles = max(1u, __shfl_sync(SFAR_FULL, n, l));
                v -= __shfl_sync(SFAR_FULL, sum - n, l) * planes;
                const uint32_t plane = v / tiles;
                p.rt = (int)(tiles - 1 - (v - plane * tiles));
                p.r = (int)(plane / (uint32_t)a.Hq);
                p.h = (int)(plane - (uint32_t)p.r * (uint32_t)a.Hq);
#pragma unroll
                for (int x = 0; x < TILES; ++x) {
                    const int from = p.rt * kRows + x * 128, last = min(p.count, from + 128) - 1;      // tile's last row
                    if (from < p.count)
                        p.steps[x] = (max(0, p.len - p.count + last + 1) + kTile - 1) / kTile;
                }
                // this part of the row tile's: p.c1 < p.c0 if it is none
                const int least = p.count - p.rt * kRows <= 32 ? kLeast : 2 * kLeast;
                const int all = max(p.steps[0], p.steps[1]), parts = min((int)cuts, max(1, (all + least - 1) / least));
                p.c0 = p.part - part;
                p.c1 = part < parts ? p.c0 + parts - 1 : -1;
                const int each = all / parts, rest = all - each * parts;            // the first `rest` have one more
                p.from = each * part + min(part, rest);
                const int to = p.from + each + (part < rest);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    p.steps[x] = max(0, min(p.steps[x], to) - p.from);
                return p;
            };
            uint32_t taken = blockIdx.x;
            Piece p = piece(taken), next;
#pragma unroll 1
            while (!dead) {
                const bool end = p.b < 0;
                // The next one is asked for early: one question for each row tile's part, so the counter is back at 0 when all
                // are taken.
                uint32_t after = 0;
                if (!end && lane == 0)
                    asm volatile("atom.relaxed.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(after) : "l"(a.next), "r"(items - 1) : "memory");
                if (!end && (p.c1 < 0 || max(p.steps[0], p.steps[1]) == 0))
                    next = piece(gridDim.x + __shfl_sync(SFAR_FULL, after, 0));
                if (end || p.c1 >= 0) {
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
                    const int steps = max(p.steps[0], p.steps[1]);
#pragma unroll 1
                    for (int k = 0; k < steps && !dead; ++k) {
#pragma unroll
                        for (int c = 0; c < Y::kK + Y::kV; ++c) {
                            if (!wait(empty + 8 * st.slot, st.phase ^ 1u)) {
                                dead = true;
                                break;
                            }
                            if (lane == 0) {
                                const uint32_t bar = full + 8 * st.slot, dst = ring + st.slot * kBox;
                                const int y = p.kfirst + (p.from + k) * kTile;
                                tc::bar_expect(bar, kBox);
                                if (c == Y::kV)
                                    tc::load_2d(dst, &a.krmap[p.r], 0, y, bar, often);
                                else
                                    tc::load_3d(dst, c < Y::kV ? &a.kmap[p.r] : &a.vmap[p.r], c < Y::kV ? 64 * c : 64 * (c - Y::kK), p.h, y, bar, often);
                            }
                            ++boxes;
                            st.next();
                            if (k == 0 && c == Y::kV) {
                                // the queries, once the last piece's scores are done with theirs
#pragma unroll 1
                                for (int x = 0; x < TILES; ++x)
                                    if (p.steps[x]) {
                                        if (!wait(qempty + 8 * x, x ? qphase[1] : qphase[0])) {
                                            dead = true;
                                            break;
                                        }
                                        (x ? qphase[1] : qphase[0]) ^= 1u;
                                        ++(x ? queries[1] : queries[0]);
                                        if (lane == 0)
                                            tc::bar_expect(qfull + 8 * x, Y::kK * kBox);
                                        __syncwarp();
                                        if (lane < Y::kK)
                                            tc::load_3d(mem + (x * Y::kK + lane) * kBox, &a.qmap[p.r], 64 * lane, p.h,
                                                        p.first + p.rt * kRows + x * 128, qfull + 8 * x, once);
                                    }
                                if (dead)
                                    break;
                            }
                        }
                        if (k == max(0, steps - 2)) {
                            next = piece(gridDim.x + __shfl_sync(SFAR_FULL, after, 0));
                            // its queries on their way to L2
                            if (lane < TILES * Y::kK && next.steps[lane / Y::kK])
                                tc::prefetch_3d(&a.qmap[next.r], 64 * (lane % Y::kK), next.h, next.first + next.rt * kRows + lane / Y::kK * 128);
                        }
                    }
                    if (dead)
                        break;
                }
                p = next;
            }
            if (dead && lane == 0) {
                sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
                // the copies in flight land before the shared memory is released
                for (uint32_t i = boxes - min(boxes, (uint32_t)Y::kSlots); i < boxes; ++i)
                    tc::bar_wait(full + 8 * (i % Y::kSlots), (i / Y::kSlots) & 1u, limit);
                for (int x = 0; x < TILES; ++x)
                    if (queries[x])
                        tc::bar_wait(qfull + 8 * x, (queries[x] - 1) & 1u, limit);
            }
        } else if (warp == kMmaWarp) {
            // -------------------------------------------------------------- MMAs
            constexpr uint32_t idS = tc::idesc_bf16(128, 128), idO = tc::idesc_bf16(128, D) | tc::kTransposeB;
            const uint64_t dq = tc::desc_k128(mem), dk = tc::desc_k128(ring);
            tc::Ring<kPieces> ps;
            uint32_t qphase[2] = {0, 0}, wphase[2] = {0, 0}, cphase = 0, slot = 0;     // slot: boxes before this step's keys, modulo 2 kSlots
            bool dead = false;
            for (;;) {
                dead = __any_sync(SFAR_FULL, dead || !tc::bar_wait(pfull + 8 * ps.slot, ps.phase, limit));
                if (dead)
                    break;
                const int n[2] = {s_piece[ps.slot].steps[0], s_piece[ps.slot].steps[1]}, b = s_piece[ps.slot].b, whole = whole_steps(s_piece[ps.slot], kRows);
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(pempty + 8 * ps.slot);
                ps.next();
                if (b < 0)
                    break;
                if (tc::elect_one()) {             // the same lane every time: the phases stay in its registers
                    const int most = max(n[0], n[1]), last = TILES == 2 && n[1] ? 1 : 0;       // last: the tile that a box is used by last
                    auto there = [&](uint32_t at) { return tc::bar_wait(full + 8 * (at % Y::kSlots), at / Y::kSlots & 1u, limit); };
                    auto wait = [&](uint32_t bar, uint32_t &phase) {
                        const bool in = tc::bar_wait(bar, phase, limit);
                        phase ^= 1u;
                        return in;
                    };
                    uint32_t keys = slot, values = 0;              // boxes before step k's keys, before the values of the one before
#pragma unroll 1
                    for (int k = 0; k <= most && !dead; ++k) {
#pragma unroll
                        for (int x = 0; x < TILES; ++x) {
                            const uint32_t tS = tmem + x * 256;
                            if (k && k <= n[x]) {
                                // O += P V of the step before
                                dead = dead || !wait(wbar + 8 * x, wphase[x]);
                                if (x == 0 || k > n[0]) {
#pragma unroll 1
                                    for (int c = 0; c < Y::kV; ++c)
                                        dead = dead || !there(values + c);
                                    if (k > whole)
                                        dead = dead || !wait(clean, cphase);
                                }
                                if (dead)
                                    break;
                                tc::fence_after();
                                const uint32_t v0 = values % Y::kSlots, v1 = (values + 1) % Y::kSlots;
                                if (D == 64 || v1 == v0 + 1) {
                                    // both boxes side by side: one product for all the head
                                    const uint64_t dv = tc::desc_n128(ring + v0 * kBox, kBox);
#pragma unroll
                                    for (int i = 0; i < kTile / 16; ++i)
                                        tc::mma_f16_ts(tS + 128, tS + (i < 4 ? 8 * i : 32 + 8 * i), dv + 128 * i, idO, k > 1 || i > 0);
                                } else {
                                    constexpr uint32_t idH = tc::idesc_bf16(128, 64) | tc::kTransposeB;
#pragma unroll
                                    for (int c = 0; c < 2; ++c) {
                                        const uint64_t dv = tc::desc_n128(ring + (c ? v1 : v0) * kBox, kBox);
#pragma unroll
                                        for (int i = 0; i < kTile / 16; ++i)
                                            tc::mma_f16_ts(tS + 128 + 64 * c, tS + (i < 4 ? 8 * i : 32 + 8 * i), dv + 128 * i, idH, k > 1 || i > 0);
                                    }
                                }
                                if (x == last)
#pragma unroll
                                    for (int c = 0; c < Y::kV; ++c)
                                        tc::commit(empty + 8 * ((values + c) % Y::kSlots));
                                if (k == n[x])
                                    tc::commit(obar + 8 * x);
                            }
                            if (k < n[x]) {
                                // S = Q K^T + Qr Kr^T
                                dead = dead || (k == 0 && !wait(qfull + 8 * x, qphase[x]));
#pragma unroll
                                for (int c = 0; c < Y::kK; ++c) {
                                    if (x == 0 || k >= n[0])
                                        dead = dead || !there(keys + c);
                                    if (dead)
                                        break;
                                    tc::fence_after();
                                    // these keys are here, so what the values' place held before them was: it may be looked at when they are
                                    if (c == Y::kV && k >= whole && (x == 0 || k >= n[0]))
                                        tc::bar_arrive(look);
                                    const uint64_t d = dk + (keys + c) % Y::kSlots * (kBox >> 4), q = dq + (x * Y::kK + c) * (kBox >> 4);
                                    const int parts = c < Y::kV ? 4 : a.rope / 16;
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        if (i < parts)
                                            tc::mma_f16_ss(tS, q + 2 * i, d + 2 * i, idS, c + i > 0);
                                    if (x == last)
                                        tc::commit(empty + 8 * ((keys + c) % Y::kSlots));
                                }
                                if (dead)
                                    break;
                                tc::commit(sbar + 8 * x);
                                if (k == n[x] - 1)
                                    tc::commit(qempty + 8 * x);
                            }
                        }
                        if (dead)
                            break;
                        values = keys + Y::kK;
                        keys += Y::kK + Y::kV;
                    }
                    slot = (slot + (uint32_t)most * (Y::kK + Y::kV)) % (2 * Y::kSlots);
                }
                dead = __any_sync(SFAR_FULL, dead);
            }
            if (tc::elect_one()) {
                if (dead)
                    sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
                // every MMA and every arrival it causes is done before the CTA leaves
                tc::commit(drain);
                tc::bar_wait(drain, 0, limit);
            }
        } else {
            // -------------------------------------------------------- values
            // Values of tokens that not every row of the piece sees: infinities and NaN become zeros (0 times them would reach
            // the rows that do not see them), and are added to the results of the rows that do see the token at the end.  A
            // warp to each box of a step; it has the time that the softmax takes.
            const int c = warp - kMmaWarp - 1;
            tc::Ring<kPieces> ps;
            uint32_t slot = 0, phase = 0;
            bool dead = false;
            while (c < Y::kV) {
                dead = !__all_sync(SFAR_FULL, tc::bar_wait(pfull + 8 * ps.slot, ps.phase, limit));
                if (dead || s_piece[ps.slot].b < 0)
                    break;
                const Piece &p = s_piece[ps.slot];
                const int most = max(p.steps[0], p.steps[1]), all_to = all_see(p, kRows), whole = whole_steps(p, kRows);
                for (int k = whole; k < most && !dead; ++k) {
                    const uint32_t at = slot + k * (Y::kK + Y::kV) + Y::kK + c;
                    dead = !__all_sync(SFAR_FULL, tc::bar_wait(look, phase, limit) && tc::bar_wait(full + 8 * (at % Y::kSlots), at / Y::kSlots & 1u, limit));
                    phase ^= 1u;
                    if (dead)
                        break;
                    unsigned char *v = gen + Y::kQ + at % Y::kSlots * kBox;
                    // times 0, whatever is not finite gives a NaN
#pragma unroll 2
                    for (int row = lane; row < kTile; row += 32) {
                        uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(v + row * 128 + ((e ^ (row & 7)) << 4));
                            sum[0] = times0(w.x, sum[0]);
                            sum[1] = times0(w.y, sum[1]);
                            sum[2] = times0(w.z, sum[2]);
                            sum[3] = times0(w.w, sum[3]);
                        }
                        const int j = (p.from + k) * kTile + row;
                        const bool found = j >= all_to && odd2(sum[0] | sum[1] | sum[2] | sum[3]);
                        if (found) {
#pragma unroll 1
                            for (int e = 0; e < 8; ++e) {
                                uint4 &w = *reinterpret_cast<uint4 *>(v + row * 128 + (e << 4));
                                w = make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
                            }
                        }
                        const uint32_t bits = __ballot_sync(SFAR_FULL, found);
                        if (lane == 0)
                            s_odd[ps.slot][c][((k - whole) * kTile + row) >> 5] = bits;
                    }
                    tc::fence_async();
                    __syncwarp();
                    if (lane == 0)
                        tc::bar_arrive(clean);
                }
                slot = (slot + (uint32_t)most * (Y::kK + Y::kV)) % (2 * Y::kSlots);        // its parity counts, too
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(pempty + 8 * ps.slot);
                ps.next();
            }
            if (dead && lane == 0)
                sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
            if (c == Y::kV - 1)
                padding<D>(a, lane);
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp)
        tc::tmem_free<1>(tmem, 256 * TILES);
}

const void *sfar_kernel_latent_prompt(int head_dim, int tiles, int *threads, int *smem)
{
#define SFAR_PROMPT(D, N) (*smem = Lay<D, N>::kBytes + 1024, (const void *)k_latent_prompt<D, N>)
    *threads = tiles == 1 ? Lay<64, 1>::kThreads : Lay<64, 2>::kThreads;
    if (tiles == 1)
        return head_dim == 64 ? SFAR_PROMPT(64, 1) : SFAR_PROMPT(128, 1);
    return head_dim == 64 ? SFAR_PROMPT(64, 2) : SFAR_PROMPT(128, 2);
#undef SFAR_PROMPT
}
