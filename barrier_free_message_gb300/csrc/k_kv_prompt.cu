// k_kv_prompt.cu -- attention of the step's tokens over the paged 8-bit cache
// (include/sfar_kv.h), for many query rows per request: chunks of prompts.
//
// The same rows, softmax and references as k_kv_attn.cu, on the tensor cores:
// per 128 rows and 128 cached tokens S = Q K^T and O += W V, both accumulated
// in tensor memory.  Compute-bound: 4 D flops per visible (row, token).
//
// Operands.  Keys are used as they lie in the cache, e4m3; the query row,
// scaled by a power of two to a largest magnitude in [128, 256), is split into
// two e4m3 numbers: the nearest, and what is left.  bf16's 8 significant bits
// are 4 + 4, so the split is exact down to 2^-9 of the row's largest element
// and off by at most 2^-18 of it below; two e4m3 products cost what one
// binary16 product would, and the keys need no conversion.  Values are widened
// to binary16 (exact) by a warpgroup of its own, once for the 256 rows that
// share them; the weights are rounded to binary16 and are the operand in
// tensor memory, in the place of the scores they come from.
//
// A CTA takes 256 rows as two tiles of 128, each with a softmax warpgroup (a
// thread per row: no shuffles).  The tensor core alternates: while it runs
// O_B += W_B V and S_B = Q_B K' of one tile, the other's softmax works.  Warp
// 12 copies tiles (TMA), one thread of warp 13 issues the MMAs.  The
// accumulator is rescaled, in tensor memory, only when a reference moves.
//
// Work: as in k_kv_attn.cu the tiles of all (rank, key head, request, 256
// rows) form one line, cut into one equal piece per SM; row tiles cut apart
// are joined by the last of their CTAs, in order.
#include "sfar_e4m3.cuh"
#include "sfar_attn.cuh"
#include "sfar_tc.cuh"

namespace {

constexpr int kTile = 128;                         // cached tokens per step
constexpr int kRows = SFAR_PROMPT_ROWS;            // query rows per CTA: two tiles of 128
constexpr int kThreads = 512;
constexpr int kKStages = 3, kVStages = 2, kHStages = 2, kMeta = 4;

template <int D> struct Lay {
    static constexpr int kK = kTile * D, kH = kTile * D * 2, kQ = 128 * D;
    static constexpr int oK = 0, oV = oK + kKStages * kK, oH = oV + kVStages * kK, oQ = oH + kHStages * kH;
    static constexpr int kBytes = oQ + 4 * kQ;     // queries: two tiles, nearest and rest
};
struct Meta {                                      // of a step
    float ks[kTile / 16], lvs[kTile / 16], sign[kTile / 16];   // each 16 tokens: key scale, log2 and sign of the value scale
    int bad;                                       // bit i: tokens 16 i .. are on no page of the pool
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
    kDrain = kQFull + 1,
    kBars = kDrain + 1
};

// One piece: 256 rows of a request and a run of its tiles.
struct Piece {
    int plane, b, rt;           // rank * Hk + head; request; row tile
    int tile0, tiles;           // first tile of this piece (in tiles of the context), how many
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
        begin = (a.window ? max(0, pos0 - a.window + 1) : 0) / kTile;
        all = max(1, (max(0, pos1 + 1) + kTile - 1) / kTile - begin);
    }
    __device__ __forceinline__ int row_tiles(int count) const { return (int)(((long long)count * a.G + kRows - 1) / kRows); }
    // by a whole warp
    __device__ __forceinline__ Piece at(long long u, long long end) const
    {
        const int lane = threadIdx.x & 31;
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
        uint32_t w = v - upto[lo];
        // the row tile that unit w lies in: 32 at a time
        const int n = row_tiles(p.count);
        for (int rt0 = 0;; rt0 += 32) {
            int begin = 0, all = 0;
            if (rt0 + lane < n)
                range(p.len, p.count, rt0 + lane, begin, all);
            uint32_t sum = (uint32_t)all;
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
                const int k = (int)(w - (__shfl_sync(SFAR_FULL, sum, l) - (uint32_t)p.all));
                p.tile0 = p.begin + k;
                p.tiles = (int)min((long long)(p.all - k), end - u);
                return p;
            }
            w -= __shfl_sync(SFAR_FULL, sum, 31);
        }
    }
};

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv_prompt(const __grid_constant__ SfarAttnArgs a)
{
    using L = Lay<D>;
    extern __shared__ __align__(1024) unsigned char dyn[];
    __shared__ __align__(8) unsigned long long bars[kBars];
    __shared__ Meta meta[kMeta];
    __shared__ uint32_t s_warp[kThreads / 32], s_tmem;
    __shared__ int s_last, s_nan[2];               // first and last context token of this piece whose value holds a NaN
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t mem = (tc::smem(dyn) + 1023u) & ~1023u;
    unsigned char *gen = dyn + (mem - tc::smem(dyn));
    uint32_t *upto = reinterpret_cast<uint32_t *>(gen + L::kBytes);
    const uint32_t b0 = tc::smem(bars);
    auto bar = [&](int i) { return b0 + 8u * (uint32_t)i; };

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            const bool four = (i >= kVEmpty && i < kVEmpty + kVStages) || (i >= kHFull && i < kHFull + kHStages) ||
                              (i >= kPFull && i < kPFull + 2) || (i >= kOEmpty && i < kOEmpty + 2);
            tc::bar_init(bar(i), i == kQFull ? 8 : four ? 4 : 1);
        }
        tc::bar_fence_init();
        tc::fence_async();
        upto[0] = 0;
        s_nan[0] = INT_MAX;
        s_nan[1] = -1;
    }
    if (warp == 13)
        tc::tmem_alloc<1>(tc::smem(&s_tmem), 512);
    pdl_wait();
    const unsigned long long limit = ld_relaxed_u64(&a.ctl->timeout_ns);

    // prefix sums of the requests' units
    const Work work{upto, a};
    uint32_t carry = 0;
    for (int r0 = 0; r0 < a.B; r0 += kThreads / 32) {
        // a warp per request
        const int b = r0 + warp;
        uint32_t v = 0;
        if (b < a.B) {
            int len, count, first;
            sfar_attn_request(a, b, len, count, first);
            const int n = work.row_tiles(count);
            for (int rt = lane; rt < n; rt += 32) {
                int begin, all;
                work.range(len, count, rt, begin, all);
                v += (uint32_t)all;
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
    sfar_attn_padding<D>(a);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;

    const long long U = (long long)carry * a.R * a.Hk;
    const long long N = min((long long)gridDim.x, U);
    const long long u0 = blockIdx.x < N ? blockIdx.x * U / N : 0, u1 = blockIdx.x < N ? (blockIdx.x + 1) * U / N : 0;
    bool dead = false;                             // a wait gave up

    if (warp < 8) {
        // -------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int x = warp >> 2;                   // which tile of rows
        const int rho = x * 128 + (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t tS = tmem + x * 256 + lanes, tO = tS + 128;
        tc::Ring<kMeta> ms;
        uint32_t sphase = 0, ophase = 0;
        for (long long u = u0; u < u1;) {
            const Piece p = work.at(u, u1);
            const int r = p.plane / a.Hk, hk = p.plane % a.Hk;
            const int rows = min(kRows, p.count * a.G - p.rt * kRows);
            const bool mine = rows > x * 128;      // the tile has rows
            const int n = p.rt * kRows + rho;      // row of the request
            const bool row = rho < rows;
            float f = 0.f;
            if (mine) {
                // this thread's query row, split, K-major with the swizzle of its row length
                const uint16_t *src = a.q[r] + (long long)(p.first + (row ? n / a.G : 0)) * a.qts + (long long)(hk * a.G + n % a.G) * a.qhs;
                uint32_t m = 0;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = row ? ld_nc_v4(src + c * 8) : make_uint4(0, 0, 0, 0);
                    m = sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(sfar_max_abs2(m, v.x), v.y), v.z), v.w);
                }
                m = sfar_max_half(m);
                const bool special = m >= 0x7f80u;
                const int e = special ? 127 : max((int)(m >> 7) - 127, -112);
                const float up = sfar_exp2i(7 - e);
                f = a.scale * 1.4426950408889634f * sfar_exp2i(max(e - 7, -126));
                const int lrow = rho & 127;
#pragma unroll 2
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 v = row ? ld_nc_v4(src + c * 16 + h * 8) : make_uint4(0, 0, 0, 0);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            uint32_t ph[2], pl[2];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float x0 = bf16_lo(w[i + y]) * up, x1 = bf16_hi(w[i + y]) * up;
                                ph[y] = cvt_e4m3x2(x0, x1);
                                const float2 b = e4m3x2_to_float2(ph[y]);
                                pl[y] = cvt_e4m3x2(x0 - b.x, x1 - b.y);
                                if (special) {     // infinities would saturate: NaN
                                    if ((w[i + y] & 0x7f80u) == 0x7f80u)
                                        ph[y] |= 0x7fu;
                                    if ((w[i + y] & 0x7f800000u) == 0x7f800000u)
                                        ph[y] |= 0x7f00u;
                                }
                            }
                            hi[2 * h + i / 2] = ph[0] | ph[1] << 16;
                            lo[2 * h + i / 2] = pl[0] | pl[1] << 16;
                        }
                    }
                    const int chunk = D == 128 ? c ^ (lrow & 7) : c ^ ((lrow >> 1) & 3);
                    unsigned char *dst = gen + L::oQ + x * 2 * L::kQ + lrow * D + chunk * 16;
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(dst + L::kQ) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                tc::fence_async();
            }
            __syncwarp();
            if (lane == 0)
                tc::bar_arrive(bar(kQFull));
            const int pos = p.len - p.count + n / a.G;
            const int hi = row ? min(p.len, pos + 1) : INT_MAX, lo = row && a.window ? max(0, pos - a.window + 1) : 0;
            // tiles that every row of this warp sees whole
            const int all_from = __reduce_max_sync(SFAR_FULL, lo), all_to = min(p.len, __reduce_min_sync(SFAR_FULL, hi));
            // log2 references: of the scores (sum), of the weights (o)
            float top = -INFINITY, wtop = -INFINITY, sum = 0.f;
            for (int k = 0; mine && k < p.tiles; ++k) {
                const int j0 = (p.tile0 + k) * kTile;
                dead = dead || !tc::bar_wait(bar(kMFull + ms.slot), ms.phase, limit);
                const Meta &m = meta[ms.slot];
                float c[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    c[i] = f * m.ks[i];
                dead = dead || !tc::bar_wait(bar(kSFull + x), sphase, limit);
                sphase ^= 1u;
                tc::fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tc::ld32(s[i], tS + 32 * i);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tc::wait_ld(s[i]);
                const bool edge = j0 < all_from || j0 + kTile > all_to || m.bad;
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 128; ++i) {
                        const int j = j0 + i;
                        const bool see = j >= lo && j < hi && j < p.len && !(m.bad >> (i >> 4) & 1);
                        s[i >> 5][i & 31] = __float_as_uint(see ? __uint_as_float(s[i >> 5][i & 31]) * c[i >> 4] : -INFINITY);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        c[i] = 1.f;
                }
                float now = -INFINITY, wnow = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float g = __uint_as_float(s[i >> 1][16 * (i & 1)]);
                    if (c[i] >= 0.f) {
#pragma unroll
                        for (int e = 1; e < 16; ++e)
                            g = fmaxf(g, __uint_as_float(s[i >> 1][16 * (i & 1) + e]));
                    } else {
#pragma unroll
                        for (int e = 1; e < 16; ++e)
                            g = fminf(g, __uint_as_float(s[i >> 1][16 * (i & 1) + e]));
                    }
                    g *= c[i];
                    now = fmaxf(now, g);
                    wnow = fmaxf(wnow, g + m.lvs[i]);
                }
                const bool move = now > top + kAttnLift || wnow > wtop + kAttnLift;
                if (__any_sync(SFAR_FULL, move)) {
                    const float next = fmaxf(top, now), wnext = fmaxf(wtop, wnow);
                    const float keep = wtop == -INFINITY ? 1.f : ex2(wtop - wnext);      // o is 0 then, or NaN
                    sum *= top == -INFINITY ? 1.f : ex2(top - next);
                    top = next;
                    wtop = wnext;
                    if (k > 0) {
                        // the scores' barrier says that the products before are complete
#pragma unroll 1
                        for (int i = 0; i < D; i += 16) {
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
                const float ref = top == -INFINITY ? 0.f : top;
                const uint64_t nref = tc::pack2(-ref, -ref);
                uint64_t add = 0ull;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[16];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int gi = 2 * i + h;
                        const float by = m.sign[gi] * (wtop == -INFINITY ? 0.f : ex2(ref + m.lvs[gi] - wtop));
                        const uint64_t c2 = tc::pack2(c[gi], c[gi]), by2 = tc::pack2(by, by);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 y = tc::unpack2(tc::fma2(tc::pack2u(s[i][16 * h + e], s[i][16 * h + e + 1]), c2, nref));
                            const uint64_t pp = tc::pack2(ex2(y.x), ex2(y.y));
                            add = tc::add2(add, pp);
                            const float2 z = tc::unpack2(tc::mul2(pp, by2));
                            w[8 * h + e / 2] = half2_of(z.x, z.y);
                        }
                    }
                    tc::st16(tS + 16 * i, w);
                }
                const float2 y = tc::unpack2(add);
                sum += y.x + y.y;
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(bar(kPFull + x));
                ms.next();
            }
            if (!mine)
                for (int k = 0; k < p.tiles; ++k)
                    ms.next();
            // --------------------------------------------------------- epilogue
            if (mine) {
                dead = dead || !tc::bar_wait(bar(kOFull + x), ophase, limit);
                ophase ^= 1u;
                tc::fence_after();
            }
            const bool part = p.tiles < p.all;
            const long long from = u - (p.tile0 - p.begin), to = from + p.all;
            const long long c0 = ((from + 1) * N - 1) / U, c1 = (to * N - 1) / U;
            // [element / 4][row] and the references last, so that neighbouring rows are neighbours
            auto slot = [&](long long cta, int which) {
                return reinterpret_cast<float4 *>(a.part) + ((size_t)cta * 2 + which) * (kRows * (D / 4 + 1));
            };
            float4 *dst = slot(blockIdx.x, p.tile0 == p.begin ? 1 : 0);
            SfarAttnState<4> mineS;
            mineS.reference(top, wtop);
            mineS.add(top, sum, wtop);
            const float inv = mineS.factor();
            uint16_t *out = a.out[r] + (long long)(p.first + n / a.G) * a.ots + (long long)(hk * a.G + n % a.G) * a.ohs;
            const bool poisoned = s_nan[1] >= 0;
            if (mine) {
#pragma unroll 1
                for (int i = 0; i < D; i += 16) {
                    uint32_t o[16];
                    tc::ld16(o, tO + i);
                    tc::wait_ld(o);
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] = __uint_as_float(o[e]);
                    if (poisoned && row && !dead) {
                        // values that were NaN and taken out: put back for the rows that see them
                        const int from_j = max(max(lo, s_nan[0]), p.tile0 * kTile), to_j = min(min(hi, s_nan[1] + 1), (p.tile0 + p.tiles) * kTile);
                        for (int j = from_j; j < to_j; ++j) {
                            const int page = a.table[(size_t)p.b * a.W + (j >> a.shift)];
                            if ((unsigned)page >= (unsigned)a.pages)
                                continue;
                            const uint8_t *vp = a.v[r] + (((long long)page * a.Hk + hk << a.shift) + (j & ((1 << a.shift) - 1))) * D + i;
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
                            __stcg(dst + (i + e) / 4 * kRows + rho, make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 8)
                            st_v4(out + i + e, make_uint4(tc::bf16x2(v[e] * inv, v[e + 1] * inv), tc::bf16x2(v[e + 2] * inv, v[e + 3] * inv),
                                                          tc::bf16x2(v[e + 4] * inv, v[e + 5] * inv), tc::bf16x2(v[e + 6] * inv, v[e + 7] * inv)));
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::bar_arrive(bar(kOEmpty + x));
                if (part && row)
                    __stcg(dst + D / 4 * kRows + rho, make_float4(top, sum, wtop, 0.f));
            }
            softmax_sync();                        // every row has been left in the workspace, every thread has read s_nan
            if (tid == 0) {
                s_nan[0] = INT_MAX;                // the next piece's values are converted after its queries are in place
                s_nan[1] = -1;
            }
            if (part) {
                __threadfence();
                softmax_sync();
                if (tid == 0) {
                    const int done = atomicAdd(a.arrived + c0, 1);
                    s_last = done == (int)(c1 - c0);
                    if (s_last)
                        a.arrived[c0] = 0;         // for the next call
                }
                softmax_sync();
                if (s_last && row) {
                    __threadfence();
                    SfarAttnState<4> st;
                    for (long long cta = c0; cta <= c1; ++cta) {
                        const float4 t = __ldcg(slot(cta, cta == c0) + D / 4 * kRows + rho);
                        st.reference(t.x, t.z);
                    }
                    for (long long cta = c0; cta <= c1; ++cta) {
                        const float4 t = __ldcg(slot(cta, cta == c0) + D / 4 * kRows + rho);
                        st.add(t.x, t.y, t.z);
                    }
                    const float by = st.factor();
#pragma unroll 1
                    for (int i = 0; i < D; i += 8) {
                        float v[8] = {};
                        for (long long cta = c0; cta <= c1; ++cta) {
                            const float4 *src = slot(cta, cta == c0) + rho;
                            const float4 t = __ldcg(src + D / 4 * kRows), y = __ldcg(src + i / 4 * kRows), z = __ldcg(src + (i / 4 + 1) * kRows);
                            const float w = t.z == -INFINITY ? 1.f : ex2(t.z - st.wtop);
                            v[0] += w * y.x;
                            v[1] += w * y.y;
                            v[2] += w * y.z;
                            v[3] += w * y.w;
                            v[4] += w * z.x;
                            v[5] += w * z.y;
                            v[6] += w * z.z;
                            v[7] += w * z.w;
                        }
                        st_v4(out + i, make_uint4(tc::bf16x2(v[0] * by, v[1] * by), tc::bf16x2(v[2] * by, v[3] * by),
                                                  tc::bf16x2(v[4] * by, v[5] * by), tc::bf16x2(v[6] * by, v[7] * by)));
                    }
                }
            }
            u += p.tiles;
        }
        if (dead && lane == 0)
            sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp < 12) {
            // --------------------------------------- values: e4m3 -> binary16
            tc::Ring<kVStages> vs;
            tc::Ring<kHStages> hs;
            tc::Ring<kMeta> ms;
            const int ct = tid - 256;
            uint32_t qphase = 0;
            for (long long u = u0; u < u1;) {
                const Piece p = work.at(u, u1);
                // the queries of a piece are in place once the piece before has been written out
                dead = dead || !tc::bar_wait(bar(kQFull), qphase, limit);
                qphase ^= 1u;
                for (int k = 0; k < p.tiles; ++k) {
                    const int j0 = (p.tile0 + k) * kTile;
                    dead = dead || !tc::bar_wait(bar(kMFull + ms.slot), ms.phase, limit);
                    const int bad = meta[ms.slot].bad;
                    dead = dead || !tc::bar_wait(bar(kVFull + vs.slot), vs.phase, limit) ||
                           !tc::bar_wait(bar(kHEmpty + hs.slot), hs.phase ^ 1u, limit);
                    const unsigned char *src = gen + L::oV + vs.slot * L::kK;
                    unsigned char *dst = gen + L::oH + hs.slot * L::kH;
                    constexpr int kC = D / 16;     // 16-byte chunks of a token
#pragma unroll 2
                    for (int i = ct; i < kTile * kC; i += 128) {
                        const int tok = i / kC, c = i % kC, j = j0 + tok;
                        const int from = D == 128 ? c ^ (tok & 7) : c ^ ((tok >> 1) & 3);
                        uint4 v = *reinterpret_cast<const uint4 *>(src + tok * D + from * 16);
                        if (j >= p.len || (bad >> (tok >> 4) & 1))
                            v = make_uint4(0, 0, 0, 0);
                        uint32_t *w = &v.x;
                        uint32_t is = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            is |= (w[e] & 0x7f7f7f7fu) + 0x01010101u;
                        if (is & 0x80808080u) {
                            // NaN reaches only the rows that see the token: taken out here, put back at the end
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] &= ~__vcmpeq4(w[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            atomicMin(&s_nan[0], j);
                            atomicMax(&s_nan[1], j);
                        }
                        uint32_t h[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            h[2 * e] = cvt_f16x2_e4m3(w[e]);
                            h[2 * e + 1] = cvt_f16x2_e4m3(w[e] >> 16);
                        }
                        // 64 elements (128 bytes) of a token to a row, swizzled; the second 64 in a block of their own
                        unsigned char *to = dst + (c >> 2) * (kTile * 128) + tok * 128;
                        const int at = 2 * (c & 3);
                        *reinterpret_cast<uint4 *>(to + ((at ^ (tok & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4 *>(to + (((at + 1) ^ (tok & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
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
                u += p.tiles;
            }
        } else if (warp == 12) {
            // ------------------------------------------------------------ copies
            tc::Ring<kKStages> kr;
            tc::Ring<kVStages> vr;
            tc::Ring<kMeta> ms;
            uint32_t issued = 0;
            const uint64_t often = tc::evict_last();
            const int per = min(1 << a.shift, SFAR_ATTN_TILE), boxes = kTile / per;   // tokens of one copy
            for (long long u = u0; u < u1 && !dead;) {
                const Piece p = work.at(u, u1);
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
                    const unsigned none = __ballot_sync(SFAR_FULL, lane < kTile / 16 && !(any >> (of & 31) & 1u));
                    Meta &m = meta[ms.slot];
                    if (lane < kTile / 16) {
                        m.ks[lane] = k16;
                        m.lvs[lane] = lg2(fabsf(v16));
                        m.sign[lane] = copysignf(1.f, v16);
                    }
                    if (lane == 0)
                        m.bad = (int)none;
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
                u += p.tiles;
            }
            if (dead && lane == 0) {
                sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
                // the copies in flight land before the shared memory is released
                for (uint32_t i = issued - min(issued, (uint32_t)kKStages); i < issued; ++i)
                    tc::bar_wait(bar(kKFull + i % kKStages), (i / kKStages) & 1u, limit);
                for (uint32_t i = issued - min(issued, (uint32_t)kVStages); i < issued; ++i)
                    tc::bar_wait(bar(kVFull + i % kVStages), (i / kVStages) & 1u, limit);
            }
        } else if (warp == 13) {
            // -------------------------------------------------------------- MMAs
            constexpr uint32_t idS = tc::idesc_e4m3(128, kTile);
            // binary16 weights in tensor memory times values with the head contiguous (N-major)
            constexpr uint32_t idO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
            tc::Ring<kKStages> kr;
            tc::Ring<kHStages> hr;
            uint32_t qphase = 0, pphase[2] = {0, 0}, ofree[2] = {1, 1};
            for (long long u = u0; u < u1 && !dead;) {
                const Piece p = work.at(u, u1);
                const int tiles = min(kRows, p.count * a.G - p.rt * kRows) > 128 ? 2 : 1;
                if (lane == 0) {
                    dead = !tc::bar_wait(bar(kQFull), qphase, limit);
                    tc::fence_after();
                    for (int k = 0; k <= p.tiles && !dead; ++k) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (x >= tiles || dead)
                                continue;
                            const uint32_t tS = tmem + x * 256, tO = tS + 128;
                            if (k > 0) {
                                if (x == 0)
                                    dead = !tc::bar_wait(bar(kHFull + hr.slot), hr.phase, limit);
                                if (k == 1) {
                                    dead = dead || !tc::bar_wait(bar(kOEmpty + x), ofree[x], limit);
                                    ofree[x] ^= 1u;
                                }
                                dead = dead || !tc::bar_wait(bar(kPFull + x), pphase[x], limit);
                                if (dead)
                                    continue;
                                pphase[x] ^= 1u;
                                tc::fence_after();
                                const uint64_t dv = tc::desc_n128(mem + L::oH + hr.slot * L::kH, kTile * 128);
#pragma unroll
                                for (int i = 0; i < kTile / 16; ++i)
                                    tc::mma_f16_ts(tO, tS + 8 * i, dv + 128 * i, idO, k > 1 || i > 0);
                                if (x == tiles - 1) {
                                    tc::commit(bar(kHEmpty + hr.slot));
                                    hr.next();
                                }
                                if (k == p.tiles)
                                    tc::commit(bar(kOFull + x));
                            }
                            if (k < p.tiles) {
                                if (x == 0) {
                                    dead = !tc::bar_wait(bar(kKFull + kr.slot), kr.phase, limit);
                                    if (dead)
                                        continue;
                                    tc::fence_after();
                                }
                                const uint64_t dk = tc::desc_k<D>(mem + L::oK + kr.slot * L::kK);
                                const uint64_t dq = tc::desc_k<D>(mem + L::oQ + x * 2 * L::kQ);
#pragma unroll
                                for (int i = 0; i < D / 32; ++i)
                                    tc::mma_f8<1>(tS, dq + 2 * i, dk + 2 * i, idS, i > 0);
#pragma unroll
                                for (int i = 0; i < D / 32; ++i)
                                    tc::mma_f8<1>(tS, dq + (L::kQ >> 4) + 2 * i, dk + 2 * i, idS, true);
                                tc::commit(bar(kSFull + x));
                                if (x == tiles - 1) {
                                    tc::commit(bar(kKEmpty + kr.slot));
                                    kr.next();
                                }
                            }
                        }
                    }
                    qphase ^= 1u;
                }
                dead = __any_sync(SFAR_FULL, dead);
                u += p.tiles;
            }
            if (lane == 0) {
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
    if (warp == 13)
        tc::tmem_free<1>(tmem, 512);
}

const void *sfar_kernel_kv_prompt(int head_dim, int *threads, int *smem)
{
    *threads = kThreads;
    *smem = (head_dim == 64 ? Lay<64>::kBytes : Lay<128>::kBytes) + 1024;
    return head_dim == 64 ? (const void *)k_kv_prompt<64> : (const void *)k_kv_prompt<128>;
}
