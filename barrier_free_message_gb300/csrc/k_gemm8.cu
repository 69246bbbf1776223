// k_gemm8.cu -- the e4m3 row-parallel projection of several tokens, with a
// scale for each block of 128 (include/sfar_fp8.h), on the tensor cores.
//
// The hardware sums the 128 exact products of a block (four MMAs of 32) into
// tensor memory; the epilogue warps read that partial sum back and fold it
// into binary32 registers, scaled, while the tensor core works on the next
// block into the other half of tensor memory: y += (sx * sw) * partial.
//
// Two forms, by which operand lies along the 128 lanes of tensor memory:
//
//  k_gemm8_few   lanes = outputs (rows of w8), columns = up to 128 tokens.
//                For few tokens: a tile of 128 outputs reads its weights once
//                from HBM at full MMA height however few tokens there are.
//  k_gemm8_many  lanes = tokens, columns = 256 outputs, on pairs of SMs
//                (cta_group::2: 256 tokens x 256 outputs a pair, each SM
//                holding half of either operand).  For many tokens: the pair
//                halves the shared-memory fills of a tile, which is what
//                bounds single tiles of e4m3, and a lane's scale is one number.
//
// Both are persistent, one CTA per SM: a producer warp keeps a ring of
// stages (one block of both operands each, TMA with the 128-byte swizzle, the
// ends of rows and columns filled with zeros) ahead across tiles, one thread
// issues the MMAs, and two tensor-memory accumulators alternate between it
// and the epilogue.
//
// Measured, 8 ranks, k = 3584, hidden 8192: 64 tokens (235 MB of weights) 43
// us, 5.8 TB/s or 0.85 of a copy's rate, bound by the weights' stream and the
// last, partly filled wave of tiles; 2048 tokens 392 us, 2455 TFLOP/s, 1.24 of
// a bf16 product's rate.  There the fold bounds it: 128 x 256 partial sums
// pass through the registers of an SM for every block (with the fold's
// arithmetic left out the same kernel takes 306 us).
#include "sfar_e4m3.cuh"
#include "sfar_kv_args.h"
#include "sfar_tc.cuh"

namespace {

// Waits until the last stages of the ring have been consumed: no MMA will
// arrive on an `empty` barrier after the CTA has left.
template <int N> __device__ __forceinline__ void drained(uint32_t empty, tc::Ring<N> st, unsigned long long limit)
{
    for (int s = 0; s < N; ++s) {
        if (!tc::bar_wait(empty + 8 * st.slot, st.phase ^ 1u, limit))
            return;
        st.next();
    }
}

// ------------------------------------------------------------------ few tokens
// Warps 0-3: epilogue; 4: TMA; 5: MMA; 6: scales.
template <int NT> struct Few {
    static constexpr int kThreads = 224;
    static constexpr int kA = 128 * 128, kB = NT * 128, kStage = kA + kB;
    static constexpr int kStages = (NT <= 16 ? 11 : NT <= 32 ? 10 : NT <= 64 ? 8 : 6);
    static constexpr int kScales = 4;                       // ring of scale rows
    static constexpr int kCols = 2 * NT < 32 ? 32 : 2 * NT; // tensor memory
    static constexpr int kSmem = kStages * kStage + kScales * NT * 4 + 1024;
};

}  // namespace

template <int NT>
__global__ void __launch_bounds__(Few<NT>::kThreads, 1) k_gemm8_few(const __grid_constant__ SfarGemm8Args a)
{
    using F = Few<NT>;
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) unsigned long long bars[2 * F::kStages + 4 + 2 * F::kScales + 1];
    __shared__ uint32_t s_tmem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = (tc::smem(dyn) + 1023u) & ~1023u;
    float *scl = reinterpret_cast<float *>(dyn + (ring - tc::smem(dyn)) + F::kStages * F::kStage);
    const uint32_t full = tc::smem(bars), empty = full + 8 * F::kStages, tfull = empty + 8 * F::kStages, tempty = tfull + 16,
                   sfull = tempty + 16, sempty = sfull + 8 * F::kScales, drain = sempty + 8 * F::kScales;
    if (warp == 4 && lane < 2 * a.R)
        tc::prefetch_map(lane & 1 ? &a.xmap[lane >> 1] : &a.wmap[lane >> 1]);
    if (threadIdx.x == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            tc::bar_init(full + 8 * s, 1);
            tc::bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::bar_init(tfull + 8 * s, 1);
            tc::bar_init(tempty + 8 * s, 4);
        }
        for (int s = 0; s < F::kScales; ++s) {
            tc::bar_init(sfull + 8 * s, 32);
            tc::bar_init(sempty + 8 * s, 4);
        }
        tc::bar_init(drain, 1);
        tc::bar_fence_init();
        tc::fence_async();
    }
    if (warp == 5)
        tc::tmem_alloc<1>(tc::smem(&s_tmem), F::kCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    const unsigned long long limit = ld_relaxed_u64(&a.ctl->timeout_ns);
    const int kb = a.kb;
    const long long tiles = (long long)a.R * a.tiles_n * a.tiles_m;
    bool gave_up = false;
    pdl_wait();

    if (warp == 4) {
        if (tc::elect_one()) {
            const uint64_t once = tc::evict_first(), often = tc::evict_last();
            tc::Ring<F::kStages> st;
            uint32_t issued = 0;
            for (long long t = blockIdx.x; t < tiles && !gave_up; t += gridDim.x) {
                const int m = (int)(t % a.tiles_m);
                const int n = (int)(t / a.tiles_m % a.tiles_n), r = (int)(t / a.tiles_m / a.tiles_n);
                for (int b = 0; b < kb; ++b) {
                    if (!tc::bar_wait(empty + 8 * st.slot, st.phase ^ 1u, limit)) {
                        gave_up = true;
                        break;
                    }
                    const uint32_t at = ring + st.slot * F::kStage, bar = full + 8 * st.slot;
                    tc::bar_expect(bar, F::kStage);
                    tc::load_2d(at, &a.wmap[r], b * 128, n * 128, bar, a.tiles_m > 1 ? often : once);
                    tc::load_2d(at + F::kA, &a.xmap[r], b * 128, m * NT, bar, often);
                    st.next();
                    ++issued;
                }
            }
            if (gave_up) {
                // the copies in flight land before the shared memory is released
                sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
                const uint32_t back = issued < (uint32_t)F::kStages ? issued : (uint32_t)F::kStages;
                for (uint32_t i = issued - back; i < issued; ++i)
                    tc::bar_wait(full + 8 * (i % F::kStages), (i / F::kStages) & 1u, limit);
            } else {
                drained<F::kStages>(empty, st, limit);
            }
        }
    } else if (warp == 5) {
        if (tc::elect_one()) {
            tc::Ring<F::kStages> st;
            tc::Ring<2> acc;
            for (long long t = blockIdx.x; t < tiles && !gave_up; t += gridDim.x)
                for (int b = 0; b < kb; ++b) {
                    if (!tc::bar_wait(tempty + 8 * acc.slot, acc.phase ^ 1u, limit) ||
                        !tc::bar_wait(full + 8 * st.slot, st.phase, limit)) {
                        gave_up = true;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t at = ring + st.slot * F::kStage;
                    const uint64_t da = tc::desc_k128(at), db = tc::desc_k128(at + F::kA);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_f8<1>(tmem + acc.slot * NT, da + 2 * k, db + 2 * k, tc::idesc_e4m3(128, NT), k > 0);
                    tc::commit(empty + 8 * st.slot);
                    tc::commit(tfull + 8 * acc.slot);
                    st.next();
                    acc.next();
                }
            if (gave_up) {
                sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
                tc::commit(drain);                      // the MMAs in flight end before their memory is released
                tc::bar_wait(drain, 0, limit);
            }
        }
    } else if (warp == 6) {
        // scales of a block's tokens times the weight block's: zeros past the last token
        tc::Ring<F::kScales> st;
        for (long long t = blockIdx.x; t < tiles && !gave_up; t += gridDim.x) {
            const long long m0 = t % a.tiles_m * NT;
            const int n = (int)(t / a.tiles_m % a.tiles_n), r = (int)(t / a.tiles_m / a.tiles_n);
            const float *sx = a.sx[r], *sw = a.sw[r] + (long long)n * kb;
            for (int b = 0; b < kb; ++b) {
                float v[(NT + 31) / 32];
                const float w = sw[b];
#pragma unroll
                for (int i = 0; i < (NT + 31) / 32; ++i) {
                    const long long m = m0 + i * 32 + lane;
                    v[i] = i * 32 + lane < NT && m < a.m ? sx[b * a.m + m] * w : 0.f;
                }
                if (!tc::bar_wait(sempty + 8 * st.slot, st.phase ^ 1u, limit)) {
                    gave_up = true;
                    break;
                }
#pragma unroll
                for (int i = 0; i < (NT + 31) / 32; ++i)
                    if (i * 32 + lane < NT)
                        scl[st.slot * NT + i * 32 + lane] = v[i];
                tc::bar_arrive(sfull + 8 * st.slot);
                st.next();
            }
        }
    } else {
        tc::Ring<2> acc;
        tc::Ring<F::kScales> st;
        const uint32_t mine = tmem + ((uint32_t)warp * 32u << 16);
        constexpr int kC = NT < 32 ? NT : 32;
        for (long long t = blockIdx.x; t < tiles && !gave_up; t += gridDim.x) {
            uint64_t y[NT / 2];
#pragma unroll
            for (int c = 0; c < NT / 2; ++c)
                y[c] = 0ull;
            for (int b = 0; b < kb; ++b) {
                if (!tc::bar_wait(sfull + 8 * st.slot, st.phase, limit) || !tc::bar_wait(tfull + 8 * acc.slot, acc.phase, limit)) {
                    gave_up = true;
                    break;
                }
                tc::fence_after();
                const float4 *s4 = reinterpret_cast<const float4 *>(scl + st.slot * NT);
#pragma unroll
                for (int c = 0; c < NT; c += kC) {
                    uint32_t p[kC];
                    if constexpr (kC == 32)
                        tc::ld32(p, mine + acc.slot * NT + c);
                    else
                        tc::ld16(p, mine + acc.slot * NT + c);
                    tc::wait_ld(p);
#pragma unroll
                    for (int e = 0; e < kC; e += 4) {
                        const float4 s = s4[(c + e) / 4];
                        y[(c + e) / 2] = tc::fma2(tc::pack2u(p[e], p[e + 1]), tc::pack2(s.x, s.y), y[(c + e) / 2]);
                        y[(c + e) / 2 + 1] = tc::fma2(tc::pack2u(p[e + 2], p[e + 3]), tc::pack2(s.z, s.w), y[(c + e) / 2 + 1]);
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) {
                    tc::bar_arrive(tempty + 8 * acc.slot);
                    tc::bar_arrive(sempty + 8 * st.slot);
                }
                acc.next();
                st.next();
            }
            if (gave_up)
                break;
            const long long m0 = t % a.tiles_m * NT;
            const int r = (int)(t / a.tiles_m / a.tiles_n);
            const long long n = t / a.tiles_m % a.tiles_n * 128 + warp * 32 + lane;
            if (n < a.n) {
                uint16_t *dst = a.y[r] + m0 * a.n + n;
                const int rows = (int)min((long long)NT, a.m - m0);
#pragma unroll
                for (int c = 0; c < NT; c += 2) {
                    const float2 v = tc::unpack2(y[c / 2]);
                    const uint32_t w = tc::bf16x2(v.x, v.y);
                    if (c < rows)
                        dst[(long long)c * a.n] = (uint16_t)w;
                    if (c + 1 < rows)
                        dst[(long long)(c + 1) * a.n] = (uint16_t)(w >> 16);
                }
            }
        }
        if (gave_up && threadIdx.x == 0)
            sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 5)
        tc::tmem_free<1>(tmem, F::kCols);
}

namespace {

// ----------------------------------------------------------------- many tokens
// Warps 0-7: epilogue (0-3 the first 128 outputs, 4-7 the second); 8: TMA; 9:
// MMA (of the pair's even CTA); 10 and 11: scales of either half.  A kernel of
// three warpgroups starts with 168 registers a thread; the epilogue's two take
// 192, the third keeps 120: the same 504 per lane of three, so no increase
// waits.
struct Many {
    static constexpr int kThreads = 384;
    static constexpr int kA = 128 * 128, kB = 128 * 128, kStage = kA + kB, kStages = 6;
    static constexpr int kAhead = 4, kScales = 2;           // blocks whose scales are handed over at once; ring of those
    static constexpr int kSmem = kStages * kStage + kScales * kAhead * 2 * 128 * 4 + 1024;
};

}  // namespace

__global__ void __launch_bounds__(Many::kThreads, 1) __cluster_dims__(2, 1, 1)
    k_gemm8_many(const __grid_constant__ SfarGemm8Args a)
{
    using F = Many;
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) unsigned long long bars[2 * F::kStages + 4 + 1 + 4 * F::kScales];
    __shared__ uint32_t s_tmem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const uint32_t ring = (tc::smem(dyn) + 1023u) & ~1023u;
    const uint32_t full = tc::smem(bars), empty = full + 8 * F::kStages, tfull = empty + 8 * F::kStages, tempty = tfull + 16, drain = tempty + 16,
                   sfull = drain + 8, sempty = sfull + 16 * F::kScales;
    float *scl = reinterpret_cast<float *>(dyn + (ring - tc::smem(dyn)) + F::kStages * F::kStage);
    if (warp == 8 && lane < 2 * a.R)
        tc::prefetch_map(lane & 1 ? &a.xmap[lane >> 1] : &a.wmap[lane >> 1]);
    if (threadIdx.x == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            tc::bar_init(full + 8 * s, 2);              // the two producers
            tc::bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::bar_init(tfull + 8 * s, 1);
            tc::bar_init(tempty + 8 * s, 2 * 8);        // the epilogue warps of both CTAs
        }
        for (int s = 0; s < 2 * F::kScales; ++s) {
            tc::bar_init(sfull + 8 * s, 1);
            tc::bar_init(sempty + 8 * s, 4);
        }
        tc::bar_init(drain, 1);
        tc::bar_fence_init();
        tc::fence_async();
    }
    if (warp == 9)
        tc::tmem_alloc<2>(tc::smem(&s_tmem), 512);
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    const unsigned long long limit = ld_relaxed_u64(&a.ctl->timeout_ns);
    const int kb = a.kb;
    const long long tiles = (long long)a.R * a.tiles_n * a.tiles_m;
    const long long first = blockIdx.x >> 1, step = gridDim.x >> 1;
    bool gave_up = false;
    pdl_wait();

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
        if (warp == 8 && tc::elect_one()) {
            const uint64_t often = tc::evict_last();
            const uint32_t lead_full = tc::map_rank(full, 0);
            tc::Ring<F::kStages> st;
            uint32_t issued = 0;
            for (long long t = first; t < tiles && !gave_up; t += step) {
                const int m = (int)(t % a.tiles_m);
                const int n = (int)(t / a.tiles_m % a.tiles_n), r = (int)(t / a.tiles_m / a.tiles_n);
                for (int b = 0; b < kb; ++b) {
                    if (!tc::bar_wait(empty + 8 * st.slot, st.phase ^ 1u, limit)) {
                        gave_up = true;
                        break;
                    }
                    const uint32_t at = ring + st.slot * F::kStage, bar = lead_full + 8 * st.slot;
                    // each CTA announces and copies its own half; the even CTA's barrier counts both
                    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar),
                                 "r"(F::kStage)
                                 : "memory");
                    tc::load_2d_pair(at, &a.xmap[r], b * 128, m * 256 + (int)rank * 128, bar, often);
                    tc::load_2d_pair(at + F::kA, &a.wmap[r], b * 128, n * 256 + (int)rank * 128, bar, often);
                    st.next();
                    ++issued;
                }
            }
            if (gave_up) {
                sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
                // the even CTA waits for the copies of both; the odd one then meets it at the cluster barrier
                const uint32_t back = issued < (uint32_t)F::kStages ? issued : (uint32_t)F::kStages;
                for (uint32_t i = issued - back; rank == 0 && i < issued; ++i)
                    tc::bar_wait(full + 8 * (i % F::kStages), (i / F::kStages) & 1u, limit);
            } else {
                drained<F::kStages>(empty, st, limit);
            }
        }
        if (warp == 9 && rank == 0 && tc::elect_one()) {
            tc::Ring<F::kStages> st;
            tc::Ring<2> acc;
            for (long long t = first; t < tiles && !gave_up; t += step)
                for (int b = 0; b < kb; ++b) {
                    if (!tc::bar_wait(tempty + 8 * acc.slot, acc.phase ^ 1u, limit) ||
                        !tc::bar_wait(full + 8 * st.slot, st.phase, limit)) {
                        gave_up = true;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t at = ring + st.slot * F::kStage;
                    const uint64_t da = tc::desc_k128(at), db = tc::desc_k128(at + F::kA);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_f8<2>(tmem + acc.slot * 256, da + 2 * k, db + 2 * k, tc::idesc_e4m3(256, 256), k > 0);
                    tc::commit_pair(empty + 8 * st.slot);
                    tc::commit_pair(tfull + 8 * acc.slot);
                    st.next();
                    acc.next();
                }
            if (gave_up) {
                sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
                tc::commit_pair(drain);
                tc::bar_wait(drain, 0, limit);
            }
        }
        if (warp >= 10) {
            // sx * sw of this half's block for the 128 tokens, several blocks' loads in flight
            const int half = warp - 10;
            tc::Ring<F::kScales> st;
            for (long long t = first; t < tiles && !gave_up; t += step) {
                const long long m0 = t % a.tiles_m * 256 + rank * 128 + lane;
                const int r = (int)(t / a.tiles_m / a.tiles_n);
                const long long nb = t / a.tiles_m % a.tiles_n * 2 + half;     // block of 128 outputs
                const float *sx = a.sx[r] + m0, *sw = a.sw[r] + (nb * 128 < a.n ? nb * kb : 0);
                for (int b0 = 0; b0 < kb && !gave_up; b0 += F::kAhead) {
                    float v[F::kAhead][4];
#pragma unroll
                    for (int u = 0; u < F::kAhead; ++u) {
                        const int b = min(b0 + u, kb - 1);
                        const float w = sw[b];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[u][i] = m0 + 32 * i < a.m ? sx[b * a.m + 32 * i] * w : 0.f;
                    }
                    if (!tc::bar_wait(sempty + 8 * (half * F::kScales + st.slot), st.phase ^ 1u, limit)) {
                        gave_up = true;
                        break;
                    }
#pragma unroll
                    for (int u = 0; u < F::kAhead; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            scl[((st.slot * F::kAhead + u) * 2 + half) * 128 + 32 * i + lane] = v[u][i];
                    __syncwarp();
                    if (lane == 0)
                        tc::bar_arrive(sfull + 8 * (half * F::kScales + st.slot));
                    st.next();
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        tc::Ring<2> acc;
        tc::Ring<F::kScales> st;
        const int half = warp >> 2, lrow = (warp & 3) * 32 + lane;
        const uint32_t mine = tmem + ((uint32_t)(warp & 3) * 32u << 16) + half * 128;
        const uint32_t lead_empty = tc::map_rank(tempty, 0);
        for (long long t = first; t < tiles && !gave_up; t += step) {
            const long long m = t % a.tiles_m * 256 + rank * 128 + lrow;
            const int r = (int)(t / a.tiles_m / a.tiles_n);
            const long long nb = t / a.tiles_m % a.tiles_n * 2 + half;     // block of 128 outputs
            const bool row = m < a.m, col = nb * 128 < a.n;
            float y[128];
#pragma unroll
            for (int c = 0; c < 128; ++c)
                y[c] = 0.f;
            for (int b = 0; b < kb; ++b) {
                const int u = b % F::kAhead;
                if ((u == 0 && !tc::bar_wait(sfull + 8 * (half * F::kScales + st.slot), st.phase, limit)) ||
                    !tc::bar_wait(tfull + 8 * acc.slot, acc.phase, limit)) {
                    gave_up = true;
                    break;
                }
                tc::fence_after();
                // 32 columns at a time: what a spilled register costs is more than what a second set in flight saves
                const uint32_t from = mine + acc.slot * 256;
                const float s = scl[((st.slot * F::kAhead + u) * 2 + half) * 128 + lrow];
                const bool spent = u == F::kAhead - 1 || b == kb - 1;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[32];
                    tc::ld32(p, from + 32 * c);
                    tc::wait_ld(p);
                    if (c == 3) {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            tc::bar_arrive_remote(lead_empty + 8 * acc.slot);
                            if (spent)
                                tc::bar_arrive(sempty + 8 * (half * F::kScales + st.slot));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        y[32 * c + e] = fmaf(__uint_as_float(p[e]), s, y[32 * c + e]);
                }
                acc.next();
                if (spent)
                    st.next();
            }
            if (gave_up)
                break;
            if (row && col) {
                uint16_t *dst = a.y[r] + m * a.n + nb * 128;
                const int cols = (int)min(128ll, a.n - nb * 128);
#pragma unroll
                for (int c = 0; c < 128; c += 16) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] = tc::bf16x2(y[c + 2 * e], y[c + 2 * e + 1]);
                    if (a.vec && c + 16 <= cols) {
                        tc::st32(dst + c, w);
                    } else if (a.vec && c < cols) {          // 8 outputs: their number is a multiple of 8
                        st_v4(dst + c, make_uint4(w[0], w[1], w[2], w[3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (c + e < cols)
                                dst[c + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                    }
                }
            }
        }
        if (gave_up && threadIdx.x == 0)
            sfar_record_fault(a.ctl, 0, blockIdx.x, -1, 0, SFAR_WAIT_COPY);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    // the partner may still read this CTA's shared memory or arrive on its barriers
    tc::cluster_sync();
    if (warp == 9)
        tc::tmem_free<2>(tmem, 512);
}

// tokens: columns of k_gemm8_few (16, 32, 64 or 128); 0: k_gemm8_many
const void *sfar_kernel_gemm8(int tokens, int *threads, int *smem)
{
#define SFAR_FEW(NT) (*threads = Few<NT>::kThreads, *smem = Few<NT>::kSmem, (const void *)k_gemm8_few<NT>)
    switch (tokens) {
    case 16: return SFAR_FEW(16);
    case 32: return SFAR_FEW(32);
    case 64: return SFAR_FEW(64);
    case 128: return SFAR_FEW(128);
    default: break;
    }
#undef SFAR_FEW
    *threads = Many::kThreads;
    *smem = Many::kSmem;
    return (const void *)k_gemm8_many;
}
