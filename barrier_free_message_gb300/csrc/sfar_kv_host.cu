// sfar_kv_host.cu -- the C ABI of the paged 8-bit cache (include/sfar_kv.h)
// and of the 8-bit projection (include/sfar_fp8.h): arguments, handle, launch.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <memory>
#include <new>

#include "sfar.h"
#include "sfar_fp8.h"
#include "sfar_kv.h"
#include "sfar_kv_args.h"
#include "sfar_test.h"

struct sfar_kv {
    int R = 0, Hq = 0, Hk = 0, D = 0, P = 0, shift = 0;
    size_t pages = 0;
    int dev = 0, sms = 0;
    void *cache[2][SFAR_MAX_R] = {};
    float *scale[2][SFAR_MAX_R] = {};
    uint8_t *ws = nullptr;
    SfarCtl *ctl = nullptr;             // at the start of ws
    float *part = nullptr;              // attention: partial results and their counters, in ws
    int *arrived = nullptr;
    SfarCtl *host_ctl = nullptr;
    cudaStream_t priv = nullptr;
    unsigned plan_ctas = SFAR_PLAN_CLUSTER;     // of a large plan's cluster
    CUtensorMap map[2][SFAR_MAX_R];     // the caches as the attention's copies see them
};

namespace {

size_t ceil_div(size_t x, size_t a) { return (x + a - 1) / a; }
bool aligned(const void *p, uintptr_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }

// Up to this many tokens the projection runs with outputs along the tensor
// core's lanes (weights read once, HBM-bound), beyond it with tokens there.
// R = 8, k = 3584, hidden 8192: 128 tokens 52 us that way and 64 the other, 256
// tokens (two tiles of tokens that way) 93 and 65.  More tokens run that way
// too if all tiles of 128 x 128 find an SM of their own, whose blocks of k then
// pass faster: 8 x 307 tokens, k = 2048, hidden 256: 10.1 us, 12.4 the other.
const size_t kFewTokens = 128;

// Up to this many query rows (new tokens x query heads per key head) of the
// longest request the attention runs 8 or 16 rows at a time (every 16 rows read
// the cache once), beyond it 256.  The host does not know the contexts' lengths,
// on which it depends between 17 and 48 rows which is faster.  us that way and
// the other, 8 ranks, one key head of 128 (64), requests of so many tokens each:
//   rows  requests x tokens:  4 x 1000     16 x 1000    64 x 1000    64 x 3000      64 x 10000
//   32, 8 query heads of 128  17.1, 21.6   29.5, 32.1   78.1, 84.8   166.5, 161.4   480, 434
//   48                        22.9, 22.1   39.2, 33.3  106.6, 85.7   239, 162       709, 436
//   24, 4 query heads of 64   10.9, 17.8   21.2, 25.7   60.3, 70.3   150, 143       467, 405
//   32                        13.5, 17.8   26.7, 25.9   76.9, 70.1   196, 143       622, 406
// so up to 32 rows the first is ahead for contexts of about 1000 tokens and less
// and behind for long ones.  16 rows read the cache once: 32 requests of 6003 to
// 10400 tokens 111 and 192.
const size_t kFewRows = 32;

// Counters of parts: six sets of one for each of the most CTAs of any of the kernels (3 per SM).
size_t arrived_bytes(int sms) { return 6 * 3 * (size_t)sms * sizeof(int); }

struct Span {
    uintptr_t lo, hi;
    Span(const void *p, size_t bytes) : lo((uintptr_t)p), hi((uintptr_t)p + bytes) {}
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

// Launches f as a programmatic dependent of the kernel before it on the
// stream (every kernel here begins with griddepcontrol.wait); plain: without.
sfar_status launch(int dev, const void *f, dim3 grid, unsigned threads, size_t smem, void *args, sfar_stream_t s, bool plain = false,
                   unsigned cluster = 1)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)s;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (!plain) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    void *params[] = {args};
    int cur = -1;
    cudaGetDevice(&cur);
    if (cur != dev)
        cudaSetDevice(dev);
    const cudaError_t err = cudaLaunchKernelExC(&cfg, f, params);
    if (cur != dev && cur >= 0)
        cudaSetDevice(cur);
    if (err != cudaSuccess) {
        cudaGetLastError();
        return SFAR_ERR_CUDA;
    }
    return SFAR_OK;
}

}  // namespace

extern "C" {

sfar_kv_t *sfar_kv_create(int R, int q_heads, int kv_heads, int head_dim, int page_tokens, size_t pages,
                          void *const k_cache[], void *const v_cache[], float *const k_scale[],
                          float *const v_scale[])
{
    auto fail = [](sfar_status st) {
        sfar_set_last_error(st);
        return (sfar_kv_t *)nullptr;
    };
    if (R < 1 || R > SFAR_MAX_R || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads || q_heads > 65535 ||
        (head_dim != 64 && head_dim != 128) ||
        (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && page_tokens != 128) || pages == 0 ||
        pages >= (1ull << 31) / (size_t)page_tokens || pages >= (1ull << 31) / (size_t)kv_heads || !k_cache || !v_cache ||
        !k_scale || !v_scale)
        return fail(SFAR_ERR_INVALID);
    const size_t cbytes = pages * (size_t)kv_heads * (size_t)page_tokens * (size_t)head_dim;
    const size_t sbytes = pages * (size_t)kv_heads * sizeof(float);
    for (int i = 0; i < 4 * R; ++i) {
        auto span = [&](int j) {
            const int r = j >> 2;
            return j & 2 ? Span(j & 1 ? v_scale[r] : k_scale[r], sbytes) : Span(j & 1 ? v_cache[r] : k_cache[r], cbytes);
        };
        if (!aligned((const void *)span(i).lo, i & 2 ? 4 : 16))
            return fail(SFAR_ERR_INVALID);
        for (int j = 0; j < i; ++j)
            if (span(i).meets(span(j)))
                return fail(SFAR_ERR_INVALID);
    }
    int dev = 0, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return fail(SFAR_ERR_CUDA);
    }
    if (major != 10 || minor != 3)
        return fail(SFAR_ERR_UNSUPPORTED);
    sfar_kv *h = new (std::nothrow) sfar_kv();
    if (!h)
        return fail(SFAR_ERR_OOM);
    h->R = R;
    h->Hq = q_heads;
    h->Hk = kv_heads;
    h->D = head_dim;
    h->P = page_tokens;
    h->shift = page_tokens == 16 ? 4 : page_tokens == 32 ? 5 : page_tokens == 64 ? 6 : 7;
    h->pages = pages;
    h->dev = dev;
    h->sms = sms;
    for (int r = 0; r < R; ++r) {
        h->cache[0][r] = k_cache[r];
        h->cache[1][r] = v_cache[r];
        h->scale[0][r] = k_scale[r];
        h->scale[1][r] = v_scale[r];
    }
    const PFN_cuTensorMapEncodeTiled_v12000 encode =
        reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(sfar_tensor_map_encoder());
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)page_tokens, (cuuint64_t)(pages * (size_t)kv_heads)};
    const cuuint64_t strides[2] = {(cuuint64_t)head_dim, (cuuint64_t)head_dim * (cuuint64_t)page_tokens};
    const cuuint32_t unit[3] = {1, 1, 1};
    const cuuint32_t box[3] = {(cuuint32_t)head_dim, (cuuint32_t)(page_tokens < SFAR_ATTN_TILE ? page_tokens : SFAR_ATTN_TILE), 1};
    for (int i = 0; i < 2 * R; ++i)
        if (!encode || encode(&h->map[i & 1][i >> 1], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, h->cache[i & 1][i >> 1], dims, strides, box, unit,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
            delete h;
            return fail(encode ? SFAR_ERR_INVALID : SFAR_ERR_UNSUPPORTED);
        }
    const size_t o_arrived = 256, o_part = (o_arrived + arrived_bytes(sms) + 255) / 256 * 256;
    const size_t few = (size_t)sms * 2 * 2 * 16, many = (size_t)sms * 2 * SFAR_PROMPT_ROWS;     // rows of partial results
    const size_t bytes = o_part + (few > many ? few : many) * ((size_t)head_dim + 4) * 4;
    if (cudaMalloc(&h->ws, bytes) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return fail(SFAR_ERR_OOM);
    }
    h->ctl = reinterpret_cast<SfarCtl *>(h->ws);
    h->arrived = reinterpret_cast<int *>(h->ws + o_arrived);
    h->part = reinterpret_cast<float *>(h->ws + o_part);
    SfarCtl init;
    memset(&init, 0, sizeof init);
    init.timeout_ns = 1000000000ull;
    init.strag_rank = init.drop_rank = -1;
    init.f_rank = init.f_cta = init.f_peer = -1;
    int threads = 0, smem = 0;
    int pthreads = 0, psmem = 0;
    const void *prompt = sfar_kernel_kv_prompt(head_dim, &pthreads, &psmem);
    if (cudaMemset(h->ws, 0, bytes) != cudaSuccess ||
        cudaFuncSetAttribute(prompt, cudaFuncAttributeMaxDynamicSharedMemorySize, psmem + (SFAR_PROMPT_REQUESTS + 1) * 4) != cudaSuccess ||
        cudaMemcpy(h->ctl, &init, sizeof init, cudaMemcpyHostToDevice) != cudaSuccess ||
        cudaFuncSetAttribute(sfar_kernel_kv_attn(head_dim, 8, &threads, &smem), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem + (SFAR_KV_MAX_REQUESTS + 1) * 4) != cudaSuccess ||
        cudaFuncSetAttribute(sfar_kernel_kv_attn(head_dim, 16, &threads, &smem), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem + (SFAR_KV_MAX_REQUESTS + 1) * 4) != cudaSuccess ||
        cudaStreamCreateWithFlags(&h->priv, cudaStreamNonBlocking) != cudaSuccess ||
        cudaMallocHost(&h->host_ctl, sizeof(SfarCtl)) != cudaSuccess ||
        cudaFuncSetAttribute(sfar_kernel_kv_plan(), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (4 * SFAR_KV_MAX_REQUESTS + 1) * 4) != cudaSuccess) {
        cudaGetLastError();
        sfar_kv_destroy(h);
        return fail(SFAR_ERR_CUDA);
    }
    // a large plan takes a cluster of 16 where the device can place one
    if (cudaFuncSetAttribute(sfar_kernel_kv_plan(), cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2 * SFAR_PLAN_CLUSTER;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2 * SFAR_PLAN_CLUSTER);
        cfg.blockDim = dim3(SFAR_PLAN_THREADS);
        cfg.dynamicSmemBytes = (4 * SFAR_KV_MAX_REQUESTS + 1) * 4;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, sfar_kernel_kv_plan(), &cfg) == cudaSuccess && clusters > 0)
            h->plan_ctas = 2 * SFAR_PLAN_CLUSTER;
    }
    cudaGetLastError();
    sfar_set_last_error(SFAR_OK);
    return h;
}

void sfar_kv_destroy(sfar_kv_t *h)
{
    if (!h)
        return;
    int cur = -1;
    cudaGetDevice(&cur);
    if (cur != h->dev)
        cudaSetDevice(h->dev);
    if (h->priv)
        cudaStreamDestroy(h->priv);
    if (h->host_ctl)
        cudaFreeHost(h->host_ctl);
    if (h->ws)
        cudaFree(h->ws);
    if (cur != h->dev && cur >= 0)
        cudaSetDevice(cur);
    cudaGetLastError();
    delete h;
}

sfar_status sfar_kv_plan(sfar_kv_t *h, const int32_t *lens, const int32_t *delta, int32_t *table, int32_t *ring,
                         const int32_t *state, int32_t *lens_out, int32_t *state_out, int32_t *starts, int32_t *slots,
                         int32_t *taken, size_t requests, size_t table_width, size_t tokens, sfar_stream_t s)
{
    if (!h || requests == 0 || requests > SFAR_KV_MAX_REQUESTS || table_width == 0 || table_width >= (1ull << 31) ||
        tokens >= (1ull << 31) || (tokens && !aligned(slots, 4)))
        return SFAR_ERR_INVALID;
    const Span spans[] = {Span(lens, requests * 4), Span(delta, requests * 4), Span(table, requests * table_width * 4),
                          Span(ring, h->pages * 4), Span(state, 8), Span(lens_out, requests * 4), Span(state_out, 8),
                          Span(starts, requests * 4 + 4), Span(slots, tokens * 4), Span(taken, requests * 4)};
    const int n = (int)(sizeof spans / sizeof spans[0]);
    for (int i = 0; i < n; ++i) {
        if (i != 8 && !aligned((const void *)spans[i].lo, 4))
            return SFAR_ERR_INVALID;
        for (int j = 0; j < i; ++j)
            if (spans[i].meets(spans[j]) && !((i == 5 && j == 0) || (i == 6 && j == 4)))
                return SFAR_ERR_INVALID;
    }
    if ((lens_out != lens && spans[5].meets(spans[0])) || (state_out != state && spans[6].meets(spans[4])))
        return SFAR_ERR_INVALID;
    SfarKvPlanArgs a{lens,  delta, table,  ring,          state,            lens_out,    state_out, starts,
                     slots, taken, h->ctl, (int)requests, (int)table_width, (int)tokens, h->shift,  (int)h->pages};
    // Small steps run on 8 CTAs of 256 threads, a request to a thread; large ones on all the CTAs that a cluster can have, of
    // 1024: their time is that of the instructions of the slots and pages.  Small and large form, us: requests of one token,
    // 64: 3.2, 4.0; 256: 3.5, 4.2; 257: 4.2, 4.2; 512: 4.6, 4.6; 1024: 6.3, 5.4; 8192: 32, 18.  16 requests with 1412 tokens
    // 4.5, 4.7; 128 with 2533 4.6, 4.9; 256 with 1767 5.7, 4.9, with 3088 4.9, 4.8, with 7118 6.6, 4.9; 64 with 7156 4.6, 4.6.
    const bool small = requests <= 256 && tokens <= 4096;
    const unsigned cluster = small ? SFAR_PLAN_CLUSTER : h->plan_ctas;
    return launch(h->dev, sfar_kernel_kv_plan(), dim3(cluster), small ? 256 : SFAR_PLAN_THREADS, (4 * requests + 1) * 4, &a, s, false, cluster);
}

sfar_status sfar_kv_append(sfar_kv_t *h, const void *const k[], const void *const v[], const int32_t *slots,
                           size_t tokens, size_t k_token_stride, size_t k_head_stride, size_t v_token_stride,
                           size_t v_head_stride, sfar_stream_t s)
{
    if (!h || !k || !v || tokens >= (1ull << 31) || (tokens && !aligned(slots, 4)) || k_token_stride % 8 ||
        k_head_stride % 8 || v_token_stride % 8 || v_head_stride % 8 ||
        (k_token_stride | k_head_stride | v_token_stride | v_head_stride) >> 40)
        return SFAR_ERR_INVALID;
    SfarKvAppendArgs a;
    memset(&a, 0, sizeof a);
    for (int r = 0; r < h->R; ++r) {
        if (tokens && (!aligned(k[r], 16) || !aligned(v[r], 16)))
            return SFAR_ERR_INVALID;
        a.x[0][r] = static_cast<const uint16_t *>(k[r]);
        a.x[1][r] = static_cast<const uint16_t *>(v[r]);
        for (int i = 0; i < 2; ++i) {
            a.cache[i][r] = static_cast<uint8_t *>(h->cache[i][r]);
            a.scale[i][r] = h->scale[i][r];
        }
    }
    if (tokens == 0)
        return SFAR_OK;
    a.slots = slots;
    a.ctl = h->ctl;
    a.ts[0] = (long long)k_token_stride;
    a.hs[0] = (long long)k_head_stride;
    a.ts[1] = (long long)v_token_stride;
    a.hs[1] = (long long)v_head_stride;
    a.T = (int)tokens;
    a.H = h->Hk;
    a.R = h->R;
    a.shift = h->shift;
    a.pages = (int)h->pages;
    // One token per CTA while that gives no more CTAs than eight per SM (few), then up to 32, doubling while there are
    // more than four per SM.
    const size_t planes = 2 * (size_t)h->R * (size_t)h->Hk;
    const bool few = tokens * ceil_div(planes, SFAR_APPEND_WARPS) <= 8 * (size_t)h->sms;
    int team = 1;
    const void *f = sfar_kernel_kv_append(h->D, 1 << h->shift, few, &team);
    const size_t groups = ceil_div(planes * (size_t)team, SFAR_APPEND_WARPS);
    a.window = 1;
    while (!few && a.window < 32 && ceil_div(tokens, (size_t)a.window) * groups > 4 * (size_t)h->sms)
        a.window *= 2;
    if (groups > 65535)
        return SFAR_ERR_INVALID;
    return launch(h->dev, f, dim3((unsigned)ceil_div(tokens, (size_t)a.window), (unsigned)groups), 32 * SFAR_APPEND_WARPS, 0, &a, s);
}

sfar_status sfar_kv_attention(sfar_kv_t *h, const void *const q[], void *const out[], const int32_t *table,
                              const int32_t *lens, const int32_t *starts, size_t requests, size_t table_width,
                              size_t tokens, size_t q_token_stride, size_t q_head_stride, size_t out_token_stride,
                              size_t out_head_stride, size_t max_q, float scale, size_t window, sfar_stream_t s)
{
    if (!h || !q || !out || requests == 0 || requests > SFAR_KV_MAX_REQUESTS || table_width == 0 ||
        table_width >= (1ull << 31) || tokens >= (1ull << 31) || !aligned(table, 4) || !aligned(lens, 4) ||
        !aligned(starts, 4) || q_token_stride % 8 || q_head_stride % 8 || out_token_stride % 8 || out_head_stride % 8 ||
        !(scale >= 0.f) || isinf(scale) || (q_token_stride | q_head_stride | out_token_stride | out_head_stride) >> 40)
        return SFAR_ERR_INVALID;
    if (tokens == 0)
        return SFAR_OK;
    // rows of out that share memory
    const size_t row = (size_t)h->D;
    if ((tokens > 1 && out_token_stride < row) || (h->Hq > 1 && out_head_stride < row) ||
        (tokens > 1 && h->Hq > 1 && out_token_stride == out_head_stride))
        return SFAR_ERR_INVALID;
    for (int i = 1; i < h->R; ++i)
        for (int j = 0; j < i; ++j)
            if (out[i] == out[j])
                return SFAR_ERR_INVALID;
    SfarAttnArgs a;
    memcpy(a.kmap, h->map[0], sizeof a.kmap);
    memcpy(a.vmap, h->map[1], sizeof a.vmap);
    auto extent = [&](size_t ts, size_t hs) { return 2 * ((tokens - 1) * ts + (size_t)(h->Hq - 1) * hs + (size_t)h->D); };
    const size_t qb = extent(q_token_stride, q_head_stride), ob = extent(out_token_stride, out_head_stride);
    for (int r = 0; r < h->R; ++r) {
        if (!aligned(q[r], 16) || !aligned(out[r], 16))
            return SFAR_ERR_INVALID;
        a.q[r] = static_cast<const uint16_t *>(q[r]);
        a.out[r] = static_cast<uint16_t *>(out[r]);
        a.v[r] = static_cast<const uint8_t *>(h->cache[1][r]);
        a.ks[r] = h->scale[0][r];
        a.vs[r] = h->scale[1][r];
    }
    for (int i = 0; i < h->R; ++i)
        for (int j = 0; j < h->R; ++j)
            if (Span(out[i], ob).meets(Span(q[j], qb)))
                return SFAR_ERR_INVALID;
    a.table = table;
    a.lens = lens;
    a.starts = starts;
    a.ctl = h->ctl;
    a.part = h->part;
    a.arrived = h->arrived;
    a.arrived_stride = 3 * h->sms;
    a.qts = (long long)q_token_stride;
    a.qhs = (long long)q_head_stride;
    a.ots = (long long)out_token_stride;
    a.ohs = (long long)out_head_stride;
    a.scale = scale;
    a.R = h->R;
    a.B = (int)requests;
    a.W = (int)table_width;
    a.T = (int)tokens;
    a.Hq = h->Hq;
    a.Hk = h->Hk;
    a.G = h->Hq / h->Hk;
    a.shift = h->shift;
    a.pages = (int)h->pages;
    a.window = window >= (1ull << 31) ? 0 : (int)window;
    const bool many = max_q > kFewRows / (size_t)a.G && requests <= SFAR_PROMPT_REQUESTS;
    const int rows = many ? SFAR_PROMPT_ROWS : max_q <= 8 / (size_t)a.G ? 8 : 16;
    // the kernels' sums over the line of (row tile, tile) are of 32 bits, its row numbers of 31
    const size_t most = tokens * (size_t)a.G / (size_t)rows + requests;
    const size_t context = table_width << h->shift, reach = context < (1ull << 31) ? context : 1ull << 31;
    if (tokens * (size_t)a.G >= 1ull << 29 || most * (ceil_div(reach, many ? 128 : SFAR_ATTN_TILE) + 8) >= 1ull << 32)
        return SFAR_ERR_INVALID;
    a.most = (int)most;
    int threads = 0, smem = 0;
    if (many) {
        const void *f = sfar_kernel_kv_prompt(h->D, &threads, &smem);
        return launch(h->dev, f, dim3((unsigned)h->sms), (unsigned)threads, (size_t)smem + (requests + 1) * 4, &a, s);
    }
    const void *f = sfar_kernel_kv_attn(h->D, rows, &threads, &smem);
    return launch(h->dev, f, dim3((unsigned)(h->sms * SFAR_ATTN_CTAS(rows))), (unsigned)threads, (size_t)smem + (requests + 1) * 4, &a, s);
}

sfar_status sfar_kv_status_get(sfar_kv_t *h, sfar_fault *info)
{
    if (!h)
        return SFAR_ERR_INVALID;
    if (cudaMemcpyAsync(h->host_ctl, h->ctl, 32, cudaMemcpyDeviceToHost, h->priv) != cudaSuccess ||
        cudaStreamSynchronize(h->priv) != cudaSuccess) {
        cudaGetLastError();
        return SFAR_ERR_CUDA;
    }
    const SfarCtl *c = h->host_ctl;
    const sfar_status code = (sfar_status)c->status;
    if (info) {
        info->code = code;
        info->rank = code ? c->f_rank : -1;
        info->cta = code ? c->f_cta : -1;
        info->peer = code ? c->f_peer : -1;
        info->epoch = code ? c->f_epoch : 0;
        info->where = code ? c->f_where : 0;
    }
    return code;
}

sfar_status sfar_kv_reset(sfar_kv_t *h, sfar_stream_t s)
{
    if (!h)
        return SFAR_ERR_INVALID;
    // the counters of parts too: a CTA that gave up has left them where they were
    if (cudaMemsetAsync(h->ctl, 0, 32, (cudaStream_t)s) != cudaSuccess ||
        cudaMemsetAsync(h->arrived, 0, arrived_bytes(h->sms), (cudaStream_t)s) != cudaSuccess) {
        cudaGetLastError();
        return SFAR_ERR_CUDA;
    }
    return SFAR_OK;
}

sfar_status sfar_test_kv_record_failure(sfar_kv_t *h)
{
    if (!h)
        return SFAR_ERR_INVALID;
    SfarCtl c;
    const size_t n = arrived_bytes(h->sms) / sizeof(int);
    std::unique_ptr<int[]> ones(new (std::nothrow) int[n]);
    if (!ones)
        return SFAR_ERR_OOM;
    std::fill_n(ones.get(), n, 1);
    if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpy(&c, h->ctl, sizeof c, cudaMemcpyDeviceToHost) != cudaSuccess)
        return SFAR_ERR_CUDA;
    c.status = SFAR_ERR_TIMEOUT;
    c.f_where = SFAR_WAIT_COPY;
    if (cudaMemcpy(h->ctl, &c, sizeof c, cudaMemcpyHostToDevice) != cudaSuccess ||
        cudaMemcpy(h->arrived, ones.get(), n * sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
        return SFAR_ERR_CUDA;
    return SFAR_OK;
}

// ---------------------------------------------------------- 8-bit projection
sfar_status sfar_quantize_fp8(sfar_t *h, const void *const x[], void *const x8[], float *const sx[], size_t m,
                              size_t k, size_t ldx, size_t ldx8, sfar_stream_t s)
{
    if (!h || !x || !x8 || !sx || m == 0 || k == 0 || m >= (1ull << 31) || k >= (1ull << 31) || ldx < k || ldx8 < k ||
        ldx >= (1ull << 40) || ldx8 >= (1ull << 40))
        return SFAR_ERR_INVALID;
    const SfarView v = sfar_view(h);
    if (v.dt != SFAR_BF16)
        return SFAR_ERR_INVALID;
    SfarQuantArgs a;
    memset(&a, 0, sizeof a);
    a.kb = (int)ceil_div(k, SFAR_FP8_BLOCK);
    a.vec = ldx % 8 == 0;
    a.vec8 = ldx8 % 8 == 0;
    const size_t xb = ((m - 1) * ldx + k) * 2, qb = (m - 1) * ldx8 + k, sb = (size_t)a.kb * m * 4;
    for (int r = 0; r < v.R; ++r) {
        if (!aligned(x[r], 2) || !x8[r] || !aligned(sx[r], 4))
            return SFAR_ERR_INVALID;
        a.vec = a.vec && aligned(x[r], 16);
        a.vec8 = a.vec8 && aligned(x8[r], 8);
        a.x[r] = static_cast<const uint16_t *>(x[r]);
        a.x8[r] = static_cast<uint8_t *>(x8[r]);
        a.sx[r] = sx[r];
    }
    for (int i = 0; i < v.R; ++i)
        for (int j = 0; j < v.R; ++j) {
            const Span q(x8[i], qb), sc(sx[i], sb), in(x[j], xb);
            if (q.meets(in) || sc.meets(in) || q.meets(Span(sx[j], sb)) ||
                (i < j && (q.meets(Span(x8[j], qb)) || sc.meets(Span(sx[j], sb)))))
                return SFAR_ERR_INVALID;
        }
    a.m = (long long)m;
    a.k = (long long)k;
    a.ldx = (long long)ldx;
    a.ldx8 = (long long)ldx8;
    a.R = v.R;
    const size_t rows = ceil_div(m, 8), cols = ceil_div(k, SFAR_QUANT_COLS);
    if (cols > 65535)
        return SFAR_ERR_INVALID;
    return launch(v.dev, sfar_kernel_quantize(), dim3((unsigned)rows, (unsigned)cols, (unsigned)v.R), 256, 0, &a, s,
                  v.mode == SFAR_LAUNCH_PLAIN);
}

sfar_status sfar_rowpar_gemm_fp8(sfar_t *h, const void *const x8[], const float *const sx[], const void *const w8[],
                                 const float *const sw[], void *const y[], size_t m, size_t k, size_t hidden,
                                 size_t ldx8, size_t ldw, sfar_stream_t s)
{
    if (!h || !x8 || !sx || !w8 || !sw || !y || m == 0 || k == 0 || hidden == 0 || m >= (1ull << 31) ||
        k >= (1ull << 31) || hidden >= (1ull << 31) || ldx8 < k || ldw < k || ldx8 % 16 || ldw % 16 ||
        ldx8 >= (1ull << 40) || ldw >= (1ull << 40))
        return SFAR_ERR_INVALID;
    const SfarView v = sfar_view(h);
    if (v.dt != SFAR_BF16)
        return SFAR_ERR_INVALID;
    const PFN_cuTensorMapEncodeTiled_v12000 encode =
        reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(sfar_tensor_map_encoder());
    if (!encode)
        return SFAR_ERR_UNSUPPORTED;
    const size_t kb = ceil_div(k, SFAR_FP8_BLOCK), nb = ceil_div(hidden, SFAR_FP8_BLOCK);
    const size_t xb = (m - 1) * ldx8 + k, wb = (hidden - 1) * ldw + k, yb = m * hidden * 2;
    SfarGemm8Args a;
    a.vec = hidden % 8 == 0;
    for (int r = 0; r < v.R; ++r) {
        if (!aligned(x8[r], 16) || !aligned(w8[r], 16) || !aligned(sx[r], 4) || !aligned(sw[r], 4) || !aligned(y[r], 2))
            return SFAR_ERR_INVALID;
        a.sx[r] = sx[r];
        a.sw[r] = sw[r];
        a.y[r] = static_cast<uint16_t *>(y[r]);
        a.vec = a.vec && aligned(y[r], 16);
    }
    for (int i = 0; i < v.R; ++i) {
        const Span out(y[i], yb);
        for (int j = 0; j < v.R; ++j)
            if (out.meets(Span(x8[j], xb)) || out.meets(Span(w8[j], wb)) || out.meets(Span(sx[j], kb * m * 4)) ||
                out.meets(Span(sw[j], nb * kb * 4)) || (i < j && out.meets(Span(y[j], yb))))
                return SFAR_ERR_INVALID;
    }
    const bool one = (size_t)v.R * ceil_div(m, 128) * ceil_div(hidden, 128) <= (size_t)v.sms;
    const int few = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : m <= kFewTokens || one ? 128 : 0;
    const cuuint32_t unit[2] = {1, 1}, wbox[2] = {SFAR_FP8_BLOCK, 128}, xbox[2] = {SFAR_FP8_BLOCK, few ? (cuuint32_t)few : 128u};
    auto map = [&](CUtensorMap *to, const void *p, size_t rows, size_t ld, const cuuint32_t *box) {
        const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
        return encode(to, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, unit,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    for (int r = 0; r < v.R; ++r)
        if (!map(&a.xmap[r], x8[r], m, ldx8, xbox) || !map(&a.wmap[r], w8[r], hidden, ldw, wbox))
            return SFAR_ERR_INVALID;
    a.ctl = v.ctl;
    a.m = (long long)m;
    a.n = (long long)hidden;
    a.R = v.R;
    a.kb = (int)kb;
    a.tiles_m = (int)ceil_div(m, few ? (size_t)few : 256);
    a.tiles_n = (int)ceil_div(hidden, few ? 128 : 256);
    const size_t tiles = (size_t)v.R * (size_t)a.tiles_m * (size_t)a.tiles_n;
    const size_t slots = few ? (size_t)v.sms : (size_t)v.sms / 2;
    const size_t grid = (tiles < slots ? tiles : slots) * (few ? 1 : 2);
    int threads = 0, smem = 0;
    const void *f = sfar_kernel_gemm8(few, &threads, &smem);
    return launch(v.dev, f, dim3((unsigned)grid), (unsigned)threads, (size_t)smem, &a, s, v.mode == SFAR_LAUNCH_PLAIN);
}

}  // extern "C"

int sfar_fp8_prepare()
{
    for (int few : {16, 32, 64, 128, 0}) {
        int threads = 0, smem = 0;
        const void *f = sfar_kernel_gemm8(few, &threads, &smem);
        const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return (int)e;
    }
    return 0;
}
