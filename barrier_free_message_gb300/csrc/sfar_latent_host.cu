// sfar_latent_host.cu -- the C ABI of the rotary positions (include/sfar_rope.h)
// and of the paged latent cache (include/sfar_latent.h): arguments, handle, launch.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <new>

#include "sfar_kv.h"
#include "sfar_latent.h"
#include "sfar_latent_args.h"
#include "sfar_launch.h"
#include "sfar_rope.h"
#include "sfar_test.h"

struct sfar_latent {
    int R = 0, Hq = 0, L = 0, rope = 0, shift = 0;
    size_t pages = 0;
    int dev = 0, sms = 0;
    void *cache[SFAR_MAX_R] = {};
    uint8_t *ws = nullptr;
    SfarCtl *ctl = nullptr;             // at the start of ws
    float *part = nullptr;              // attention: partial results and their counters, in ws
    int *arrived = nullptr;
    unsigned *next = nullptr;           // prompt: the counter of row tiles
    SfarCtl *host_ctl = nullptr;
    cudaStream_t priv = nullptr;
    unsigned plan_ctas = SFAR_PLAN_CLUSTER;
    CUtensorMap map[SFAR_MAX_R];        // the caches as the attention's copies see them
};

namespace {

// Counters: three sets of one for each part of a row tile (the absorbed form has one to a CTA), and one of the prompt's row
// tiles.
size_t counter_stride(int sms) { return SFAR_PROMPT_PARTS * (size_t)sms; }
size_t counter_bytes(int sms) { return (3 * counter_stride(sms) + 1) * sizeof(int); }

// A tensor [tokens][heads][numbers] in memory, in bytes; strides of dimensions of one entry do not count.
struct Rows {
    uintptr_t p;
    size_t ts, hs, row, ext, tokens, heads;     // ext: what lies between a token's first and last byte
    size_t whole;                       // from the first byte to past the last
    Rows(const void *ptr, size_t tokens, size_t heads, size_t row, size_t ts, size_t hs)
        : p((uintptr_t)ptr), ts(ts), hs(hs), row(row), ext((heads - 1) * hs + row), tokens(tokens), heads(heads), whole((tokens - 1) * ts + ext)
    {
    }
    bool every(size_t m) const { return (tokens == 1 || ts % m == 0) && (heads == 1 || hs % m == 0); }
    bool meets(const Rows &o) const
    {
        if (p >= o.p + o.whole || o.p >= p + whole)
            return false;
        // Slices of one tensor's last dimension: rows at places of one period that all strides are multiples of, where those
        // of the one lie beside those of the other.
        for (size_t m : {tokens > 1 ? ts : 0, heads > 1 ? hs : 0})
            if (m && every(m) && o.every(m)) {
                const size_t d = (o.p % m + m - p % m) % m;
                if (d >= row && d + o.row <= m)
                    return false;
            }
        // beside one another in rows of one length
        if (tokens > 1 && o.tokens > 1 && ts == o.ts && ext <= ts && o.ext <= ts) {
            const size_t d = (o.p >= p ? o.p - p : ts - (p - o.p) % ts) % ts;
            return d < ext || d + o.ext > ts;
        }
        return true;
    }
    bool meets(const Span &o) const { return p < o.hi && o.lo < p + whole; }
};
// Whether no row of [tokens][heads][row] lies in another: the rows along one of the dimensions fit the other's stride.
bool apart(size_t tokens, size_t heads, size_t row, size_t ts, size_t hs)
{
    if (heads > 1 && hs < row)
        return false;
    if (tokens > 1 && ts < row)
        return false;
    return tokens == 1 || heads == 1 || ts >= (heads - 1) * hs + row || hs >= (tokens - 1) * ts + row;
}
bool strides_fit(std::initializer_list<size_t> s, size_t of)
{
    for (size_t v : s)
        if (v % of || v >> 39)
            return false;
    return true;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() { return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(sfar_tensor_map_encoder()); }

}  // namespace

extern "C" {

// ------------------------------------------------------------ rotary positions
sfar_status sfar_rope(sfar_t *h, const void *const q[], void *const q_out[], const void *const k[], void *const k_out[],
                      const int32_t *pos, const float *freq, size_t tokens, size_t q_heads, size_t k_heads, size_t rot,
                      size_t q_token_stride, size_t q_head_stride, size_t q_out_token_stride, size_t q_out_head_stride,
                      size_t k_token_stride, size_t k_head_stride, size_t k_out_token_stride, size_t k_out_head_stride,
                      int layout, float scale, sfar_stream_t s)
{
    if (!h || (q_heads && (!q || !q_out)) || (k_heads && (!k || !k_out)) || q_heads + k_heads == 0 || q_heads > 65535 || k_heads > 65535 ||
        rot == 0 || rot % 16 || rot > 1024 || (q_heads + k_heads) * rot >= 1u << 22 || tokens >= (1ull << 31) || (layout != SFAR_ROPE_HALF && layout != SFAR_ROPE_INTERLEAVED) ||
        !isfinite(scale))
        return SFAR_ERR_INVALID;
    if (tokens == 0)
        return SFAR_OK;
    if (!aligned(pos, 4) || !aligned(freq, 4))
        return SFAR_ERR_INVALID;
    const SfarView v = sfar_view(h);
    const size_t each = v.dt == SFAR_BF16 ? 2 : 4;
    const size_t heads[2] = {q_heads, k_heads};
    const size_t its[2] = {q_token_stride, k_token_stride}, ihs[2] = {q_head_stride, k_head_stride};
    const size_t ots[2] = {q_out_token_stride, k_out_token_stride}, ohs[2] = {q_out_head_stride, k_out_head_stride};
    const void *const *in[2] = {q, k};
    void *const *out[2] = {q_out, k_out};
    SfarRopeArgs a;
    memset(&a, 0, sizeof a);
    for (int i = 0; i < 2; ++i) {
        if (!heads[i])
            continue;
        if (!strides_fit({its[i], ihs[i], ots[i], ohs[i]}, 16 / each) || !apart(tokens, heads[i], rot, ots[i], ohs[i]))
            return SFAR_ERR_INVALID;
        for (int r = 0; r < v.R; ++r) {
            if (!aligned(in[i][r], 16) || !aligned(out[i][r], 16))
                return SFAR_ERR_INVALID;
            a.in[i][r] = in[i][r];
            a.out[i][r] = out[i][r];
        }
        a.its[i] = (long long)its[i];
        a.ihs[i] = (long long)ihs[i];
        a.ots[i] = (long long)ots[i];
        a.ohs[i] = (long long)ohs[i];
        a.H[i] = (int)heads[i];
    }
    // an output meets no other tensor, and its own input only as a whole
    for (int i = 0; i < 2; ++i)
        for (int r = 0; heads[i] && r < v.R; ++r) {
            const Rows o(out[i][r], tokens, heads[i], rot * each, ots[i] * each, ohs[i] * each);
            if (o.meets(Span(pos, tokens * 4)) || o.meets(Span(freq, rot * 2)))
                return SFAR_ERR_INVALID;
            for (int j = 0; j < 2; ++j)
                for (int e = 0; heads[j] && e < v.R; ++e) {
                    const bool same = i == j && r == e;
                    const bool place = same && in[j][e] == out[i][r] && (tokens == 1 || its[i] == ots[i]) && (heads[i] == 1 || ihs[i] == ohs[i]);
                    if (!place && o.meets(Rows(in[j][e], tokens, heads[j], rot * each, its[j] * each, ihs[j] * each)))
                        return SFAR_ERR_INVALID;
                    if (!same && o.meets(Rows(out[j][e], tokens, heads[j], rot * each, ots[j] * each, ohs[j] * each)))
                        return SFAR_ERR_INVALID;
                }
        }
    a.pos = pos;
    a.freq = freq;
    a.scale = scale;
    a.T = (int)tokens;
    a.R = v.R;
    a.half = (int)(rot / 2);
    // a thread to 8 pairs, whole rows to a CTA, equally many to each
    const size_t rows = (size_t)v.R * (q_heads + k_heads), chunks = rot / 16;
    const size_t cuts = ceil_div(rows, SFAR_ROPE_THREADS / chunks);
    a.span = (int)ceil_div(rows, cuts);
    const unsigned threads = (unsigned)(ceil_div((size_t)a.span * chunks, 32) * 32);
    return launch(v.dev, sfar_kernel_rope(v.dt == SFAR_BF16 ? 0 : 1, layout == SFAR_ROPE_INTERLEAVED), dim3((unsigned)tokens, (unsigned)cuts),
                  threads, chunks * 80, &a, s, v.mode == SFAR_LAUNCH_PLAIN);
}

sfar_status sfar_rope_frequencies(float *freq, float *scale, size_t rot, double base, int scaling, double factor, double trained,
                                  double low, double high)
{
    const bool banded = scaling == SFAR_ROPE_WAVELENGTH || scaling == SFAR_ROPE_RAMP;
    if (!freq || !scale || rot == 0 || rot % 2 || rot > 65536 || !(base > 1) || !isfinite(base) || scaling < SFAR_ROPE_PLAIN ||
        scaling > SFAR_ROPE_RAMP || (scaling != SFAR_ROPE_PLAIN && (!(factor >= 1) || !isfinite(factor))) ||
        (banded && (!(trained > 0) || !isfinite(trained) || !(low > 0) || !(high > low) || !isfinite(high))))
        return SFAR_ERR_INVALID;
    const double pi = 3.14159265358979323846, n = (double)rot;
    double from = 0, to = 0;
    if (scaling == SFAR_ROPE_RAMP) {
        auto pair = [&](double turns) { return n * log(trained / (2 * pi * turns)) / (2 * log(base)); };
        from = std::max(floor(pair(high)), 0.0);
        to = std::min(ceil(pair(low)), n - 1);
    }
    for (size_t i = 0; i < rot / 2; ++i) {
        const double f = pow(base, -2.0 * (double)i / n);
        double y = f;
        if (scaling == SFAR_ROPE_LINEAR)
            y = f / factor;
        if (scaling == SFAR_ROPE_WAVELENGTH) {
            const double turns = trained * f / (2 * pi), s = (turns - low) / (high - low);
            y = turns > high ? f : turns < low ? f / factor : (1 - s) * f / factor + s * f;
        }
        if (scaling == SFAR_ROPE_RAMP) {
            const double s = std::min(1.0, std::max(0.0, ((double)i - from) / std::max(to - from, 0.001)));
            y = s * f / factor + (1 - s) * f;
        }
        freq[i] = (float)y;
    }
    *scale = scaling == SFAR_ROPE_RAMP ? (float)(0.1 * log(factor) + 1) : 1.f;
    return SFAR_OK;
}

// ----------------------------------------------------------------- latent cache
sfar_latent_t *sfar_latent_create(int R, int q_heads, int latent_dim, int rope_dim, int page_tokens, size_t pages,
                                  void *const cache[])
{
    auto fail = [](sfar_status st) {
        sfar_set_last_error(st);
        return (sfar_latent_t *)nullptr;
    };
    if (R < 1 || R > SFAR_MAX_R || q_heads < 1 || q_heads > 65535 || (latent_dim != 256 && latent_dim != 512) ||
        (rope_dim != 32 && rope_dim != 64) || (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && page_tokens != 128) ||
        pages == 0 || pages >= (1ull << 31) / (size_t)page_tokens || !cache)
        return fail(SFAR_ERR_INVALID);
    const size_t row = (size_t)(latent_dim + rope_dim), bytes = pages * (size_t)page_tokens * row * 2;
    for (int i = 0; i < R; ++i) {
        if (!aligned(cache[i], 16))
            return fail(SFAR_ERR_INVALID);
        for (int j = 0; j < i; ++j)
            if (Span(cache[i], bytes).meets(Span(cache[j], bytes)))
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
    const PFN_cuTensorMapEncodeTiled_v12000 encode = encoder();
    if (major != 10 || minor != 3 || !encode)
        return fail(SFAR_ERR_UNSUPPORTED);
    sfar_latent *h = new (std::nothrow) sfar_latent();
    if (!h)
        return fail(SFAR_ERR_OOM);
    h->R = R;
    h->Hq = q_heads;
    h->L = latent_dim;
    h->rope = rope_dim;
    h->shift = page_tokens == 16 ? 4 : page_tokens == 32 ? 5 : page_tokens == 64 ? 6 : 7;
    h->pages = pages;
    h->dev = dev;
    h->sms = sms;
    const cuuint64_t dims[3] = {(cuuint64_t)row, (cuuint64_t)page_tokens, (cuuint64_t)pages};
    const cuuint64_t strides[2] = {(cuuint64_t)row * 2, (cuuint64_t)row * 2 * (cuuint64_t)page_tokens};
    const cuuint32_t unit[3] = {1, 1, 1}, box[3] = {64, (cuuint32_t)std::min(page_tokens, SFAR_LATENT_TILE), 1};
    for (int r = 0; r < R; ++r) {
        h->cache[r] = cache[r];
        if (encode(&h->map[r], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, cache[r], dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
            delete h;
            return fail(SFAR_ERR_INVALID);
        }
    }
    const size_t o_arrived = 256, o_part = (o_arrived + counter_bytes(sms) + 255) / 256 * 256;
    const size_t absorbed = 2 * SFAR_LATENT_ROWS * ((size_t)latent_dim + 2), expanded = SFAR_PROMPT_PARTS * 256 * (size_t)(128 + 2);
    const size_t ws = o_part + (size_t)sms * std::max(absorbed, expanded) * 4;
    if (cudaMalloc(&h->ws, ws) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return fail(SFAR_ERR_OOM);
    }
    h->ctl = reinterpret_cast<SfarCtl *>(h->ws);
    h->arrived = reinterpret_cast<int *>(h->ws + o_arrived);
    h->next = reinterpret_cast<unsigned *>(h->arrived + 3 * counter_stride(sms));
    h->part = reinterpret_cast<float *>(h->ws + o_part);
    const SfarCtl init = fresh_ctl();
    bool ok = cudaMemset(h->ws, 0, ws) == cudaSuccess && cudaMemcpy(h->ctl, &init, sizeof init, cudaMemcpyHostToDevice) == cudaSuccess &&
              cudaStreamCreateWithFlags(&h->priv, cudaStreamNonBlocking) == cudaSuccess &&
              cudaMallocHost(&h->host_ctl, sizeof(SfarCtl)) == cudaSuccess && sfar_pool_prepare(&h->plan_ctas);
    auto room = [&](const void *f, int smem) { ok = ok && cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess; };
    int threads = 0, smem = 0;
    for (int rows : {16, 32, 64}) {
        const void *f = sfar_kernel_latent_attn(latent_dim, rows, &threads, &smem);
        room(f, smem);
    }
    for (int tiles : {1, 2})
        for (int dim : {64, 128}) {
            const void *f = sfar_kernel_latent_prompt(dim, tiles, &threads, &smem);
            room(f, smem);
        }
    if (!ok) {
        cudaGetLastError();
        sfar_latent_destroy(h);
        return fail(SFAR_ERR_CUDA);
    }
    sfar_set_last_error(SFAR_OK);
    return h;
}

void sfar_latent_destroy(sfar_latent_t *h)
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

sfar_status sfar_latent_plan(sfar_latent_t *h, const int32_t *lens, const int32_t *delta, int32_t *table, int32_t *ring,
                             const int32_t *state, int32_t *lens_out, int32_t *state_out, int32_t *starts, int32_t *slots,
                             int32_t *taken, size_t requests, size_t table_width, size_t tokens, sfar_stream_t s)
{
    if (!h)
        return SFAR_ERR_INVALID;
    return sfar_pool_plan(SfarPool{h->dev, h->shift, h->pages, h->ctl, h->plan_ctas}, lens, delta, table, ring, state, lens_out,
                          state_out, starts, slots, taken, requests, table_width, tokens, s);
}

sfar_status sfar_latent_append(sfar_latent_t *h, const void *const x[], const void *weight, const int32_t *pos,
                               const float *freq, const int32_t *slots, size_t tokens, size_t token_stride, float eps,
                               int layout, float scale, sfar_stream_t s)
{
    if (!h || !x || tokens >= (1ull << 31) || !strides_fit({token_stride}, 8) || !(eps >= 0.f) || isinf(eps) || !isfinite(scale) ||
        (layout != SFAR_ROPE_HALF && layout != SFAR_ROPE_INTERLEAVED))
        return SFAR_ERR_INVALID;
    if (tokens == 0)
        return SFAR_OK;
    const size_t row = (size_t)(h->L + h->rope);
    if (!aligned(weight, 16) || !aligned(pos, 4) || !aligned(freq, 4) || !aligned(slots, 4) || (tokens > 1 && token_stride < row))
        return SFAR_ERR_INVALID;
    SfarLatentAppendArgs a;
    memset(&a, 0, sizeof a);
    const size_t bytes = 2 * ((tokens - 1) * token_stride + row), cached = (h->pages << h->shift) * row * 2;
    for (int r = 0; r < h->R; ++r) {
        if (!aligned(x[r], 16))
            return SFAR_ERR_INVALID;
        const Span cache(h->cache[r], cached);
        for (int j = 0; j < h->R; ++j)
            if (cache.meets(Span(x[j], bytes)))
                return SFAR_ERR_INVALID;
        if (cache.meets(Span(weight, 2 * (size_t)h->L)) || cache.meets(Span(pos, 4 * tokens)) || cache.meets(Span(slots, 4 * tokens)) ||
            cache.meets(Span(freq, 2 * (size_t)h->rope)))
            return SFAR_ERR_INVALID;
        a.x[r] = static_cast<const uint16_t *>(x[r]);
        a.cache[r] = static_cast<uint16_t *>(h->cache[r]);
    }
    a.weight = static_cast<const uint16_t *>(weight);
    a.pos = pos;
    a.slots = slots;
    a.freq = freq;
    a.ctl = h->ctl;
    a.ts = (long long)token_stride;
    a.eps = eps;
    a.scale = scale;
    a.T = (int)tokens;
    a.R = h->R;
    a.rope = h->rope;
    a.slot_end = (int)(h->pages << h->shift);
    a.inter = layout == SFAR_ROPE_INTERLEAVED;
    const size_t ctas = ceil_div(tokens * (size_t)h->R, SFAR_LATENT_APPEND_WARPS);
    if (ctas >= (1ull << 31))
        return SFAR_ERR_INVALID;
    return launch(h->dev, sfar_kernel_latent_append(h->L), dim3((unsigned)ctas), 32 * SFAR_LATENT_APPEND_WARPS, 0, &a, s);
}

sfar_status sfar_latent_gather(sfar_latent_t *h, void *const out[], const int32_t *table, const int32_t *lens,
                               const int32_t *starts, size_t requests, size_t table_width, size_t tokens,
                               size_t token_stride, sfar_stream_t s)
{
    if (!h || !out || requests == 0 || requests > SFAR_KV_MAX_REQUESTS || table_width == 0 || table_width >= (1ull << 31) ||
        tokens >= (1ull << 31) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(starts, 4) || !strides_fit({token_stride}, 8))
        return SFAR_ERR_INVALID;
    if (tokens == 0)
        return SFAR_OK;
    const size_t row = (size_t)(h->L + h->rope);
    if (tokens > 1 && token_stride < row)
        return SFAR_ERR_INVALID;
    SfarLatentGatherArgs a;
    memset(&a, 0, sizeof a);
    const size_t bytes = 2 * ((tokens - 1) * token_stride + row), cached = (h->pages << h->shift) * row * 2;
    for (int r = 0; r < h->R; ++r) {
        if (!aligned(out[r], 16))
            return SFAR_ERR_INVALID;
        const Rows o(out[r], tokens, 1, 2 * row, 2 * token_stride, 0);
        const Span all(out[r], bytes);
        for (int j = 0; j < h->R; ++j)
            if (all.meets(Span(h->cache[j], cached)) || (j < r && o.meets(Rows(out[j], tokens, 1, 2 * row, 2 * token_stride, 0))))
                return SFAR_ERR_INVALID;
        if (all.meets(Span(table, requests * table_width * 4)) || all.meets(Span(lens, requests * 4)) || all.meets(Span(starts, requests * 4 + 4)))
            return SFAR_ERR_INVALID;
        a.cache[r] = static_cast<const uint16_t *>(h->cache[r]);
        a.out[r] = static_cast<uint16_t *>(out[r]);
    }
    a.table = table;
    a.lens = lens;
    a.starts = starts;
    a.ctl = h->ctl;
    a.ots = (long long)token_stride;
    a.B = (int)requests;
    a.W = (int)table_width;
    a.T = (int)tokens;
    a.vecs = (int)(row / 8);
    a.shift = h->shift;
    a.pages = (int)h->pages;
    return launch(h->dev, sfar_kernel_latent_gather(),
                  dim3((unsigned)ceil_div(tokens, SFAR_GATHER_WARPS * SFAR_GATHER_ROWS), (unsigned)h->R), 32 * SFAR_GATHER_WARPS, 0, &a, s);
}

sfar_status sfar_latent_attention(sfar_latent_t *h, const void *const q[], void *const out[], const int32_t *table,
                                  const int32_t *lens, const int32_t *starts, size_t requests, size_t table_width,
                                  size_t tokens, size_t q_token_stride, size_t q_head_stride, size_t out_token_stride,
                                  size_t out_head_stride, size_t max_q, float scale, sfar_stream_t s)
{
    if (!h || !q || !out || requests == 0 || requests > SFAR_KV_MAX_REQUESTS || table_width == 0 || table_width >= (1ull << 31) ||
        tokens >= (1ull << 31) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(starts, 4) ||
        !strides_fit({q_token_stride, q_head_stride, out_token_stride, out_head_stride}, 8) || !(scale >= 0.f) || isinf(scale))
        return SFAR_ERR_INVALID;
    if (tokens == 0)
        return SFAR_OK;
    const size_t H = (size_t)h->Hq, L = (size_t)h->L, row = L + (size_t)h->rope;
    if (!apart(tokens, H, L, out_token_stride, out_head_stride))
        return SFAR_ERR_INVALID;
    SfarLatentAttnArgs a;
    memcpy(a.map, h->map, sizeof a.map);
    const size_t cached = (h->pages << h->shift) * row * 2;
    for (int r = 0; r < h->R; ++r) {
        if (!aligned(q[r], 16) || !aligned(out[r], 16))
            return SFAR_ERR_INVALID;
        a.q[r] = static_cast<const uint16_t *>(q[r]);
        a.out[r] = static_cast<uint16_t *>(out[r]);
    }
    for (int i = 0; i < h->R; ++i) {
        const Rows o(out[i], tokens, H, 2 * L, 2 * out_token_stride, 2 * out_head_stride);
        for (int j = 0; j < h->R; ++j)
            if (o.meets(Rows(q[j], tokens, H, 2 * row, 2 * q_token_stride, 2 * q_head_stride)) || o.meets(Span(h->cache[j], cached)) ||
                (j < i && o.meets(Rows(out[j], tokens, H, 2 * L, 2 * out_token_stride, 2 * out_head_stride))))
                return SFAR_ERR_INVALID;
        if (o.meets(Span(table, requests * table_width * 4)) || o.meets(Span(lens, requests * 4)) || o.meets(Span(starts, requests * 4 + 4)))
            return SFAR_ERR_INVALID;
    }
    a.table = table;
    a.lens = lens;
    a.starts = starts;
    a.part = h->part;
    a.arrived = h->arrived;
    a.arrived_stride = (int)counter_stride(h->sms);
    a.ctl = h->ctl;
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
    a.shift = h->shift;
    a.pages = (int)h->pages;
    a.rope = h->rope;
    // As few rows as hold a request's: their products and softmax are what a tile costs beside its bytes (64 requests of 2000
    // tokens, 16 heads, 8 ranks: 200 us with 16 rows, 204 with 32, 258 with 64; 300 of 60 tokens 67, 75 and 101; 32 of 3000, 32
    // heads: 159 with 32, 197 with 64; 16 of 2000, 40 heads: 113 and 85).
    const int rows = max_q <= 16 / H ? 16 : max_q <= 32 / H ? 32 : 64;
    // the kernel's sums over the line of (row tile, tile) are of 32 bits, its row numbers of 31
    const size_t context = table_width << h->shift, reach = context < (1ull << 31) ? context : 1ull << 31;
    if (tokens * H >= 1ull << 29 || (tokens * H / 16 + requests) * (ceil_div(reach, SFAR_LATENT_TILE) + 8) >= 1ull << 32)
        return SFAR_ERR_INVALID;
    a.most = (int)(tokens * H / (size_t)rows + requests);
    const size_t step = H > 1 ? q_head_stride : q_token_stride;        // of a row
    a.q_flat = tokens * H == 1 || (step >= row && (H == 1 || tokens == 1 || q_token_stride == H * q_head_stride));
    if (a.q_flat) {
        const cuuint64_t dims[2] = {(cuuint64_t)row, (cuuint64_t)(tokens * H)}, strides[1] = {(cuuint64_t)(tokens * H == 1 ? row : step) * 2};
        const cuuint32_t unit[2] = {1, 1}, box[2] = {64, (cuuint32_t)rows};
        const PFN_cuTensorMapEncodeTiled_v12000 encode = encoder();
        for (int r = 0; r < h->R; ++r)
            if (!encode || encode(&a.qmap[r], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(q[r]), dims, strides, box, unit,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return encode ? SFAR_ERR_INVALID : SFAR_ERR_UNSUPPORTED;
    }
    int threads = 0, smem = 0;
    const void *f = sfar_kernel_latent_attn(h->L, rows, &threads, &smem);
    return launch(h->dev, f, dim3((unsigned)h->sms), (unsigned)threads, (size_t)smem, &a, s);
}

sfar_status sfar_latent_prompt(sfar_latent_t *h, const void *const q[], const void *const k[], const void *const v[],
                               const void *const kr[], void *const out[], const int32_t *starts, const int32_t *k_starts,
                               size_t requests, size_t tokens, size_t k_tokens, size_t head_dim, size_t q_token_stride,
                               size_t q_head_stride, size_t k_token_stride, size_t k_head_stride, size_t v_token_stride,
                               size_t v_head_stride, size_t kr_token_stride, size_t out_token_stride,
                               size_t out_head_stride, size_t max_q, float scale, sfar_stream_t s)
{
    if (!h || !q || !out || requests == 0 || requests > SFAR_KV_MAX_REQUESTS || tokens >= (1ull << 31) - 1024 ||
        k_tokens >= (1ull << 31) - 1024 || (head_dim != 64 && head_dim != 128) || !aligned(starts, 4) || !aligned(k_starts, 4) ||
        !strides_fit({q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride, kr_token_stride,
                      out_token_stride, out_head_stride},
                     8) ||
        !(scale >= 0.f) || isinf(scale) || (k_tokens && (!k || !v || !kr)))
        return SFAR_ERR_INVALID;
    if (tokens == 0)
        return SFAR_OK;
    const size_t H = (size_t)h->Hq, D = head_dim, rope = (size_t)h->rope, S = k_tokens;
    // a copy needs a stride above 0, and a tensor of at least a row
    auto moves = [&](size_t n, size_t ts, size_t hs, size_t heads) { return (n <= 1 || ts > 0) && (heads <= 1 || hs > 0); };
    if (!apart(tokens, H, D, out_token_stride, out_head_stride) || !moves(tokens, q_token_stride, q_head_stride, H) ||
        !moves(S, k_token_stride, k_head_stride, H) || !moves(S, v_token_stride, v_head_stride, H) || !moves(S, kr_token_stride, 0, 1))
        return SFAR_ERR_INVALID;
    const PFN_cuTensorMapEncodeTiled_v12000 encode = encoder();
    if (!encode)
        return SFAR_ERR_UNSUPPORTED;
    SfarLatentPromptArgs a;
    memset(&a, 0, sizeof a);
    const cuuint32_t unit[3] = {1, 1, 1}, box[3] = {64, 1, 128}, flat[2] = {64, 128};
    auto map = [&](CUtensorMap *to, const void *p, size_t row, size_t heads, size_t n, size_t ts, size_t hs) {
        const cuuint64_t dims[3] = {row, heads, n}, strides[2] = {heads > 1 ? 2 * hs : 2 * row, n > 1 ? 2 * ts : 2 * row * heads};
        return encode(to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    for (int r = 0; r < h->R; ++r) {
        if (!aligned(q[r], 16) || !aligned(out[r], 16) || (S && (!aligned(k[r], 16) || !aligned(v[r], 16) || !aligned(kr[r], 16))))
            return SFAR_ERR_INVALID;
        a.v[r] = S ? static_cast<const uint16_t *>(v[r]) : nullptr;
        a.out[r] = static_cast<uint16_t *>(out[r]);
    }
    for (int i = 0; i < h->R; ++i) {
        const Rows o(out[i], tokens, H, 2 * D, 2 * out_token_stride, 2 * out_head_stride);
        for (int j = 0; j < h->R; ++j)
            if (o.meets(Rows(q[j], tokens, H, 2 * (D + rope), 2 * q_token_stride, 2 * q_head_stride)) ||
                (S && (o.meets(Rows(k[j], S, H, 2 * D, 2 * k_token_stride, 2 * k_head_stride)) ||
                       o.meets(Rows(v[j], S, H, 2 * D, 2 * v_token_stride, 2 * v_head_stride)) ||
                       o.meets(Rows(kr[j], S, 1, 2 * rope, 2 * kr_token_stride, 0)))) ||
                (j < i && o.meets(Rows(out[j], tokens, H, 2 * D, 2 * out_token_stride, 2 * out_head_stride))))
                return SFAR_ERR_INVALID;
        if (o.meets(Span(starts, requests * 4 + 4)) || o.meets(Span(k_starts, requests * 4 + 4)))
            return SFAR_ERR_INVALID;
    }
    for (int r = 0; r < h->R; ++r) {
        if (!map(&a.qmap[r], q[r], D + rope, H, tokens, q_token_stride, q_head_stride))
            return SFAR_ERR_INVALID;
        if (S) {
            const cuuint64_t dims[2] = {(cuuint64_t)rope, (cuuint64_t)S}, strides[1] = {S > 1 ? 2 * kr_token_stride : 2 * rope};
            if (!map(&a.kmap[r], k[r], D, H, S, k_token_stride, k_head_stride) || !map(&a.vmap[r], v[r], D, H, S, v_token_stride, v_head_stride) ||
                encode(&a.krmap[r], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(kr[r]), dims, strides, flat, unit,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return SFAR_ERR_INVALID;
        } else {
            a.kmap[r] = a.vmap[r] = a.krmap[r] = a.qmap[r];     // never read
        }
    }
    a.starts = starts;
    a.kstarts = k_starts;
    a.next = h->next;
    a.part = h->part;
    a.arrived = h->arrived;
    a.arrived_stride = (int)counter_stride(h->sms);
    a.ctl = h->ctl;
    a.vts = (long long)v_token_stride;
    a.vhs = (long long)v_head_stride;
    a.ots = (long long)out_token_stride;
    a.ohs = (long long)out_head_stride;
    a.scale = scale;
    a.R = h->R;
    a.B = (int)requests;
    a.T = (int)tokens;
    a.S = (int)S;
    a.Hq = h->Hq;
    a.rope = h->rope;
    // Two tiles of 128 rows at a time read keys and values once for both and let one's products run beside the other's softmax
    // (8 ranks, 8 heads, 4 requests of 900 tokens after 1100: 229 us against 343); one leaves no half empty (128 tokens each: 66
    // against 72) and, where row tiles are few, gives twice as many to the SMs (one request of 1000 tokens, 8 heads: 32 us
    // against 36; after 7000 tokens 78 against 83; 16 heads 35 against 39, but 123 against 99).
    const int tiles = max_q <= 128 || tokens * H * (size_t)h->R / 128 <= (size_t)h->sms * 2 / 3 ? 1 : 2;
    const size_t most = tokens / (128 * (size_t)tiles) + requests;
    if ((tokens / 128 + requests) * H * (size_t)h->R >= 1ull << 31)
        return SFAR_ERR_INVALID;
    a.most = (int)most;
    int threads = 0, smem = 0;
    const void *f = sfar_kernel_latent_prompt((int)D, tiles, &threads, &smem);
    // no more CTAs than there can be row tiles and, where these are few, parts of theirs
    const size_t grid = std::min((size_t)h->sms, most * H * (size_t)h->R * (S / 512 + 1));
    return launch(h->dev, f, dim3((unsigned)grid), (unsigned)threads, (size_t)smem, &a, s);
}

sfar_status sfar_latent_status_get(sfar_latent_t *h, sfar_fault *info)
{
    return h ? read_ctl(h->ctl, h->host_ctl, h->priv, info) : SFAR_ERR_INVALID;
}

sfar_status sfar_latent_reset(sfar_latent_t *h, sfar_stream_t s)
{
    if (!h)
        return SFAR_ERR_INVALID;
    // the counters too: a CTA that gave up has left them where they were
    if (cudaMemsetAsync(h->ctl, 0, 32, (cudaStream_t)s) != cudaSuccess ||
        cudaMemsetAsync(h->arrived, 0, counter_bytes(h->sms), (cudaStream_t)s) != cudaSuccess) {
        cudaGetLastError();
        return SFAR_ERR_CUDA;
    }
    return SFAR_OK;
}

sfar_status sfar_test_latent_record_failure(sfar_latent_t *h)
{
    return h ? record_failure(h->ctl, h->arrived, counter_bytes(h->sms) / sizeof(int)) : SFAR_ERR_INVALID;
}

}  // extern "C"
