// sfar_kv_args.h -- kernel parameters of the paged 8-bit cache's operators and of
// the 8-bit projection.
#pragma once
#include <cuda.h>

#include "sfar_internal.h"

// What the translation units beside the AllReduce's need of a handle.
struct SfarView {
    int R, dt, dev, sms, mode;
    SfarCtl *ctl;
};
struct sfar;
SfarView sfar_view(const sfar *h);
// sets what sfar_last_error reports
void sfar_set_last_error(int status);
// The driver's cuTensorMapEncodeTiled (PFN_cuTensorMapEncodeTiled_v12000), or NULL.
extern "C" void *sfar_tensor_map_encoder();

struct SfarKvPlanArgs {
    const int *lens, *delta;
    int *table, *ring;
    const int *state;
    int *lens_out, *state_out, *starts, *slots, *taken;
    SfarCtl *ctl;
    int B, W, T, shift, pages;      // requests, table width, token rows, log2 page_tokens, pool
};

struct SfarKvAppendArgs {
    const uint16_t *x[2][SFAR_MAX_R];       // new keys, values
    uint8_t *cache[2][SFAR_MAX_R];
    float *scale[2][SFAR_MAX_R];
    const int *slots;
    SfarCtl *ctl;
    long long ts[2], hs[2];                 // strides of a token and of a head, elements
    int T, H, R, shift, pages, window;      // window: tokens per CTA
};

struct SfarAttnArgs {
    // caches of every rank as 3-D tensor maps: head_dim bytes (innermost) by
    // page_tokens by pages * kv_heads, a box of up to SFAR_ATTN_TILE tokens
    CUtensorMap kmap[SFAR_MAX_R];
    CUtensorMap vmap[SFAR_MAX_R];
    const uint8_t *v[SFAR_MAX_R];           // the value caches
    const float *ks[SFAR_MAX_R], *vs[SFAR_MAX_R];
    const uint16_t *q[SFAR_MAX_R];
    uint16_t *out[SFAR_MAX_R];
    const int *table, *lens, *starts;
    float *part;                            // partial results, two per CTA
    int *arrived;                           // [6][arrived_stride] counters of parts (SfarJoin); 0 between calls
    SfarCtl *ctl;
    long long qts, qhs, ots, ohs;
    float scale;
    int R, B, W, T, Hq, Hk, G, shift, pages, window, arrived_stride;
    int most;                               // row tiles of all requests, at most
};

struct SfarQuantArgs {
    const uint16_t *x[SFAR_MAX_R];
    uint8_t *x8[SFAR_MAX_R];
    float *sx[SFAR_MAX_R];
    long long m, k, ldx, ldx8;
    int R, kb, vec, vec8;                   // 16-byte loads, 8-byte stores are aligned
};

struct SfarGemm8Args {
    // x8 and w8 of every rank as 2-D tensor maps: k bytes (innermost) by rows,
    // boxes of 128 bytes x the tile's tokens (x) or 128 rows (w), 128-byte
    // swizzle, zeros outside
    CUtensorMap xmap[SFAR_MAX_R];
    CUtensorMap wmap[SFAR_MAX_R];
    const float *sx[SFAR_MAX_R], *sw[SFAR_MAX_R];
    uint16_t *y[SFAR_MAX_R];
    SfarCtl *ctl;
    long long m, n;
    int R, kb, tiles_m, tiles_n, vec;       // vec: rows of y are 16-byte aligned
};

const void *sfar_kernel_kv_plan();
// few: for a decode step; *team: warps to a run
const void *sfar_kernel_kv_append(int head_dim, int page_tokens, int few, int *team);
const void *sfar_kernel_kv_attn(int head_dim, int rows, int *threads, int *smem);
const void *sfar_kernel_kv_prompt(int head_dim, int *threads, int *smem);
const void *sfar_kernel_quantize();
const void *sfar_kernel_gemm8(int tokens, int *threads, int *smem);
// once per device: what the 8-bit projection's kernels need of it; 0 or a cudaError_t
int sfar_fp8_prepare();

#define SFAR_PLAN_THREADS 1024
#define SFAR_PLAN_CLUSTER 8                 // twice that for many requests or tokens
#define SFAR_QUANT_COLS 1024                // columns a warp of the quantisation takes of a row
#define SFAR_APPEND_WARPS 8
#define SFAR_ATTN_TILE 64
#define SFAR_ATTN_CTAS(rows) ((rows) == 8 ? 3 : 2)   // per SM
#define SFAR_PROMPT_ROWS 256
#define SFAR_PROMPT_REQUESTS 2048           // whose prefix sums fit beside the prompt kernel's tiles
