// sfar_latent_args.h -- kernel parameters of the rotary positions and of the
// paged latent cache's operators.
#pragma once
#include <cuda.h>

#include "sfar_internal.h"
#include "sfar_kv_args.h"

struct SfarRopeArgs {
    const void *in[2][SFAR_MAX_R];          // queries, keys
    void *out[2][SFAR_MAX_R];
    const int *pos;
    const float *freq;
    long long its[2], ihs[2], ots[2], ohs[2];   // strides of a token and of a head, elements
    float scale;
    int T, R, H[2], half;                   // half: pairs of a row
    int span;                               // (rank, head) rows of a token that a CTA takes
};

struct SfarLatentAppendArgs {
    const uint16_t *x[SFAR_MAX_R];
    uint16_t *cache[SFAR_MAX_R];
    const uint16_t *weight;
    const int *pos, *slots;
    const float *freq;
    SfarCtl *ctl;
    long long ts;
    float eps, scale;
    int T, R, rope, slot_end, inter;        // slot_end: slots of the pool; inter: interleaved pairs
};

struct SfarLatentGatherArgs {
    const uint16_t *cache[SFAR_MAX_R];
    uint16_t *out[SFAR_MAX_R];
    const int *table, *lens, *starts;
    SfarCtl *ctl;
    long long ots;
    int B, W, T, vecs, shift, pages;        // vecs: 16-byte vectors of a row
};

struct SfarLatentAttnArgs {
    // caches of every rank as 3-D tensor maps: a row's numbers (innermost) by
    // page_tokens by pages; boxes of 64 numbers by up to 64 tokens, 128-byte swizzle
    CUtensorMap map[SFAR_MAX_R];
    // q_flat: query rows (tokens, their heads) lie one stride apart, and are 2-D tensor maps too; boxes of 64 numbers by a row
    // tile, zeros past the last row
    CUtensorMap qmap[SFAR_MAX_R];
    const uint16_t *q[SFAR_MAX_R];
    uint16_t *out[SFAR_MAX_R];
    const int *table, *lens, *starts;
    float *part;                            // partial results, two per CTA
    int *arrived;                           // [3][arrived_stride] counters of parts (SfarJoin); 0 between calls
    SfarCtl *ctl;
    long long qts, qhs, ots, ohs;
    float scale;
    int R, B, W, T, Hq, shift, pages, rope, arrived_stride, q_flat;
    int most;                               // row tiles of all requests, at most
};

struct SfarLatentPromptArgs {
    // per rank, 3-D tensor maps: numbers of a head (innermost) by heads by tokens, boxes of 64 numbers of one head of 128 tokens,
    // 128-byte swizzle, zeros outside; kr 2-D
    CUtensorMap qmap[SFAR_MAX_R], kmap[SFAR_MAX_R], vmap[SFAR_MAX_R], krmap[SFAR_MAX_R];
    const uint16_t *v[SFAR_MAX_R];          // values that are not finite are read again
    uint16_t *out[SFAR_MAX_R];
    const int *starts, *kstarts;
    unsigned *next;                         // counter of row tiles taken; 0 between calls
    float *part;                            // partial results, SFAR_PROMPT_PARTS for each SM
    int *arrived;                           // [3][arrived_stride] counters of parts (SfarJoin); 0 between calls
    int arrived_stride;
    SfarCtl *ctl;
    long long vts, vhs, ots, ohs;
    float scale;
    int R, B, T, S, Hq, rope;               // T, S: rows of q, of k
    int most;                               // row tiles of all requests, at most
};

// Dtype: 0 bf16, 1 fp32.
const void *sfar_kernel_rope(int dt, int interleaved);
const void *sfar_kernel_latent_append(int latent);
const void *sfar_kernel_latent_gather();
// rows: 16, 32 or 64 at a time
const void *sfar_kernel_latent_attn(int latent, int rows, int *threads, int *smem);
// tiles: 128 query rows at a time, or twice that
const void *sfar_kernel_latent_prompt(int head_dim, int tiles, int *threads, int *smem);

#define SFAR_ROPE_THREADS 256
#define SFAR_LATENT_APPEND_WARPS 8
#define SFAR_GATHER_WARPS 8
#define SFAR_LATENT_TILE 64                // cached tokens of a step of the attention
#define SFAR_LATENT_ROWS 64                 // query rows at a time, at most
#define SFAR_PROMPT_PARTS 2                 // parts of row tiles that the expanded attention makes, for each SM
#define SFAR_LATENT_GROUP 32                // requests to a prefix sum
#define SFAR_GATHER_ROWS 4                  // rows of a warp
