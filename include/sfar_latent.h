/*
 * sfar_latent.h -- attention whose keys and values come from one latent
 * vector a token, for R simulated ranks on one GB300: the paged cache of
 * latents, and attention in its absorbed and its expanded form.
 *
 * A token is held as a row of latent_dim + rope_dim numbers in bf16: its
 * normalised latent c and its rotated key kr, both shared by all heads.  Key
 * and value of head h are (U_h c, kr) and V_h c.
 *   absorbed   U_h is multiplied into the query and V_h onto the result, by
 *              the caller: attention over the rows as they are cached, with
 *              q = (U_h^T q', q_rot) of latent_dim + rope_dim numbers and
 *              results of latent_dim.  Reads a row once for all heads: for
 *              steps of few tokens.
 *   expanded   keys U_h c and values V_h c are computed first, from rows read
 *              back by sfar_latent_gather: fewer products for each pair of
 *              tokens.  For prompts.
 * The cache of rank r is cache[r]: [pages][page_tokens][latent_dim +
 * rope_dim].  Block tables, slots, plan and statuses are those of sfar_kv.h,
 * and its rules hold here: every call enqueues one kernel, allocates and
 * synchronises nothing and can be captured; arrays of requests and tokens are
 * DEVICE memory, 4-byte aligned, and are read on the device; what is out of
 * range is left out and recorded in the handle's status (SFAR_KV_BAD_*).
 * Calls on one handle must not overlap on the GPU (sfar_latent_attention
 * keeps partial results in the handle, sfar_latent_append writes the cache);
 * a handle may be used from one host thread at a time.
 */
#ifndef SFAR_LATENT_H
#define SFAR_LATENT_H

#include "sfar_kv.h"
#include "sfar_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sfar_latent sfar_latent_t;

/*
 * sfar_latent_create: a handle on caller-owned caches (HOST array of R DEVICE
 * pointers, 16-byte aligned, no two overlapping).  1 <= R <= 16; latent_dim
 * 256 or 512; rope_dim 32 or 64; page_tokens 16, 32, 64 or 128;
 * 1 <= q_heads <= 65535; pages * page_tokens below 2^31.  The handle holds a
 * workspace for partial results, about 40 MB.  NULL on failure (reason:
 * sfar_last_error).  The caches' contents are not touched.
 */
sfar_latent_t *sfar_latent_create(int R, int q_heads, int latent_dim, int rope_dim, int page_tokens, size_t pages,
                                  void *const cache[]);
void sfar_latent_destroy(sfar_latent_t *h);

/* sfar_latent_plan: sfar_kv_plan for this cache's pages. */
sfar_status sfar_latent_plan(sfar_latent_t *h, const int32_t *lens, const int32_t *delta, int32_t *table, int32_t *ring,
                             const int32_t *state, int32_t *lens_out, int32_t *state_out, int32_t *starts, int32_t *slots,
                             int32_t *taken, size_t requests, size_t table_width, size_t tokens, sfar_stream_t s);

/*
 * sfar_latent_append: the step's tokens into the cache.  x[r]: bf16, row t at
 * t * token_stride (elements), latent_dim numbers l and rope_dim numbers k:
 *   c_i = l_i * weight_i / sqrt(mean of l^2 + eps),
 *   kr  = k turned by pos[t] as sfar_rope does (freq: [rope_dim / 2]
 *         binary32, layout, scale),
 * in binary32 (a row whose sum of squares passes its range has zeros for its
 * finite latents; squares below it are 0, so that with eps = 0 a row of numbers
 * below 2^-75 has infinities or NaN), rounded once to bf16, to slots[t].  A
 * token whose slot is -1 or whose position is negative is left out; the slots
 * of a call are distinct.  weight: [latent_dim] bf16.  Pointers 16-byte aligned (pos, freq, slots 4),
 * token_stride a multiple of 8, at least a row (with more than one token) and
 * below 2^39; tokens < 2^31; eps >= 0, scale finite.  Nothing overlaps the
 * caches.
 */
sfar_status sfar_latent_append(sfar_latent_t *h, const void *const x[], const void *weight, const int32_t *pos,
                               const float *freq, const int32_t *slots, size_t tokens, size_t token_stride, float eps,
                               int layout, float scale, sfar_stream_t s);

/*
 * sfar_latent_gather: cached rows in order.  Row starts[b] + i of out[r] (i
 * from 0, up to row starts[b + 1]) becomes token i of request b, the same
 * bits.  Rows of tokens that the request does not hold (i >= lens[b];
 * SFAR_KV_BAD_TOKENS) or that are on no page of the pool (SFAR_KV_BAD_PAGE),
 * and rows past starts[requests], are left as they are.  out[r]: bf16, rows of
 * latent_dim + rope_dim, token_stride a multiple of 8, at least a row, below
 * 2^39; pointers 16-byte aligned; out overlaps no other argument nor the
 * caches.  1 <= requests <= SFAR_KV_MAX_REQUESTS; tokens, table_width < 2^31.
 */
sfar_status sfar_latent_gather(sfar_latent_t *h, void *const out[], const int32_t *table, const int32_t *lens,
                               const int32_t *starts, size_t requests, size_t table_width, size_t tokens,
                               size_t token_stride, sfar_stream_t s);

/*
 * sfar_latent_attention: the absorbed form.  out = softmax(scale * q C^T) L,
 * with C the cached rows that a query row attends to and L their first
 * latent_dim numbers.  q[r]: bf16 [tokens][q_heads][latent_dim + rope_dim],
 * out[r]: bf16 [tokens][q_heads][latent_dim], with the given strides in
 * elements (multiples of 8, pointers 16-byte aligned).  Requests, positions
 * and rows are those of sfar_kv_attention without a window: the new tokens of
 * request b are the last of its lens[b] cached tokens, and the one at position
 * p attends to the cached tokens j <= p.  A row that has none, and a row past
 * starts[requests], is zeros.  Scores, maxima, the sum of the exponentials and
 * the products' sums are binary32, a weight is rounded to bf16 (8 bits,
 * relative to itself) before the second product.  A row's result does not
 * depend on what the other rows hold, nor on tokens it does not see.
 * Infinities (a score that passes binary32 is one): a token whose score is -inf
 * has weight 0; a row that attends to tokens and has no other scores, or a score
 * of +inf or NaN, is NaN (so is a row with an infinity or NaN among its queries,
 * whatever the signs), and so is one that attends to a latent that is not finite
 * (or whose sum of weights, up to 2^7.9 each, times latents passes binary32).
 * max_q: the most new tokens any request has in this call (a hint that picks
 * the kernel; a request that has more is still computed).  out overlaps no
 * other argument nor the caches, no row of it another, and the ranks' arrays
 * not one another.  1 <= requests <= SFAR_KV_MAX_REQUESTS; tokens,
 * table_width < 2^31; strides below 2^39; scale finite and at least 0.  (Two
 * tensors that lie in one another's memory without meeting are taken if they
 * are beside one another in rows of one length, as slices of one tensor's
 * last dimensions are, and refused otherwise; a strided out whose rows along
 * one dimension do not fit the other's stride is refused too.)  The kernel
 * counts in 32 bits: tokens * q_heads is below 2^29, and the product of
 * tokens * q_heads / 16 + requests (row tiles) and table_width * page_tokens
 * / 64 + 8 (tiles of a context) below 2^32.
 */
sfar_status sfar_latent_attention(sfar_latent_t *h, const void *const q[], void *const out[], const int32_t *table,
                                  const int32_t *lens, const int32_t *starts, size_t requests, size_t table_width,
                                  size_t tokens, size_t q_token_stride, size_t q_head_stride, size_t out_token_stride,
                                  size_t out_head_stride, size_t max_q, float scale, sfar_stream_t s);

/*
 * sfar_latent_prompt: the expanded form, over tensors in order (no cache is
 * read).  Request b's context is rows k_starts[b] .. k_starts[b + 1] of
 *   k[r]: [k_tokens][q_heads][head_dim], v[r]: [k_tokens][q_heads][head_dim],
 *   kr[r]: [k_tokens][rope_dim] (shared by the heads),
 * its new tokens, rows starts[b] .. starts[b + 1] of q[r]: [tokens][q_heads]
 * [head_dim + rope_dim] and out[r]: [tokens][q_heads][head_dim], are the last
 * of them: row starts[b] + i stands at position p = (rows of the context) -
 * (new tokens) + i and attends to context rows j <= p, with score
 * scale * (q[:head_dim] . k_j + q[head_dim:] . kr_j).  Softmax, numbers, rows
 * of nothing, infinite scores and rows past starts[requests] as in
 * sfar_latent_attention; a value that is not finite leaves the rows that attend
 * to it an infinity or NaN in its own element and nothing in the others.  A
 * scale below 2^-123 counts as about that.  All
 * bf16, strides in elements, multiples of 8 and below 2^39 (those of q, k, v
 * and kr above 0 for a dimension of more than one entry), pointers 16-byte
 * aligned; head_dim 64 or 128.  out overlaps no other argument, no row of it
 * another, and the ranks' arrays not one another.
 * 1 <= requests <= SFAR_KV_MAX_REQUESTS; tokens, k_tokens < 2^31 - 1024;
 * tokens / 128 + requests, times q_heads and R, below 2^31; scale finite and
 * at least 0.  Offsets out of order or beyond the tensors' rows:
 * SFAR_KV_BAD_TOKENS, and the request's rows are left as they are.
 */
sfar_status sfar_latent_prompt(sfar_latent_t *h, const void *const q[], const void *const k[], const void *const v[],
                               const void *const kr[], void *const out[], const int32_t *starts, const int32_t *k_starts,
                               size_t requests, size_t tokens, size_t k_tokens, size_t head_dim, size_t q_token_stride,
                               size_t q_head_stride, size_t k_token_stride, size_t k_head_stride, size_t v_token_stride,
                               size_t v_head_stride, size_t kr_token_stride, size_t out_token_stride,
                               size_t out_head_stride, size_t max_q, float scale, sfar_stream_t s);

/* As sfar_kv_status_get and sfar_kv_reset. */
sfar_status sfar_latent_status_get(sfar_latent_t *h, sfar_fault *info);
sfar_status sfar_latent_reset(sfar_latent_t *h, sfar_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* SFAR_LATENT_H */
