/*
 * sfar_kv.h -- the paged key/value cache of a tensor-parallel decode layer,
 * held in 8-bit floating point (e4m3) with one scale for each page and head,
 * and the attention that reads it, for R simulated ranks on one GB300.
 *
 * Rank r holds kv_heads heads of keys and values and answers for q_heads
 * heads of queries (q_heads a multiple of kv_heads: query head i reads key
 * head i / (q_heads / kv_heads)).  The cache of a rank is a pool of pages of
 * page_tokens tokens; page p holds
 *   k_cache[r], v_cache[r]: [pages][kv_heads][page_tokens][head_dim] e4m3,
 *   k_scale[r], v_scale[r]: [pages][kv_heads] binary32,
 * and the value it stands for is e4m3 * scale.  All ranks share the block
 * tables: table[b][i] is the page of tokens [i * page_tokens, (i + 1) *
 * page_tokens) of request b, slot = page * page_tokens + offset names one
 * token.  One step of a model is
 *   sfar_kv_plan       once: pages for the new tokens, slots, offsets;
 *   sfar_kv_append     per layer: the new keys and values into the cache;
 *   sfar_kv_attention  per layer: the new tokens over their contexts.
 *
 * Every call enqueues one kernel on stream s, allocates and synchronises
 * nothing and can be captured in a CUDA graph.  Arrays of requests and tokens are DEVICE memory, 4-byte aligned;
 * lengths are read on the device, so a captured step replays with new ones.
 * Calls on one handle must not overlap on the GPU (sfar_kv_attention keeps
 * partial results in the handle); a handle may be used from one host thread
 * at a time.
 *
 * Page numbers, slots and lengths live on the device, so the kernels check
 * them: what is out of range is left out, never read or written, and
 * recorded in the handle's status (sfar_kv_status_get: SFAR_ERR_INVALID with
 * where = SFAR_KV_BAD_*, cta = the request or token it was seen at).
 */
#ifndef SFAR_KV_H
#define SFAR_KV_H

#include "sfar.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sfar_kv sfar_kv_t;

#define SFAR_KV_MAX_REQUESTS 8192

/* sfar_fault.where of a handle's device-side checks */
#define SFAR_KV_BAD_PAGE 32   /* a page number outside the pool                                */
#define SFAR_KV_BAD_LENGTH 33 /* a length below 0 or beyond the block table                    */
#define SFAR_KV_BAD_SLOT 34   /* a slot outside the pool                                       */
#define SFAR_KV_BAD_TOKENS 35 /* more new tokens than the call has rows, or offsets out of order */
#define SFAR_KV_BAD_RING 36   /* the ring's state: first page or count out of range            */

/*
 * sfar_kv_create: a handle on caller-owned caches (HOST arrays of R DEVICE
 * pointers; caches 16-byte, scales 4-byte aligned, no two overlapping).
 * 1 <= R <= 16; head_dim 64 or 128; page_tokens 16, 32, 64 or 128; q_heads a
 * multiple of kv_heads; pages * page_tokens and pages * kv_heads below 2^31.
 * The handle holds a workspace for partial results, about 41 MB at head_dim 128.  NULL on
 * failure (reason: sfar_last_error).  The caches' contents are not touched.
 */
sfar_kv_t *sfar_kv_create(int R, int q_heads, int kv_heads, int head_dim, int page_tokens, size_t pages,
                          void *const k_cache[], void *const v_cache[], float *const k_scale[],
                          float *const v_scale[]);
void sfar_kv_destroy(sfar_kv_t *kv);

/*
 * sfar_kv_plan: block tables, slot map and token offsets of a step, from the
 * requests' lengths.  With P = page_tokens, request b holds lens[b] tokens
 * and changes by delta[b]:
 *   delta[b] > 0   adds tokens; the pages it lacks, ceil((lens + delta) / P) -
 *                  ceil(lens / P), are taken from the ring of free pages, in
 *                  the order of the requests.  It is refused (taken[b] = 0,
 *                  its length stays, its slots are -1) when it does not fit
 *                  its row of the table, or when it needs pages and they,
 *                  with those of all requests before it that fit their rows,
 *                  are more than are free;
 *   delta[b] == 0  nothing;
 *   delta[b] < 0   drops its last -delta[b] tokens (all, if there are fewer)
 *                  and gives the pages it no longer needs back to the ring,
 *                  behind the pages that were free before the call.
 * ring: [pages] page numbers; state = {index of the first free page, number
 * of free pages}; the free pages are ring[(state[0] + i) mod pages].
 * Writes lens_out[b], taken[b], starts[0 .. requests] (the exclusive sums of
 * max(delta, 0): request b's new tokens are rows starts[b] .. starts[b + 1]
 * of the step's tensors, taken or not), slots[0 .. tokens) (-1 past the last
 * new token), the table entries of new pages, the ring entries of pages given
 * back, and state_out.  Pages given back beyond those that the state says are
 * held are dropped (SFAR_KV_BAD_RING); a page number outside the pool
 * (SFAR_KV_BAD_PAGE) becomes -1, in the ring when it is given back and in the
 * table when it is taken, and its tokens' slots are -1.  The rows of a request
 * that was refused mean nothing to sfar_kv_attention.  Other entries stay.
 * table: [requests][table_width].
 * lens_out may be lens and state_out may be state; nothing else overlaps.
 * 1 <= requests <= SFAR_KV_MAX_REQUESTS, 1 <= table_width, tokens < 2^31.
 */
sfar_status sfar_kv_plan(sfar_kv_t *kv, const int32_t *lens, const int32_t *delta, int32_t *table, int32_t *ring,
                         const int32_t *state, int32_t *lens_out, int32_t *state_out, int32_t *starts, int32_t *slots,
                         int32_t *taken, size_t requests, size_t table_width, size_t tokens, sfar_stream_t s);

/*
 * sfar_kv_append: the keys and values of the step's tokens into the cache.
 * k[r], v[r]: bf16, element (token t, head h, d) at t * token_stride + h *
 * head_stride + d (strides in elements, multiples of 8, below 2^40; pointers
 * 16-byte aligned).  Token t goes to slots[t]; -1 leaves it out.  Tokens of one page
 * must be neighbours in t with consecutive slots (as sfar_kv_plan gives
 * them), and the page's offsets before the first of them are held tokens.
 * For each page, head and cache, with amax the largest magnitude of the new
 * values: need = 2^e, e >= -100 least with amax <= 448 * 2^e; the scale
 * becomes need when the new tokens start the page, and otherwise the larger
 * of need and the present scale s.  If it grows, the held tokens are
 * rewritten: their e4m3 value times s / scale, rounded to the nearest e4m3
 * (exact between powers of two until a value leaves e4m3's normal range).
 * New values are stored as value / scale, rounded to the nearest e4m3, ties
 * to even.  Infinities and NaN do not count for amax and are stored as NaN.
 */
sfar_status sfar_kv_append(sfar_kv_t *kv, const void *const k[], const void *const v[], const int32_t *slots,
                           size_t tokens, size_t k_token_stride, size_t k_head_stride, size_t v_token_stride,
                           size_t v_head_stride, sfar_stream_t s);

/*
 * sfar_kv_attention: out = softmax(scale * q K^T) V for the step's tokens.
 * q[r], out[r]: bf16 [tokens][q_heads][head_dim] with the given strides in
 * elements (multiples of 8, pointers 16-byte aligned).  Request b's context
 * is its lens[b] cached tokens, its new tokens (rows starts[b] ..
 * starts[b + 1]) are the last of them: row starts[b] + i stands at position
 * p = lens[b] - (starts[b + 1] - starts[b]) + i and attends to the cached
 * tokens j <= p and, with window > 0, j > p - window.  A row that has none
 * (and a row past starts[requests]) is zeros.  The largest score and the sum
 * of the exponentials are held in binary32, as are the products' sums; a
 * weight (exponential times value scale) is rounded to 11 bits, and to a
 * multiple of 2^-32 of the row's largest where that is coarser.  A query's
 * elements are taken exactly down to 2^-29 of its row's largest (2^-9 by the
 * kernel for many rows, see max_q), smaller ones to within 2^-39 (2^-17) of
 * that.  The result does not depend on what the other rows or masked tokens
 * hold; a row with an infinity or NaN among its queries, or among what it
 * attends to (NaN, cached), is NaN there.  A page's scales may be zero, and negative.  A value scale of magnitude 2^-100
 * or less counts as zero (2^-100 is what sfar_kv_append gives to zeros); the
 * others of one request's context are at most 2^100 and within a factor of
 * 2^100 of one another: beyond it tokens with the smaller scales lose their
 * part of the sum of the exponentials.
 * max_q: the most new tokens any request has in this call (a hint that picks
 * the kernel; a request that has more is still computed).  out overlaps no
 * other argument, no row of it another, and the ranks' arrays not one another.
 * 1 <= requests <= SFAR_KV_MAX_REQUESTS; tokens, table_width < 2^31; strides
 * below 2^40; scale finite and at least 0.  The kernels count
 * in 32 bits: with G = q_heads / kv_heads, tokens * G is below 2^29 and the
 * product of tokens * G / n + requests (row tiles) and table_width *
 * page_tokens / m + 8 (tiles of a context) below 2^32, where n = 256, m = 128,
 * or n = 8, m = 64 if max_q * G is at most 32 or requests above 2048.
 */
sfar_status sfar_kv_attention(sfar_kv_t *kv, const void *const q[], void *const out[], const int32_t *table,
                              const int32_t *lens, const int32_t *starts, size_t requests, size_t table_width,
                              size_t tokens, size_t q_token_stride, size_t q_head_stride, size_t out_token_stride,
                              size_t out_head_stride, size_t max_q, float scale, size_t window, sfar_stream_t s);

/*
 * sfar_kv_status_get: SFAR_OK, or the first failure recorded on the device
 * (synchronise the calls' streams first).  It stays until sfar_kv_reset.
 * Calls go on computing after it, but after SFAR_ERR_TIMEOUT (a wait of an
 * attention call that ran out after a second: where = SFAR_WAIT_COPY) the
 * results of attention are undefined until sfar_kv_reset, which puts the
 * handle's workspace in order too, on stream s.
 */
sfar_status sfar_kv_status_get(sfar_kv_t *kv, sfar_fault *info);
sfar_status sfar_kv_reset(sfar_kv_t *kv, sfar_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* SFAR_KV_H */
