/*
 * sfar_rope.h -- rotary positions of queries and keys, for R simulated ranks
 * on one GB300, with any table of frequencies.
 */
#ifndef SFAR_ROPE_H
#define SFAR_ROPE_H

#include "sfar.h"

#ifdef __cplusplus
extern "C" {
#endif

/* which elements of the rotated part are a pair */
#define SFAR_ROPE_HALF 0        /* i and i + rot / 2   */
#define SFAR_ROPE_INTERLEAVED 1 /* 2 i and 2 i + 1     */

/*
 * sfar_rope: turns the pairs of every row by its position.  With
 * theta = pos[t] * freq[i] (the product of the two numbers, not rounded) and
 * (a, b) pair i of a row,
 *   a' = scale * (a cos theta - b sin theta),
 *   b' = scale * (b cos theta + a sin theta),
 * computed in binary32 from an angle that is within 2^-20 + 2^-46 |theta|
 * radians of theta, and rounded once to the handle's type.
 * q[r], q_out[r]: element (token t, head h, d) at t * token_stride +
 * h * head_stride + d (strides in elements), d below rot: the rotated part of
 * a head, wherever in it that lies; nothing beside it is read or written.
 * k, k_out: the same for k_heads heads (k_heads 0: both may be NULL).  An
 * output may be its input (same pointers and strides) and otherwise overlaps
 * no argument; queries and keys may lie beside one another in one tensor of
 * one token stride.  pos: [tokens], freq: [rot / 2] binary32, DEVICE memory.
 * A row whose position is negative is left as it is.
 * Types: the handle's (bf16 or fp32).  rot a multiple of 16, at most 1024;
 * pointers 16-byte aligned, strides multiples of 16 bytes and below 2^39,
 * tokens < 2^31, heads < 65536, (q_heads + k_heads) * rot < 2^22; scale
 * finite.  tokens = 0 does nothing.  One kernel on stream s; allocates and
 * synchronises nothing.
 */
sfar_status sfar_rope(sfar_t *h, const void *const q[], void *const q_out[], const void *const k[], void *const k_out[],
                      const int32_t *pos, const float *freq, size_t tokens, size_t q_heads, size_t k_heads, size_t rot,
                      size_t q_token_stride, size_t q_head_stride, size_t q_out_token_stride, size_t q_out_head_stride,
                      size_t k_token_stride, size_t k_head_stride, size_t k_out_token_stride, size_t k_out_head_stride,
                      int layout, float scale, sfar_stream_t s);

/* how frequencies are changed for contexts longer than the trained ones */
#define SFAR_ROPE_PLAIN 0      /* not at all                                                         */
#define SFAR_ROPE_LINEAR 1     /* all by 1 / factor                                                  */
#define SFAR_ROPE_WAVELENGTH 2 /* by the turns a pair makes in the trained context                   */
#define SFAR_ROPE_RAMP 3       /* by the pair's index, between the pairs that make `high` and `low` turns */

/*
 * sfar_rope_frequencies: freq[i] (HOST memory, rot / 2 numbers) and *scale,
 * computed in binary64 and rounded once.  With f = base^(-2 i / rot):
 *   PLAIN       f;                                             scale 1
 *   LINEAR      f / factor;                                    scale 1
 *   WAVELENGTH  n = trained * f / (2 pi): f if n > high, f / factor if
 *               n < low, else (1 - s) f / factor + s f with
 *               s = (n - low) / (high - low);                  scale 1
 *   RAMP        d(n) = rot ln(trained / (2 pi n)) / (2 ln base),
 *               from = max(floor(d(high)), 0), to = min(ceil(d(low)), rot - 1),
 *               s = clamp((i - from) / max(to - from, 0.001), 0, 1):
 *               s f / factor + (1 - s) f;                      scale 0.1 ln(factor) + 1
 * base > 1, factor >= 1, 0 < low < high, trained > 0 (the last three count for
 * WAVELENGTH and RAMP only); rot even.
 */
sfar_status sfar_rope_frequencies(float *freq, float *scale, size_t rot, double base, int scaling, double factor, double trained,
                                  double low, double high);

#ifdef __cplusplus
}
#endif

#endif /* SFAR_ROPE_H */
