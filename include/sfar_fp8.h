/*
 * sfar_fp8.h -- the row-parallel projection of several tokens with weights in
 * 8-bit floating point (e4m3: 4 exponent bits of bias 7, 3 mantissa bits,
 * largest finite value 448, no infinities) and a scale for each block of 128:
 * the producer of the AllReduce when a tensor-parallel layer runs a batch.
 *
 *   y[r][i][j] = sum over blocks b of  sx[r][b][i] * sw[r][j / 128][b]
 *                * (sum over k in block b of x8[r][i][k] * w8[r][j][k])
 *
 * for the R simulated ranks of a handle, blocks of 128 consecutive k.  The
 * AllReduce of y then gives every rank the layer's output.
 */
#ifndef SFAR_FP8_H
#define SFAR_FP8_H

#include "sfar.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SFAR_FP8_BLOCK 128 /* elements of k (and rows of w8) that share a scale */

/*
 * sfar_quantize_fp8: x[r] (m rows of k bf16, row stride ldx elements) into
 *   x8[r]: m rows of k e4m3 (row stride ldx8 bytes) and
 *   sx[r]: ceil(k / 128) x m binary32, sx[r][b * m + i] the scale of block b
 *          of row i.
 * A scale is 2^e with the least e >= -100 such that the block's largest
 * magnitude is at most 448 * 2^e (2^-100 for a block of zeros); the stored
 * value is x / scale (exact) rounded to the nearest e4m3, ties to even.  A
 * power of two costs a floating format no precision and makes the quantised
 * values independent of how they are computed.  Infinities and NaN do not
 * count for the scale and are stored as NaN.
 * HOST arrays of R DEVICE pointers; x 2-byte, sx 4-byte aligned; the outputs
 * overlap nothing.  bf16 handles only.  m below 2^31, k up to 2^26 - 1024.  One kernel on stream s, capturable;
 * SFAR_ERR_INVALID for a bad argument, SFAR_ERR_CUDA if the launch fails.
 */
sfar_status sfar_quantize_fp8(sfar_t *h, const void *const x[], void *const x8[], float *const sx[], size_t m,
                              size_t k, size_t ldx, size_t ldx8, sfar_stream_t s);

/*
 * sfar_rowpar_gemm_fp8: the product above.
 *   x8[r]: m rows of k e4m3, row stride ldx8 bytes, 16-byte aligned, ldx8 a
 *          multiple of 16;
 *   sx[r]: ceil(k / 128) x m binary32 (as sfar_quantize_fp8 writes);
 *   w8[r]: hidden rows of k e4m3 (row j = the weights of output j), row
 *          stride ldw bytes, 16-byte aligned, ldw a multiple of 16;
 *   sw[r]: ceil(hidden / 128) x ceil(k / 128) binary32;
 *   y[r]:  m x hidden bf16, contiguous (ready for sfar_allreduce when 16-byte
 *          aligned), 2-byte aligned, overlapping nothing.
 * Products are exact; sums within a block and over the blocks are held in
 * binary32, in an order that depends on the sizes alone; one rounding to
 * bf16 (nearest even).  m, k, hidden from 1 to 2^31 - 1 (k need not be a
 * multiple of 128; the last block is then short).  One kernel on stream s,
 * capturable.  SFAR_ERR_INVALID for a bad argument (nothing enqueued),
 * SFAR_ERR_UNSUPPORTED if the driver offers no tensor-map encoder,
 * SFAR_ERR_CUDA if the launch fails.  Every wait on the device is bounded by
 * the handle's timeout and recorded in its status (where = SFAR_WAIT_COPY).
 */
sfar_status sfar_rowpar_gemm_fp8(sfar_t *h, const void *const x8[], const float *const sx[], const void *const w8[],
                                 const float *const sw[], void *const y[], size_t m, size_t k, size_t hidden,
                                 size_t ldx8, size_t ldw, sfar_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* SFAR_FP8_H */
