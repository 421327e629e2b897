/*
 * blockint8_lora.h -- C ABI of low-rank adapters beside a shared projection: what
 * the requests of a batch, each with an adapter of its own or none, add to the
 * output of an 8-bit linear layer (blockint8.h, blockint8_fp8.h), for AMD
 * Instinct MI355X (gfx950, CDNA4).  Conventions as in blockint8.h.
 */
#ifndef BLOCKINT8_LORA_H_
#define BLOCKINT8_LORA_H_

#include "blockint8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Parts of a projection, and the largest rank of an adapter over all its parts. */
#define BI8_MAX_PARTS 4
#define BI8_MAX_RANKS 256
/*
 * y += s (x A^T) B^T, row by row with the row's adapter, in two launches.  The
 * projection may be several side by side (query, key and value; gate and up):
 * part p is the columns [n_p, n_(p+1)) of y and has R ranks of its own.  For row m
 * with adapter e = adapter[m]:
 *
 *   t[r]    = scales[e] * sum_k x[m, k] a[e, r, k]          r in [0, parts * R)
 *   y[m, n] = bf16( y[m, n] + sum_j t[p R + j] b[e, n, j] )   j in [0, R), n in
 *                                                              part p
 *
 * Sums are held in fp32; t enters the second product as the sum of two bf16
 * values, within 2^-16 of itself.  The order of the sums depends on the sizes
 * alone: a row's result does not depend on the other rows' values or adapters.
 *
 *   x        bf16 [M, ldx], the first K columns of each row
 *   a        bf16 [L, parts * R, K]      b  bf16 [L, N, R]
 *   scales   fp32 [L], or NULL: 1
 *   adapter  int32 [M] on the device; a row whose value lies outside [0, L) has no
 *            adapter and is left as it was
 *   y        bf16 [M, ldy], the first N columns of each row (updated in place)
 *   part_columns  int64 [parts] in HOST memory: the parts' widths, their sum N
 *   workspace     device memory, 16-byte aligned, of at least
 *            blockint8_lora_add_workspace_size(M, K, R, parts) bytes; contents
 *            undefined before and after.  Calls that share one must not overlap
 *            in time.
 *
 * Rows are taken 64 at a time, those of one adapter together: a batch whose rows
 * of one adapter lie next to each other reads the adapters least often.  Adapters
 * of smaller rank are padded with zeros (in a or in b, and no NaN or infinity in
 * the other).  An infinity in b may give NaN where the formula gives an infinity: it
 * meets both of t's values, of which one may be 0.  x and y may not overlap.
 *
 * Errors: NULL pointer (M > 0; scales may be) -> BI8_ERR_NULL; M < 0, N, K, L, R
 * or parts < 1, K, N, ldx or ldy > BI8_MAX_K, L > 2^24, parts > BI8_MAX_PARTS,
 * parts * R > BI8_MAX_RANKS, a width < 1 or another sum than N, ldx < K, ldy < N,
 * a workspace too small -> BI8_ERR_SHAPE; R % 8 != 0, a, b or workspace not
 * 16-byte, x or y not 2-byte, scales or adapter not 4-byte aligned ->
 * BI8_ERR_ALIGN; more rows than launches of 2^32 threads hold (by N, L
 * and parts) -> BI8_ERR_HIP, and nothing is launched.
 */
int32_t blockint8_lora_add(const uint16_t *x, int64_t ldx, const uint16_t *a, const uint16_t *b, const float *scales,
                           const int32_t *adapter, uint16_t *y, int64_t ldy, int64_t M, int64_t N, int64_t K, int32_t L,
                           int32_t R, int32_t parts, const int64_t *part_columns, void *workspace,
                           int64_t workspace_bytes, void *stream);

/* Enough for any batch of up to M rows: it does not fall as M grows.  0 for sizes that
 * blockint8_lora_add rejects, and for M = 0. */
int64_t blockint8_lora_add_workspace_size(int64_t M, int64_t K, int32_t R, int32_t parts);

#ifdef __cplusplus
}
#endif

#endif /* BLOCKINT8_LORA_H_ */
