/*
 * blockint8_norm.h -- C ABI of the root-mean-square norm that feeds the 8-bit
 * linear layers of blockint8.h (int8 codes) and blockint8_fp8.h (e4m3 codes),
 * for AMD Instinct MI355X (gfx950, CDNA4).  Conventions as in blockint8.h.
 */
#ifndef BLOCKINT8_NORM_H_
#define BLOCKINT8_NORM_H_

#include "blockint8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Addition of the residual, RMS norm and dynamic quantisation in one launch.
 * For each row of H columns:
 *
 *   h    = bf16_rne(fl32(x + residual))        (h = x when residual is NULL)
 *   rstd = fl32(1 / sqrt(sum(h^2) / H + eps))  (the sum, the quotient and the
 *                                               root in binary64)
 *   y    = fl32(fl32(h * rstd) * weight)
 *   per group of 128 columns: amax = max |y|, s = amax / T (binary32),
 *   xq = clamp(rne(y / s), -T, T), 0 when s == 0, xs = s
 *
 * with T = 127 and integer codes (blockint8_rmsnorm_quant) or T = 448 and e4m3
 * codes (blockint8_rmsnorm_quant_fp8); y is quantised from binary32, without a
 * rounding to bf16 in between.  Codes and scales are exactly these values for
 * finite inputs.  A row that holds a NaN or an infinity gets a NaN scale in
 * every group where y is NaN; the codes there are unspecified.  With eps = 0 a
 * row of zeros is 0 / 0: NaN scales.
 *
 *   x         bf16 [M, ldx]                    any ldx >= H
 *   residual  bf16 [M, ldr] or NULL            any ldr >= H
 *   weight    bf16 [H]
 *   h         bf16 [M, ldh], ldh >= H          (output; with a residual only:
 *             required then, NULL otherwise).  May be x or residual
 *             itself (same address and leading dimension): the sum is then
 *             formed in place.  No other overlap of inputs and outputs.
 *   y         bf16 [M, H] or NULL              (output, y rounded once: what a
 *             router or another bf16 consumer reads)
 *   xq        int8 / e4m3 [M, H]               (output)
 *   xs        fp32 [M, ceil(H / 128)]          (output)
 *
 * ldr and ldh are ignored without a residual.
 *
 * Errors: NULL x / weight / xq / xs (M > 0), NULL h with a residual or an h
 * without one -> BI8_ERR_NULL; M < 0, H <= 0, H > BI8_MAX_K, a leading
 * dimension < H, eps negative, infinite or NaN -> BI8_ERR_SHAPE; block_k not
 * 128 -> BI8_ERR_BLOCK; x / residual / weight / h / y not 2-byte, xq not
 * 16-byte or xs not 4-byte aligned -> BI8_ERR_ALIGN.
 */
int32_t blockint8_rmsnorm_quant(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                const uint16_t *weight, double eps, int64_t M, int64_t H, int32_t block_k, uint16_t *h,
                                int64_t ldh, uint16_t *y, int8_t *xq, float *xs, void *stream);

int32_t blockint8_rmsnorm_quant_fp8(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                    const uint16_t *weight, double eps, int64_t M, int64_t H, int32_t block_k,
                                    uint16_t *h, int64_t ldh, uint16_t *y, uint8_t *xq, float *xs, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BLOCKINT8_NORM_H_ */
