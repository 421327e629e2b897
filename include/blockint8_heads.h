/*
 * blockint8_heads.h -- C ABI of the norm and the rotation of query and key
 * heads, what reads the output of a query / key / value projection
 * (blockint8.h, blockint8_fp8.h), for AMD Instinct MI355X (gfx950, CDNA4).
 * Conventions as in blockint8.h.
 */
#ifndef BLOCKINT8_HEADS_H_
#define BLOCKINT8_HEADS_H_

#include "blockint8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head size, and the largest number of axes that positions have. */
#define BI8_MAX_HEAD_DIM 1024
#define BI8_MAX_AXES 4

/*
 * The root-mean-square norm of each query and key head and the rotation by its
 * token's position, in one launch.  For each token t and head x of D values:
 *
 *   u  = x / sqrt(mean(x^2) + eps) * weight      (u = x where weight is NULL)
 *   pair i in [0, rot / 2):  values i and i + rot / 2 of the head (2 i and
 *        2 i + 1 with `interleaved`), turned by the angle whose cosine c and
 *        sine s are table[p, i] and table[p, rot / 2 + i]:
 *            o1 = u1 c - u2 s,   o2 = u2 c + u1 s
 *        with p = positions[axis of i, t]
 *   values from rot on are u
 *
 * in binary32 (the sum of squares in binary64), rounded once to bf16.
 *
 *   q          bf16, token t's head h begins at q + t q_token + h q_head
 *              (elements; any strides), Hq heads
 *   k          the same with Hk heads; NULL with Hk = 0
 *   q_weight   bf16 [D] or NULL (no norm); k_weight the same for the key heads
 *   table      fp32 [P, rot]: cosines, then sines, of the rot / 2 pairs
 *   positions  int32, axis a of token t at positions[a * positions_axis + t].
 *              A token with a position outside [0, P) is left out: its outputs
 *              are not written (padding), and row 0 of the table is read for it.
 *   sections   int32 [axes] in HOST memory: axis 0 turns the first sections[0]
 *              pairs, axis 1 the next sections[1], ...; their sum is rot / 2.
 *              Text has one axis, {rot / 2}; images and video have three (time,
 *              height, width).
 *   q_out, k_out  bf16 with strides as q and k (outputs).  An output may be its
 *              input (same address and strides); no other overlap.
 *
 * Errors: NULL pointer (T > 0; k, k_out with Hk > 0) -> BI8_ERR_NULL; T < 0,
 * Hq < 1, Hk < 0 or more than 65536 heads, D odd, < 2 or > BI8_MAX_HEAD_DIM,
 * rot odd, < 2 or > D, P < 1, axes outside [1, BI8_MAX_AXES], a negative
 * section or another sum than rot / 2, a negative stride, eps negative,
 * infinite or NaN -> BI8_ERR_SHAPE; q, k, weights, outputs not 2-byte, table or
 * positions not 4-byte aligned -> BI8_ERR_ALIGN.
 */
int32_t blockint8_qk_norm_rope(const uint16_t *q, int64_t q_token, int64_t q_head, int32_t Hq, const uint16_t *k,
                               int64_t k_token, int64_t k_head, int32_t Hk, const uint16_t *q_weight,
                               const uint16_t *k_weight, double eps, const float *table, int64_t P,
                               const int32_t *positions, int64_t positions_axis, int32_t axes,
                               const int32_t *sections, int32_t interleaved, int64_t T, int32_t D, int32_t rot,
                               uint16_t *q_out, int64_t q_out_token, int64_t q_out_head, uint16_t *k_out,
                               int64_t k_out_token, int64_t k_out_head, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BLOCKINT8_HEADS_H_ */
