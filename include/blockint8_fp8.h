/*
 * blockint8_fp8.h -- C ABI of the e4m3 form of the block-wise 8-bit linear
 * layer for AMD Instinct MI355X (gfx950, CDNA4).
 *
 * The same layer as blockint8.h with OCP e4m3 codes in the place of int8:
 * 4 exponent bits, 3 mantissa bits, largest value 448, subnormals down to
 * 2^-9, no infinities, codes 0x7F and 0xFF NaN.  One byte a value, the layout
 * of torch.float8_e4m3fn.  Scales, blocks, layouts, statuses and the
 * conventions on pointers, streams, checks and errors are those of
 * blockint8.h:
 *
 *   - device pointers on the current HIP device, row-major and dense unless a
 *     leading dimension is given; bf16 values as uint16_t bits;
 *   - work is enqueued on `stream`, nothing is synchronised, no device memory
 *     is allocated and no state is kept but the thread's error message;
 *   - every argument is checked on the host; a failed check enqueues nothing;
 *   - blocks are [128, 128] (BI8_ERR_BLOCK otherwise); empty inputs are no-ops.
 *
 * Encoding of a group of values:  amax = max |x|,  s = amax / 448 (binary32),
 * code = rne(x / s) with x / s the correctly rounded binary32 quotient, all
 * codes zero when s == 0.  A group that holds a NaN has scale NaN, one that
 * holds an infinity has scale infinity; their codes are unspecified and
 * every product with them is NaN.
 */
#ifndef BLOCKINT8_FP8_H_
#define BLOCKINT8_FP8_H_

#include "blockint8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Dynamic activation quantisation, as blockint8_quant_act with e4m3 codes.
 *
 *   x   bf16 [M, ldx], the first K columns of each row (any ldx >= K, x 2-byte
 *       aligned)
 *   xq  e4m3 [M, K]                   (output)
 *   xs  fp32 [M, ceil(K / 128)]       (output)
 *
 * Errors: as blockint8_quant_act, with block_k 128 only.
 */
int32_t blockint8_quant_act_fp8(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, int32_t block_k, uint8_t *xq,
                                float *xs, void *stream);

/*
 * blockint8_quant_act_fp8 of the rows x[rows[0]], ..., x[rows[R - 1]], as
 * blockint8_quant_act_gather: x [T, ldx], rows int32 [R] on the device; an
 * index outside [0, T) quantises a row of zeros.
 */
int32_t blockint8_quant_act_gather_fp8(const uint16_t *x, int64_t T, int64_t ldx, const int32_t *rows, int64_t R,
                                       int64_t K, int32_t block_k, uint8_t *xq, float *xs, void *stream);

/*
 * h = [gate | up] bf16 [R, 2 I] -> a = bf16(silu(gate) up) quantised in groups
 * of 128 columns, as blockint8_silu_mul_quant with e4m3 codes:
 *   aq  e4m3 [R, I]   as  fp32 [R, ceil(I / 128)]   a  bf16 [R, I] or NULL
 * I % 16 == 0; h, aq and a 16-byte aligned.  Errors: as
 * blockint8_silu_mul_quant.
 */
int32_t blockint8_silu_mul_quant_fp8(const uint16_t *h, int64_t R, int64_t I, int32_t block_k, uint8_t *aq, float *as,
                                     uint16_t *a, void *stream);

/*
 * Offline block quantisation of a bf16 weight, one scale per 128 x 128 block:
 *   w   bf16 [N, ldw] (any ldw >= K, 2-byte aligned)
 *   wq  e4m3 [N, K] (16-byte aligned)   ws  fp32 [ceil(N / 128), ceil(K / 128)]
 * Any K from 1; N <= 65535 * 128.  Errors: as blockint8_quant_weight, without
 * its rules on K, ldw and the alignment of w (2 bytes here).
 */
int32_t blockint8_quant_weight_fp8(const uint16_t *w, int64_t N, int64_t K, int64_t ldw, int32_t block_n,
                                   int32_t block_k, uint8_t *wq, float *ws, void *stream);

/*
 * Block-scaled e4m3 GEMM, y = x . W^T:
 *
 *   xq    e4m3 [M, K]                       xs  fp32 [M, ceil(K / 128)]
 *   w     e4m3 [N, K]                       ws  fp32 [ceil(N / 128), ceil(K / 128)]
 *   bias  bf16 [N] or NULL
 *   y     bf16 [M, N]                       (output)
 *
 *   y[m, n] = bf16_rne( sum_g (sum_{k in g} xq[m, k] w[n, k])
 *                             (xs[m, g] ws[n / 128, g])  (+ bias[n]) )
 * The sums are held in fp32 (in an order that is unspecified, and the same
 * from call to call), with one step in the tiled kernels that is the matrix
 * core's own: it adds the products of eight consecutive codes aligned to the
 * largest of them and cuts each off 2^-13 below that one's leading bit.  The
 * streaming kernel (BI8_GEMM_SKINNY) and BI8_GEMM_TILE_256X128_F16 multiply the
 * codes as f16 values and do not.
 *
 *   workspace        device memory, 16-byte aligned, or NULL; its contents need
 *                    no initialisation and are undefined on return.  With at
 *                    least blockint8_gemm_fp8_workspace_size(M, N, K) bytes,
 *                    problems of few tiles split K between workgroups; with
 *                    less (or NULL) they do not.  Calls that share a
 *                    workspace must not overlap in time.
 *   workspace_bytes  its size
 *
 * Any M, N and K (K <= BI8_MAX_K); with K % 16 != 0 rows start at any byte and
 * a slower kernel runs.  Products of 2^23 tiles or more are not launched (the
 * bound that blockint8.h gives beside BI8_MAX_K; the quantisers and the norm have
 * none).  Errors: as blockint8_gemm_ws, blocks [128, 128] only.
 */
int32_t blockint8_gemm_fp8(const uint8_t *xq, const float *xs, const uint8_t *w, const float *ws, const uint16_t *bias,
                           uint16_t *y, int64_t M, int64_t N, int64_t K, int32_t block_n, int32_t block_k,
                           void *workspace, int64_t workspace_bytes, void *stream);

/* Workspace bytes that blockint8_gemm_fp8 uses for this problem (0: none, and
 * for sizes that it rejects). */
int64_t blockint8_gemm_fp8_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * The linear layer in one call: blockint8_quant_act_fp8 of x into
 * (xq_workspace e4m3 [M, K], xs_workspace fp32 [M, ceil(K / 128)]), which hold
 * the quantised activations on return, then blockint8_gemm_fp8.  Two or three
 * launches; y equals the two calls' exactly.  Errors: as those two; NULL xq /
 * xs workspace -> BI8_ERR_NULL.
 */
int32_t blockint8_linear_fp8(const uint16_t *x, int64_t ldx, const uint8_t *w, const float *ws, const uint16_t *bias,
                             uint16_t *y, int64_t M, int64_t N, int64_t K, int32_t block_n, int32_t block_k,
                             uint8_t *xq_workspace, float *xs_workspace, void *workspace, int64_t workspace_bytes,
                             void *stream);

/*
 * Grouped block-scaled e4m3 GEMM over rows sorted by expert, as
 * blockint8_moe_gemm: rows [off[e], off[e + 1]) of xq [R, K] meet w[e].
 *
 *   expert_offsets  int32 [E + 1] on the device, off[0] = 0, off[E] = R,
 *                   non-decreasing (a precondition: the host cannot read it;
 *                   offsets are clamped to [0, R], so none addresses outside
 *                   the tensors)
 *   w  e4m3 [E, N, K]   ws  fp32 [E, ceil(N / 128), ceil(K / 128)]
 *   y  bf16 [R, N]
 *   workspace, workspace_bytes: as blockint8_gemm_fp8, of
 *                   blockint8_moe_gemm_fp8_workspace_size(R, N, K, E) bytes
 *
 * Segments may be empty or of any length.  K % 16 == 0.  Errors: as
 * blockint8_moe_gemm_ws.
 */
int32_t blockint8_moe_gemm_fp8(const uint8_t *xq, const float *xs, const int32_t *expert_offsets, const uint8_t *w,
                               const float *ws, uint16_t *y, int64_t R, int64_t N, int64_t K, int32_t E,
                               int32_t block_n, int32_t block_k, void *workspace, int64_t workspace_bytes,
                               void *stream);

int64_t blockint8_moe_gemm_fp8_workspace_size(int64_t R, int64_t N, int64_t K, int32_t E);

/*
 * The w13 grouped GEMM with the gating and its quantisation as the epilogue, as
 * blockint8_moe_gemm_silu_quant: one launch computes what
 * blockint8_moe_gemm_fp8 (into h, N = 2 I) followed by
 * blockint8_silu_mul_quant_fp8 computes, without writing h.  It runs the
 * 256 x 128 or the 256 x 256 kernel; with the same variant of the grouped GEMM
 * the two launches give the same bits, with another the products may differ in
 * the order of their sums.
 *
 *   w13   e4m3 [E, 2 I, K]: rows [0, I) gate, rows [I, 2 I) up
 *   ws13  fp32 [E, 2 I / 128, ceil(K / 128)]
 *   aq    e4m3 [R, I]   as  fp32 [R, I / 128]   (outputs)
 *
 * Errors: as blockint8_moe_gemm_silu_quant.
 */
int32_t blockint8_moe_gemm_silu_quant_fp8(const uint8_t *xq, const float *xs, const int32_t *expert_offsets,
                                          const uint8_t *w13, const float *ws13, uint8_t *aq, float *as, int64_t R,
                                          int64_t I, int64_t K, int32_t E, int32_t block_n, int32_t block_k,
                                          void *stream);

/*
 * The whole MoE layer in one call: blockint8_moe_route of the logits (two
 * launches), blockint8_quant_act_gather_fp8, the w13 GEMM with the gating, the w2
 * GEMM and blockint8_moe_combine.  The w13 GEMM is the variant that
 * blockint8_moe_layer_fp8_select tells: BI8_GEMM_SKINNY or
 * BI8_GEMM_TILE_256X128_F16, which hold its sums for the second quantiser, where
 * the weights' stream bounds the product; else blockint8_moe_gemm_fp8's own choice.
 * With 256 x 128 (F16 or not) or 256 x 256 tiles and I % 128 == 0 the gating is its
 * epilogue (blockint8_moe_gemm_silu_quant_fp8), else blockint8_silu_mul_quant_fp8.
 * That makes six launches, seven where the gating is one of its own, and one more
 * for each grouped GEMM that splits a partial round over K.  Those have their part
 * of the layer's workspace: out equals the separate calls' exactly where w13 is
 * that variant and each other blockint8_moe_gemm_fp8 gets a workspace of its size.
 *
 *   x       bf16 [T, ldx], the first H columns of each row (2-byte aligned)
 *   logits  fp32 [T, E]
 *   w13     e4m3 [E, 2 I, H]   ws13  fp32 [E, ceil(2 I / 128), ceil(H / 128)]
 *   w2      e4m3 [E, H, I]     ws2   fp32 [E, ceil(H / 128), ceil(I / 128)]
 *   out     bf16 [T, H]   (output, 16-byte aligned)
 *   workspace        device memory, 256-byte aligned, of at least
 *                    blockint8_moe_layer_fp8_workspace_size(T, H, I, E, k)
 *                    bytes; contents undefined before and after.  Calls that
 *                    share one must not overlap in time.
 *
 * Limits: 1 <= E <= 1024, 1 <= k <= min(E, 8), H and I multiples of 16,
 * T * k < 2^31.  Errors: NULL pointer (T > 0) -> BI8_ERR_NULL; a limit broken,
 * ldx < H or a workspace too small -> BI8_ERR_SHAPE; blocks other than [128,
 * 128] -> BI8_ERR_BLOCK; H % 16, I % 16 or a pointer's alignment ->
 * BI8_ERR_ALIGN.
 */
int32_t blockint8_moe_layer_fp8(const uint16_t *x, int64_t ldx, const float *logits, const uint8_t *w13,
                                const float *ws13, const uint8_t *w2, const float *ws2, uint16_t *out, int64_t T,
                                int64_t H, int64_t I, int32_t E, int32_t k, int32_t renormalize, int32_t block_n,
                                int32_t block_k, void *workspace, int64_t workspace_bytes, void *stream);

/* 0 for sizes that blockint8_moe_layer_fp8 rejects, and for T = 0.  It falls where the
 * products take another kernel: a workspace for several sizes is of the largest. */
int64_t blockint8_moe_layer_fp8_workspace_size(int64_t T, int64_t H, int64_t I, int32_t E, int32_t k);

/*
 * Kernel variants, as in blockint8.h: the *_select functions tell which kernel
 * blockint8_gemm_fp8 / blockint8_moe_gemm_fp8 choose for a size without a
 * workspace, the *_variant forms run a named one (which leaves the workspace
 * alone), with the same arguments, results and errors.  Every
 * variant runs every size with K % 16 == 0, dense and grouped; with K % 16 != 0
 * only BI8_GEMM_AUTO is accepted (BI8_ERR_ALIGN otherwise).  An unknown variant
 * is BI8_ERR_SHAPE.  The ids are those of blockint8.h and two more:
 *
 *   BI8_GEMM_TILE_128X128      128 weight rows x 128 activation rows
 *   BI8_GEMM_TILE_256X128_F16  256 x 128, the codes multiplied as f16 values:
 *                              every sum is held in binary32, without the matrix
 *                              core's cut (see blockint8_gemm_fp8), at half its
 *                              rate.  The GEMMs never choose it by themselves:
 *                              for results that are quantised again.
 *
 * blockint8_moe_layer_fp8_variant is blockint8_moe_layer_fp8 with BI8_GEMM_AUTO or
 * with BI8_GEMM_TILE_256X128_F16 for the w13 GEMM, whatever its size; another id is
 * BI8_ERR_SHAPE.  The workspace is the same.  blockint8_moe_layer_fp8_select: the
 * w13 GEMM's variant of blockint8_moe_layer_fp8 (BI8_GEMM_AUTO for sizes that it
 * rejects).
 */
enum { BI8_GEMM_TILE_128X128 = 5, BI8_GEMM_TILE_256X128_F16 = 8 };

int32_t blockint8_gemm_fp8_select(int64_t M, int64_t N, int64_t K);

int32_t blockint8_moe_gemm_fp8_select(int64_t R, int64_t N, int64_t K, int32_t E);

int32_t blockint8_gemm_fp8_variant(int32_t variant, const uint8_t *xq, const float *xs, const uint8_t *w,
                                   const float *ws, const uint16_t *bias, uint16_t *y, int64_t M, int64_t N, int64_t K,
                                   int32_t block_n, int32_t block_k, void *workspace, int64_t workspace_bytes,
                                   void *stream);

int32_t blockint8_moe_gemm_fp8_variant(int32_t variant, const uint8_t *xq, const float *xs,
                                       const int32_t *expert_offsets, const uint8_t *w, const float *ws, uint16_t *y,
                                       int64_t R, int64_t N, int64_t K, int32_t E, int32_t block_n, int32_t block_k,
                                       void *workspace, int64_t workspace_bytes, void *stream);

int32_t blockint8_moe_layer_fp8_select(int64_t T, int64_t H, int64_t I, int32_t E, int32_t k);

int32_t blockint8_moe_layer_fp8_variant(int32_t variant, const uint16_t *x, int64_t ldx, const float *logits,
                                        const uint8_t *w13, const float *ws13, const uint8_t *w2, const float *ws2,
                                        uint16_t *out, int64_t T, int64_t H, int64_t I, int32_t E, int32_t k,
                                        int32_t renormalize, int32_t block_n, int32_t block_k, void *workspace,
                                        int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BLOCKINT8_FP8_H_ */
