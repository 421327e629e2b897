/*
 * blockint8_route.h -- C ABI of the router of a mixture of experts with scores,
 * a bias for balance and groups of experts, and of the MoE layer that takes its
 * result, for AMD Instinct MI355X (gfx950, CDNA4).  Beside blockint8_moe_route
 * (blockint8.h), whose outputs it shares.  Conventions as in blockint8.h.
 */
#ifndef BLOCKINT8_ROUTE_H_
#define BLOCKINT8_ROUTE_H_

#include "blockint8.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { BI8_SCORE_SOFTMAX = 0, BI8_SCORE_SIGMOID = 1 };

/* Most tokens of a call: its launches are of fewer than 2^32 threads. */
#define BI8_MAX_ROUTE_TOKENS ((1 << 28) - 64)

/*
 * Router and dispatch order: one launch for a few tokens, else two (three for
 * more than 2^14).  For each token t with logits l:
 *
 *   score   p[e] = exp(l[e] - max l) / sum exp(l - max l)   (softmax)
 *           p[e] = 1 / (1 + exp(-l[e]))                     (sigmoid)
 *   choice  c[e] = p[e] + bias[e]; without a bias the experts are ordered by
 *           their logits, which order them as their scores do
 *   groups  of E / groups consecutive experts.  A group's value is its largest
 *           c (group_top = 1) or the sum of its two largest (2; of one where it
 *           has one; without a bias, of p); the topk_groups groups of the
 *           largest values are kept, of equal ones the lower
 *   ids     the k experts of the kept groups with the largest c, in that order;
 *           of equal ones the lower
 *   weight  p[id] (without the bias), divided by the sum of the k with
 *           `renormalize` (0 where that sum is 0), times `scale`
 *
 * Scores that decide an order (with a bias, or sums of two) and those of the
 * chosen experts are held in binary64, so the order is that of the definition;
 * the weights are rounded once.  A logit that is NaN or -infinity has score 0
 * (a row of them: all weights 0) and, without a bias, stands behind all others;
 * +infinity counts as the largest finite value.  A bias or a choice that is NaN
 * counts as -infinity: a bias of -infinity switches an expert off, and one that
 * is off is taken only where the kept groups hold fewer than k others.
 *
 *   logits        [T, ldl], the first E columns of each row: fp32, or bf16 with
 *                 `logits_bf16`
 *   bias          fp32 [E] or NULL
 *   topk_ids, topk_weights, sorted_token, expert_offsets, row_of: as
 *                 blockint8_moe_route
 *   workspace     device memory, 16-byte aligned, of at least
 *                 blockint8_moe_route_grouped_workspace_size(T, E) bytes;
 *                 contents undefined before and after.  Calls that share one
 *                 must not overlap in time.  NULL where that size is 0.
 *
 * Limits: 1 <= E <= 1024, 1 <= k <= min(E, 32), T <= BI8_MAX_ROUTE_TOKENS, T * k <
 * 2^31, groups a divisor of E of at most 64, 1 <= topk_groups <= groups, k experts
 * at least in the kept groups.  T == 0 writes expert_offsets (all zero).
 *
 * Errors: NULL pointer -> BI8_ERR_NULL; a limit broken, ldl < E, an unknown
 * score, group_top not 1 or 2, a scale that is not finite, a workspace too small
 * -> BI8_ERR_SHAPE; a pointer not aligned to its type, workspace not to 16
 * bytes -> BI8_ERR_ALIGN.
 */
int32_t blockint8_moe_route_grouped(const void *logits, int32_t logits_bf16, int64_t ldl, const float *bias, int64_t T,
                                    int32_t E, int32_t k, int32_t score, int32_t groups, int32_t topk_groups,
                                    int32_t group_top, int32_t renormalize, double scale, int32_t *topk_ids,
                                    float *topk_weights, int32_t *sorted_token, int32_t *expert_offsets,
                                    int32_t *row_of, void *workspace, int64_t workspace_bytes, void *stream);

/* Enough for any batch of up to T tokens: it does not fall as T grows.  0 for few tokens
 * and for sizes that blockint8_moe_route_grouped rejects. */
int64_t blockint8_moe_route_grouped_workspace_size(int64_t T, int32_t E);

/*
 * blockint8_moe_layer_fp8_variant (blockint8_fp8.h) with the routing given: its
 * launches but the router's two, on what blockint8_moe_route or
 * blockint8_moe_route_grouped wrote.  The same bits as
 * blockint8_moe_layer_fp8_variant on the same routing.
 *
 *   topk_weights fp32 [T, k], sorted_token int32 [T * k], expert_offsets int32
 *   [E + 1], row_of int32 [T, k], on the device: as those two write them
 *   (offsets are clamped to [0, T * k]; a token outside [0, T) reads as zeros, a
 *   row outside [0, T * k) adds nothing)
 *   workspace: of blockint8_moe_layer_fp8_routed_workspace_size bytes
 *
 * k <= min(E, 32); other limits and errors as blockint8_moe_layer_fp8_variant.
 */
int32_t blockint8_moe_layer_fp8_routed(int32_t variant, const uint16_t *x, int64_t ldx, const float *topk_weights,
                                       const int32_t *sorted_token, const int32_t *expert_offsets,
                                       const int32_t *row_of, const uint8_t *w13, const float *ws13, const uint8_t *w2,
                                       const float *ws2, uint16_t *out, int64_t T, int64_t H, int64_t I, int32_t E,
                                       int32_t k, int32_t block_n, int32_t block_k, void *workspace,
                                       int64_t workspace_bytes, void *stream);

/* 0 for sizes that blockint8_moe_layer_fp8_routed rejects, and for T = 0.  It falls where
 * the products take another kernel: a workspace for several sizes is of the largest. */
int64_t blockint8_moe_layer_fp8_routed_workspace_size(int64_t T, int64_t H, int64_t I, int32_t E, int32_t k);

#ifdef __cplusplus
}
#endif

#endif /* BLOCKINT8_ROUTE_H_ */
