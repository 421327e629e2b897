// C ABI of the operators beside the 8-bit products: argument checks on the host,
// then the launches on the caller's stream.  See include/blockint8_heads.h,
// include/blockint8_route.h and include/blockint8_lora.h for the contracts.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/blockint8_heads.h"
#include "../../include/blockint8_lora.h"
#include "../../include/blockint8_route.h"
#include "checks.hpp"
#include "internal.hpp"

namespace {

using namespace bi8::checks;
using bi8::fail_status;

// T tokens of H heads of D values, apart by these strides: whether no two share
// an element.
bool heads_apart(int64_t T, int64_t token, int64_t H, int64_t head, int64_t D) {
    if (T <= 1) return H <= 1 || head >= D;
    if (H <= 1) return token >= D;
    return (head >= D && token >= (H - 1) * head + D) || (token >= D && head >= (T - 1) * token + D);
}

int32_t check_strides(const char *fn, const char *what, int64_t token, int64_t head) {
    constexpr int64_t kMost = 1ll << 40;
    if (token < 0 || head < 0 || token > kMost || head > kMost)
        return fail_status(BI8_ERR_SHAPE, "%s: strides (%lld, %lld) of %s out of range", fn, (long long)token,
                           (long long)head, what);
    return BI8_OK;
}

int32_t check_heads_output(const char *fn, const char *what, int64_t T, int64_t token, int64_t H, int64_t head,
                           int64_t D) {
    BI8_TRY(check_strides(fn, what, token, head));
    if (!heads_apart(T, token, H, head, D))
        return fail_status(BI8_ERR_SHAPE, "%s: heads of %s overlap (strides %lld, %lld)", fn, what, (long long)token,
                           (long long)head);
    return BI8_OK;
}

}  // namespace

extern "C" {

int32_t blockint8_qk_norm_rope(const uint16_t *q, int64_t q_token, int64_t q_head, int32_t Hq, const uint16_t *k,
                               int64_t k_token, int64_t k_head, int32_t Hk, const uint16_t *q_weight,
                               const uint16_t *k_weight, double eps, const float *table, int64_t P,
                               const int32_t *positions, int64_t positions_axis, int32_t axes,
                               const int32_t *sections, int32_t interleaved, int64_t T, int32_t D, int32_t rot,
                               uint16_t *q_out, int64_t q_out_token, int64_t q_out_head, uint16_t *k_out,
                               int64_t k_out_token, int64_t k_out_head, void *stream) {
    static const char fn[] = "blockint8_qk_norm_rope";
    static_assert(BI8_MAX_AXES == bi8::kMaxAxes, "axes");
    BI8_TRY(check_rows(fn, "T", T));
    if (Hq < 1 || Hk < 0 || Hq > 65536 || Hk > 65536)
        return fail_status(BI8_ERR_SHAPE, "%s: %d query and %d key heads out of range", fn, Hq, Hk);
    if (D < 2 || D > BI8_MAX_HEAD_DIM || D % 2 != 0)
        return fail_status(BI8_ERR_SHAPE, "%s: D = %d must be even, in [2, %d]", fn, D, BI8_MAX_HEAD_DIM);
    if (rot < 2 || rot > D || rot % 2 != 0)
        return fail_status(BI8_ERR_SHAPE, "%s: rot = %d must be even, in [2, D]", fn, rot);
    if (P < 1 || P > kMaxRows) return fail_status(BI8_ERR_SHAPE, "%s: P = %lld out of range", fn, (long long)P);
    if (axes < 1 || axes > BI8_MAX_AXES || positions_axis < 0)
        return fail_status(BI8_ERR_SHAPE, "%s: axes = %d out of range [1, %d], or their stride", fn, axes, BI8_MAX_AXES);
    if (!(eps >= 0.0) || !std::isfinite(eps))
        return fail_status(BI8_ERR_SHAPE, "%s: eps = %g must be finite and not negative", fn, eps);
    BI8_TRY(check_strides(fn, "q", q_token, q_head));
    BI8_TRY(check_heads_output(fn, "q_out", T, q_out_token, Hq, q_out_head, D));
    if (Hk > 0) {
        BI8_TRY(check_strides(fn, "k", k_token, k_head));
        BI8_TRY(check_heads_output(fn, "k_out", T, k_out_token, Hk, k_out_head, D));
    }
    if (!sections) return null_pointer(fn);
    bi8::HeadsArgs p{};
    int64_t pairs = 0;
    for (int32_t a = 0; a < BI8_MAX_AXES; ++a) {
        p.first[a] = a < axes ? static_cast<int32_t>(pairs) : INT_MAX;
        if (a >= axes) continue;
        if (sections[a] < 0 || sections[a] > rot)
            return fail_status(BI8_ERR_SHAPE, "%s: section %d = %d out of range", fn, a, sections[a]);
        pairs += sections[a];
    }
    if (2 * pairs != rot)
        return fail_status(BI8_ERR_SHAPE, "%s: the sections hold %lld pairs, not %d", fn, (long long)pairs, rot / 2);
    if (T == 0) return done(fn);
    if (!q || !q_out || !table || !positions || (Hk > 0 && (!k || !k_out))) return null_pointer(fn);
    BI8_TRY(check_align(fn, "q", q, 2));
    BI8_TRY(check_align(fn, "q_out", q_out, 2));
    BI8_TRY(check_align(fn, "q_weight", q_weight, 2));
    BI8_TRY(check_align(fn, "k_weight", k_weight, 2));
    BI8_TRY(check_align(fn, "table", table, 4));
    BI8_TRY(check_align(fn, "positions", positions, 4));
    p.q = q, p.q_weight = q_weight, p.q_out = q_out;
    p.q_token = q_token, p.q_head = q_head, p.q_out_token = q_out_token, p.q_out_head = q_out_head;
    if (Hk > 0) {
        BI8_TRY(check_align(fn, "k", k, 2));
        BI8_TRY(check_align(fn, "k_out", k_out, 2));
        p.k = k, p.k_weight = k_weight, p.k_out = k_out;
        p.k_token = k_token, p.k_head = k_head, p.k_out_token = k_out_token, p.k_out_head = k_out_head;
    }
    p.table = table, p.P = P, p.positions = positions, p.positions_axis = positions_axis, p.axes = axes;
    p.eps = eps, p.T = T, p.Hq = Hq, p.Hk = Hk, p.D = D, p.rot = rot, p.interleaved = interleaved != 0;
    return bi8::call_status(fn, bi8::launch_qk_norm_rope(p, static_cast<hipStream_t>(stream)));
}

int64_t blockint8_moe_route_grouped_workspace_size(int64_t T, int32_t E) {
    if (T <= 0 || T > BI8_MAX_ROUTE_TOKENS || E < 1 || E > 1024) return 0;
    return bi8::route_grouped_workspace_bytes(T, E);
}

int32_t blockint8_moe_route_grouped(const void *logits, int32_t logits_bf16, int64_t ldl, const float *bias, int64_t T,
                                    int32_t E, int32_t k, int32_t score, int32_t groups, int32_t topk_groups,
                                    int32_t group_top, int32_t renormalize, double scale, int32_t *topk_ids,
                                    float *topk_weights, int32_t *sorted_token, int32_t *expert_offsets,
                                    int32_t *row_of, void *workspace, int64_t workspace_bytes, void *stream) {
    static const char fn[] = "blockint8_moe_route_grouped";
    if (E < 1 || E > 1024) return fail_status(BI8_ERR_SHAPE, "%s: E = %d out of range [1, 1024]", fn, E);
    if (k < 1 || k > 32 || k > E) return fail_status(BI8_ERR_SHAPE, "%s: k = %d out of range [1, min(E, 32)]", fn, k);
    if (T < 0 || T > kMaxRows / k || T > BI8_MAX_ROUTE_TOKENS)
        return fail_status(BI8_ERR_SHAPE, "%s: T = %lld out of range", fn, (long long)T);
    if (score != BI8_SCORE_SOFTMAX && score != BI8_SCORE_SIGMOID)
        return fail_status(BI8_ERR_SHAPE, "%s: unknown score %d", fn, score);
    if (groups < 1 || groups > 64 || E % groups != 0)
        return fail_status(BI8_ERR_SHAPE, "%s: groups = %d must divide E = %d, in [1, 64]", fn, groups, E);
    if (topk_groups < 1 || topk_groups > groups || topk_groups * (E / groups) < k)
        return fail_status(BI8_ERR_SHAPE, "%s: topk_groups = %d must be in [1, %d] and hold k = %d experts", fn,
                           topk_groups, groups, k);
    if (group_top != 1 && group_top != 2)
        return fail_status(BI8_ERR_SHAPE, "%s: group_top = %d must be 1 or 2", fn, group_top);
    if (!std::isfinite(scale)) return fail_status(BI8_ERR_SHAPE, "%s: scale = %g must be finite", fn, scale);
    BI8_TRY(check_pitch(fn, "ldl", ldl, E));
    BI8_TRY(check_workspace(fn, workspace, workspace_bytes));
    if (!expert_offsets || (T > 0 && (!logits || !topk_ids || !topk_weights || !sorted_token || !row_of)))
        return null_pointer(fn);
    BI8_TRY(check_align(fn, "logits", logits, logits_bf16 ? 2 : 4));
    BI8_TRY(check_align(fn, "bias", bias, 4));
    BI8_TRY(check_align(fn, "topk_ids", topk_ids, 4));
    BI8_TRY(check_align(fn, "topk_weights", topk_weights, 4));
    BI8_TRY(check_align(fn, "sorted_token", sorted_token, 4));
    BI8_TRY(check_align(fn, "expert_offsets", expert_offsets, 4));
    BI8_TRY(check_align(fn, "row_of", row_of, 4));
    const int64_t need = T > 0 ? bi8::route_grouped_workspace_need(T, E) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail_status(BI8_ERR_SHAPE, "%s: workspace_bytes = %lld < %lld", fn,
                           (long long)(workspace ? workspace_bytes : 0), (long long)need);
    bi8::RouteArgs p{};
    p.logits = logits, p.bf16 = logits_bf16 != 0, p.ldl = ldl, p.bias = bias, p.T = T, p.E = E, p.k = k;
    p.score = score, p.groups = groups, p.topk_groups = topk_groups, p.group_top = group_top;
    p.renormalize = renormalize != 0, p.scale = scale;
    p.ids = topk_ids, p.weights = topk_weights, p.sorted_token = sorted_token, p.offsets = expert_offsets;
    p.row_of = row_of;
    return bi8::call_status(fn, bi8::launch_moe_route_grouped(p, workspace, static_cast<hipStream_t>(stream)));
}

int64_t blockint8_lora_add_workspace_size(int64_t M, int64_t K, int32_t R, int32_t parts) {
    if (M <= 0 || M > kMaxRows || K <= 0 || K > BI8_MAX_K || R < 8 || R % 8 != 0 || parts < 1 ||
        parts > BI8_MAX_PARTS || R > BI8_MAX_RANKS / parts)
        return 0;
    return bi8::lora_workspace_bytes(M, K, parts * R);
}

int32_t blockint8_lora_add(const uint16_t *x, int64_t ldx, const uint16_t *a, const uint16_t *b, const float *scales,
                           const int32_t *adapter, uint16_t *y, int64_t ldy, int64_t M, int64_t N, int64_t K, int32_t L,
                           int32_t R, int32_t parts, const int64_t *part_columns, void *workspace,
                           int64_t workspace_bytes, void *stream) {
    static const char fn[] = "blockint8_lora_add";
    static_assert(BI8_MAX_PARTS == bi8::kMaxParts, "parts");
    BI8_TRY(check_rows(fn, "M", M));
    if (N <= 0 || N > BI8_MAX_K)
        return fail_status(BI8_ERR_SHAPE, "%s: N = %lld out of range [1, 2^23]", fn, (long long)N);
    BI8_TRY(check_columns(fn, "K", K));
    if (L < 1 || L > 1 << 24) return fail_status(BI8_ERR_SHAPE, "%s: L = %d out of range [1, 2^24]", fn, L);
    if (parts < 1 || parts > BI8_MAX_PARTS)
        return fail_status(BI8_ERR_SHAPE, "%s: parts = %d out of range [1, %d]", fn, parts, BI8_MAX_PARTS);
    if (R < 1 || R > BI8_MAX_RANKS / parts)
        return fail_status(BI8_ERR_SHAPE, "%s: R = %d out of range [1, %d] for %d parts", fn, R, BI8_MAX_RANKS / parts,
                           parts);
    if (R % 8 != 0) return fail_status(BI8_ERR_ALIGN, "%s: R = %d must be a multiple of 8", fn, R);
    if (!part_columns) return null_pointer(fn);
    int64_t columns = 0;
    for (int32_t i = 0; i < parts; ++i) {
        if (part_columns[i] < 1 || part_columns[i] > N)
            return fail_status(BI8_ERR_SHAPE, "%s: part %d has %lld columns", fn, i, (long long)part_columns[i]);
        columns += part_columns[i];
    }
    if (columns != N)
        return fail_status(BI8_ERR_SHAPE, "%s: the parts have %lld columns, not %lld", fn, (long long)columns,
                           (long long)N);
    BI8_TRY(check_pitch(fn, "ldx", ldx, K));
    BI8_TRY(check_pitch(fn, "ldy", ldy, N));
    if (ldx > BI8_MAX_K || ldy > BI8_MAX_K)
        return fail_status(BI8_ERR_SHAPE, "%s: ldx = %lld or ldy = %lld above 2^23", fn, (long long)ldx, (long long)ldy);
    BI8_TRY(check_workspace(fn, workspace, workspace_bytes));
    if (M == 0) return done(fn);
    if (!x || !a || !b || !adapter || !y || !workspace) return null_pointer(fn);
    BI8_TRY(check_align(fn, "x", x, 2));
    BI8_TRY(check_align(fn, "a", a, 16));
    BI8_TRY(check_align(fn, "b", b, 16));
    BI8_TRY(check_align(fn, "scales", scales, 4));
    BI8_TRY(check_align(fn, "adapter", adapter, 4));
    BI8_TRY(check_align(fn, "y", y, 2));
    const int64_t need = bi8::lora_workspace_need(M, K, parts * R);
    if (workspace_bytes < need)
        return fail_status(BI8_ERR_SHAPE, "%s: workspace_bytes = %lld < %lld", fn, (long long)workspace_bytes,
                           (long long)need);
    bi8::LoraArgs p{};
    p.x = x, p.ldx = ldx, p.a = a, p.b = b, p.scales = scales, p.adapter = adapter, p.y = y, p.ldy = ldy;
    p.M = M, p.N = N, p.K = K, p.L = L, p.R = R, p.ranks = parts * R, p.t = static_cast<float *>(workspace);
    return bi8::call_status(fn, bi8::launch_lora_add(p, part_columns, parts, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
