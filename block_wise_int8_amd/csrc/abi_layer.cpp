// C ABI of the operators beside the 8-bit products: argument checks on the host,
// then the launches on the caller's stream.  See include/blockint8_heads.h for the
// contracts.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/blockint8_heads.h"
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

}  // extern "C"
