// C ABI of the e4m3 layer and of the normalising quantiser: argument checks on
// the host, then the launches on the caller's stream.  See
// include/blockint8_fp8.h and include/blockint8_norm.h for the contracts.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/blockint8_fp8.h"
#include "../../include/blockint8_norm.h"
#include "internal.hpp"

namespace {

using bi8::fail_status;

constexpr int64_t kMaxRows = 0x7FFFFFFFll;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int32_t done(const char *fn) { return bi8::call_status(fn, hipSuccess); }

int32_t check_rows(const char *fn, const char *what, int64_t rows) {
    if (rows < 0 || rows > kMaxRows)
        return fail_status(BI8_ERR_SHAPE, "%s: %s = %lld out of range", fn, what, (long long)rows);
    return BI8_OK;
}

int32_t check_columns(const char *fn, const char *what, int64_t K) {
    if (K <= 0 || K > BI8_MAX_K)
        return fail_status(BI8_ERR_SHAPE, "%s: %s = %lld out of range [1, %d]", fn, what, (long long)K, BI8_MAX_K);
    return BI8_OK;
}

int32_t check_pitch(const char *fn, const char *what, int64_t ld, int64_t K) {
    if (ld < K)
        return fail_status(BI8_ERR_SHAPE, "%s: %s = %lld < %lld columns", fn, what, (long long)ld, (long long)K);
    return BI8_OK;
}

int32_t check_block(const char *fn, int32_t block_n, int32_t block_k) {
    if (block_n != 128 || block_k != 128)
        return fail_status(BI8_ERR_BLOCK, "%s: only the [128, 128] block is implemented, got [%d, %d]", fn, block_n,
                           block_k);
    return BI8_OK;
}

int32_t check_align(const char *fn, const char *what, const void *p, uintptr_t a) {
    if (!aligned(p, a))
        return fail_status(BI8_ERR_ALIGN, "%s: %s must be %d-byte aligned", fn, what, (int)a);
    return BI8_OK;
}

int32_t null_pointer(const char *fn) { return fail_status(BI8_ERR_NULL, "%s: NULL tensor pointer", fn); }

int32_t check_workspace(const char *fn, const void *workspace, int64_t bytes) {
    if (bytes < 0) return fail_status(BI8_ERR_SHAPE, "%s: workspace_bytes = %lld < 0", fn, (long long)bytes);
    return check_align(fn, "workspace", workspace, 16);
}

#define BI8_TRY(expr)               \
    do {                            \
        const int32_t s_ = (expr);  \
        if (s_ != BI8_OK) return s_; \
    } while (0)

// The weight side, the output and the bias of a product (rows > 0).
int32_t check_product(const char *fn, const uint8_t *w, const float *ws, const uint16_t *bias, const uint16_t *y) {
    if (!w || !ws || !y) return null_pointer(fn);
    BI8_TRY(check_align(fn, "w", w, 16));
    BI8_TRY(check_align(fn, "ws", ws, 4));
    BI8_TRY(check_align(fn, "y", y, 2));
    return check_align(fn, "bias", bias, 2);
}

int32_t check_codes(const char *fn, const void *xq, const float *xs) {
    if (!xq || !xs) return null_pointer(fn);
    BI8_TRY(check_align(fn, "xq", xq, 16));
    return check_align(fn, "xs", xs, 4);
}

int32_t check_gemm_sizes(const char *fn, int64_t rows, int64_t N, int64_t K, int32_t block_n, int32_t block_k) {
    BI8_TRY(check_rows(fn, "row count", rows));
    if (N <= 0 || N > kMaxRows) return fail_status(BI8_ERR_SHAPE, "%s: N = %lld out of range", fn, (long long)N);
    BI8_TRY(check_columns(fn, "K", K));
    return check_block(fn, block_n, block_k);
}

int32_t check_experts(const char *fn, int32_t E) {
    if (E <= 0 || E > 65536) return fail_status(BI8_ERR_SHAPE, "%s: E = %d out of range [1, 65536]", fn, E);
    return BI8_OK;
}

int32_t check_variant(const char *fn, int32_t variant, int64_t K) {
    if (variant < BI8_GEMM_AUTO || (variant > BI8_GEMM_TILE_128X128 && variant != BI8_GEMM_TILE_256X128_F16))
        return fail_status(BI8_ERR_SHAPE, "%s: unknown kernel variant %d", fn, variant);
    if (K % 16 != 0 && variant != BI8_GEMM_AUTO)
        return fail_status(BI8_ERR_ALIGN, "%s: K = %lld is not a multiple of 16; that form has one kernel (variant "
                           "must be AUTO)", fn, (long long)K);
    return BI8_OK;
}

int32_t rmsnorm_quant(const char *fn, bool fp8, const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                      const uint16_t *weight, double eps, int64_t M, int64_t H, int32_t block_k, uint16_t *h,
                      int64_t ldh, uint16_t *y, void *xq, float *xs, void *stream) {
    BI8_TRY(check_rows(fn, "M", M));
    BI8_TRY(check_columns(fn, "H", H));
    BI8_TRY(check_pitch(fn, "ldx", ldx, H));
    if (residual) {
        BI8_TRY(check_pitch(fn, "ldr", ldr, H));
        BI8_TRY(check_pitch(fn, "ldh", ldh, H));
    }
    if (!(eps >= 0.0) || !std::isfinite(eps))
        return fail_status(BI8_ERR_SHAPE, "%s: eps = %g must be finite and not negative", fn, eps);
    BI8_TRY(check_block(fn, 128, block_k));
    if (M == 0) return done(fn);
    if (!x || !weight) return null_pointer(fn);
    if (residual && !h) return fail_status(BI8_ERR_NULL, "%s: a residual needs h for the sum", fn);
    if (!residual && h) return fail_status(BI8_ERR_NULL, "%s: h without a residual", fn);
    BI8_TRY(check_codes(fn, xq, xs));
    BI8_TRY(check_align(fn, "x", x, 2));
    BI8_TRY(check_align(fn, "residual", residual, 2));
    BI8_TRY(check_align(fn, "weight", weight, 2));
    BI8_TRY(check_align(fn, "h", h, 2));
    BI8_TRY(check_align(fn, "y", y, 2));
    return bi8::call_status(fn, bi8::launch_rmsnorm_quant(fp8, x, ldx, residual, ldr, weight, eps, M, H, h, ldh, y, xq,
                                                          xs, static_cast<hipStream_t>(stream)));
}

// The layer's workspace: parts at multiples of 256 bytes.  The w13 GEMM's output
// and the w2 GEMM's share one (the first is read before the second is written).
struct LayerPlan {
    bi8::Fp8Path w13;   // kAuto, or the kernel that holds the sums (see select_layer_w13_path)
    bool gated;         // w13 and the gating in one launch
    int64_t ids, weights, sorted_token, offsets, row_of, xq, xs, h, aq, as, partial, partial_bytes, bytes;
    LayerPlan(int64_t T, int64_t H, int64_t I, int32_t E, int32_t k, int32_t variant) {
        const int64_t R = T * k, HB = (H + 127) / 128, IB = (I + 127) / 128;
        w13 = variant == BI8_GEMM_AUTO ? bi8::select_layer_w13_path(R, 2 * I, H, E) : static_cast<bi8::Fp8Path>(variant);
        const bi8::Fp8Path path = w13 == bi8::Fp8Path::kAuto ? bi8::select_moe_gemm_fp8_path(R, 2 * I, H, E) : w13;
        gated = I % 128 == 0 && (path == bi8::Fp8Path::kTile256x128F16 || path == bi8::Fp8Path::kTile256x128 ||
                                 path == bi8::Fp8Path::kTile256x256);
        const int64_t p13 =
            gated || w13 != bi8::Fp8Path::kAuto ? 0 : bi8::moe_gemm_fp8_workspace_bytes(R, 2 * I, H, E);
        const int64_t p2 = bi8::moe_gemm_fp8_workspace_bytes(R, H, I, E);
        partial_bytes = p13 > p2 ? p13 : p2;
        const int64_t wide = !gated && 2 * I > H ? 2 * I : H;
        bytes = 0;
        auto take = [this](int64_t n) {
            const int64_t at = bytes;
            bytes += (n + 255) / 256 * 256;
            return at;
        };
        ids = take(R * 4);
        weights = take(R * 4);
        sorted_token = take(R * 4);
        offsets = take((E + 1) * 4);
        row_of = take(R * 4);
        xq = take(R * H);
        xs = take(R * HB * 4);
        h = take(R * wide * 2);
        aq = take(R * I);
        as = take(R * IB * 4);
        partial = take(partial_bytes);
    }
};

int32_t check_layer(const char *fn, int64_t T, int64_t H, int64_t I, int32_t E, int32_t k) {
    if (E < 1 || E > 1024) return fail_status(BI8_ERR_SHAPE, "%s: E = %d out of range [1, 1024]", fn, E);
    if (k < 1 || k > 8 || k > E) return fail_status(BI8_ERR_SHAPE, "%s: k = %d out of range [1, min(E, 8)]", fn, k);
    if (T < 0 || T > kMaxRows / k)
        return fail_status(BI8_ERR_SHAPE, "%s: T = %lld out of range", fn, (long long)T);
    BI8_TRY(check_columns(fn, "H", H));
    BI8_TRY(check_columns(fn, "I", I));
    if (H % 16 != 0 || I % 16 != 0)
        return fail_status(BI8_ERR_ALIGN, "%s: H = %lld and I = %lld must be multiples of 16", fn, (long long)H,
                           (long long)I);
    return BI8_OK;
}

}  // namespace

extern "C" {

int32_t blockint8_quant_act_fp8(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, int32_t block_k, uint8_t *xq,
                                float *xs, void *stream) {
    static const char fn[] = "blockint8_quant_act_fp8";
    BI8_TRY(check_rows(fn, "M", M));
    BI8_TRY(check_columns(fn, "K", K));
    BI8_TRY(check_pitch(fn, "ldx", ldx, K));
    BI8_TRY(check_block(fn, 128, block_k));
    if (M == 0) return done(fn);
    if (!x) return null_pointer(fn);
    BI8_TRY(check_codes(fn, xq, xs));
    BI8_TRY(check_align(fn, "x", x, 2));
    return bi8::call_status(fn, bi8::launch_quant_act_fp8(x, M, ldx, nullptr, M, K, xq, xs,
                                                          static_cast<hipStream_t>(stream)));
}

int32_t blockint8_quant_act_gather_fp8(const uint16_t *x, int64_t T, int64_t ldx, const int32_t *rows, int64_t R,
                                       int64_t K, int32_t block_k, uint8_t *xq, float *xs, void *stream) {
    static const char fn[] = "blockint8_quant_act_gather_fp8";
    BI8_TRY(check_rows(fn, "R", R));
    BI8_TRY(check_rows(fn, "T", T));
    BI8_TRY(check_columns(fn, "K", K));
    BI8_TRY(check_pitch(fn, "ldx", ldx, K));
    BI8_TRY(check_block(fn, 128, block_k));
    if (R == 0) return done(fn);
    if (!rows || (T > 0 && !x)) return null_pointer(fn);
    BI8_TRY(check_codes(fn, xq, xs));
    BI8_TRY(check_align(fn, "x", x, 2));
    BI8_TRY(check_align(fn, "rows", rows, 4));
    return bi8::call_status(fn, bi8::launch_quant_act_fp8(x, T, ldx, rows, R, K, xq, xs,
                                                          static_cast<hipStream_t>(stream)));
}

int32_t blockint8_silu_mul_quant_fp8(const uint16_t *h, int64_t R, int64_t I, int32_t block_k, uint8_t *aq, float *as,
                                     uint16_t *a, void *stream) {
    static const char fn[] = "blockint8_silu_mul_quant_fp8";
    BI8_TRY(check_rows(fn, "R", R));
    BI8_TRY(check_columns(fn, "I", I));
    if (I % 16 != 0) return fail_status(BI8_ERR_ALIGN, "%s: I = %lld must be a multiple of 16", fn, (long long)I);
    BI8_TRY(check_block(fn, 128, block_k));
    if (R == 0) return done(fn);
    if (!h) return null_pointer(fn);
    BI8_TRY(check_codes(fn, aq, as));
    BI8_TRY(check_align(fn, "h", h, 16));
    BI8_TRY(check_align(fn, "a", a, 16));
    return bi8::call_status(fn, bi8::launch_silu_mul_quant_fp8(h, R, I, aq, as, a, static_cast<hipStream_t>(stream)));
}

int32_t blockint8_quant_weight_fp8(const uint16_t *w, int64_t N, int64_t K, int64_t ldw, int32_t block_n,
                                   int32_t block_k, uint8_t *wq, float *ws, void *stream) {
    static const char fn[] = "blockint8_quant_weight_fp8";
    if (N < 0 || N > 65535ll * 128)
        return fail_status(BI8_ERR_SHAPE, "%s: N = %lld out of range", fn, (long long)N);
    BI8_TRY(check_columns(fn, "K", K));
    BI8_TRY(check_pitch(fn, "ldw", ldw, K));
    BI8_TRY(check_block(fn, block_n, block_k));
    if (N == 0) return done(fn);
    if (!w) return null_pointer(fn);
    BI8_TRY(check_codes(fn, wq, ws));
    BI8_TRY(check_align(fn, "w", w, 2));
    return bi8::call_status(fn, bi8::launch_quant_weight_fp8(w, N, K, ldw, wq, ws, static_cast<hipStream_t>(stream)));
}

int32_t blockint8_gemm_fp8_select(int64_t M, int64_t N, int64_t K) {
    return static_cast<int32_t>(bi8::select_gemm_fp8_path(M, N, K));
}

int32_t blockint8_moe_gemm_fp8_select(int64_t R, int64_t N, int64_t K, int32_t E) {
    return static_cast<int32_t>(bi8::select_moe_gemm_fp8_path(R, N, K, E > 0 ? E : 1));
}

int32_t blockint8_gemm_fp8_variant(int32_t variant, const uint8_t *xq, const float *xs, const uint8_t *w,
                                   const float *ws, const uint16_t *bias, uint16_t *y, int64_t M, int64_t N, int64_t K,
                                   int32_t block_n, int32_t block_k, void *workspace, int64_t workspace_bytes,
                                   void *stream) {
    static const char fn[] = "blockint8_gemm_fp8";
    BI8_TRY(check_variant(fn, variant, K));
    BI8_TRY(check_gemm_sizes(fn, M, N, K, block_n, block_k));
    BI8_TRY(check_workspace(fn, workspace, workspace_bytes));
    if (M == 0) return done(fn);
    BI8_TRY(check_codes(fn, xq, xs));
    BI8_TRY(check_product(fn, w, ws, bias, y));
    return bi8::call_status(fn, bi8::launch_gemm_fp8(static_cast<bi8::Fp8Path>(variant), xq, xs, w, ws, bias, y, M, N,
                                                     K, static_cast<float *>(workspace),
                                                     workspace ? workspace_bytes : 0,
                                                     static_cast<hipStream_t>(stream)));
}

int32_t blockint8_gemm_fp8(const uint8_t *xq, const float *xs, const uint8_t *w, const float *ws, const uint16_t *bias,
                           uint16_t *y, int64_t M, int64_t N, int64_t K, int32_t block_n, int32_t block_k,
                           void *workspace, int64_t workspace_bytes, void *stream) {
    return blockint8_gemm_fp8_variant(BI8_GEMM_AUTO, xq, xs, w, ws, bias, y, M, N, K, block_n, block_k, workspace,
                                      workspace_bytes, stream);
}

int64_t blockint8_gemm_fp8_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || M > kMaxRows || N <= 0 || N > kMaxRows || K <= 0 || K > BI8_MAX_K) return 0;
    return bi8::gemm_fp8_workspace_bytes(M, N, K);
}

int32_t blockint8_linear_fp8(const uint16_t *x, int64_t ldx, const uint8_t *w, const float *ws, const uint16_t *bias,
                             uint16_t *y, int64_t M, int64_t N, int64_t K, int32_t block_n, int32_t block_k,
                             uint8_t *xq_workspace, float *xs_workspace, void *workspace, int64_t workspace_bytes,
                             void *stream) {
    static const char fn[] = "blockint8_linear_fp8";
    BI8_TRY(check_gemm_sizes(fn, M, N, K, block_n, block_k));
    BI8_TRY(check_pitch(fn, "ldx", ldx, K));
    BI8_TRY(check_workspace(fn, workspace, workspace_bytes));
    if (M == 0) return done(fn);
    if (!x) return null_pointer(fn);
    BI8_TRY(check_align(fn, "x", x, 2));
    BI8_TRY(check_codes(fn, xq_workspace, xs_workspace));
    BI8_TRY(check_product(fn, w, ws, bias, y));
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = bi8::launch_quant_act_fp8(x, M, ldx, nullptr, M, K, xq_workspace, xs_workspace, st);
    if (e == hipSuccess)
        e = bi8::launch_gemm_fp8(bi8::Fp8Path::kAuto, xq_workspace, xs_workspace, w, ws, bias, y, M, N, K, static_cast<float *>(workspace),
                                 workspace ? workspace_bytes : 0, st);
    return bi8::call_status(fn, e);
}

int32_t blockint8_moe_gemm_fp8_variant(int32_t variant, const uint8_t *xq, const float *xs,
                                       const int32_t *expert_offsets, const uint8_t *w, const float *ws, uint16_t *y,
                                       int64_t R, int64_t N, int64_t K, int32_t E, int32_t block_n, int32_t block_k,
                                       void *workspace, int64_t workspace_bytes, void *stream) {
    static const char fn[] = "blockint8_moe_gemm_fp8";
    BI8_TRY(check_variant(fn, variant, 16));
    BI8_TRY(check_experts(fn, E));
    BI8_TRY(check_gemm_sizes(fn, R, N, K, block_n, block_k));
    if (K % 16 != 0) return fail_status(BI8_ERR_ALIGN, "%s: K = %lld must be a multiple of 16", fn, (long long)K);
    BI8_TRY(check_workspace(fn, workspace, workspace_bytes));
    if (R == 0) return done(fn);
    if (!expert_offsets) return null_pointer(fn);
    BI8_TRY(check_align(fn, "expert_offsets", expert_offsets, 4));
    BI8_TRY(check_codes(fn, xq, xs));
    BI8_TRY(check_product(fn, w, ws, nullptr, y));
    return bi8::call_status(fn, bi8::launch_moe_gemm_fp8(static_cast<bi8::Fp8Path>(variant), xq, xs, expert_offsets, w,
                                                         ws, y, R, N, K, E, static_cast<float *>(workspace),
                                                         workspace ? workspace_bytes : 0,
                                                         static_cast<hipStream_t>(stream)));
}

int32_t blockint8_moe_gemm_fp8(const uint8_t *xq, const float *xs, const int32_t *expert_offsets, const uint8_t *w,
                               const float *ws, uint16_t *y, int64_t R, int64_t N, int64_t K, int32_t E,
                               int32_t block_n, int32_t block_k, void *workspace, int64_t workspace_bytes,
                               void *stream) {
    return blockint8_moe_gemm_fp8_variant(BI8_GEMM_AUTO, xq, xs, expert_offsets, w, ws, y, R, N, K, E, block_n, block_k,
                                          workspace, workspace_bytes, stream);
}

int32_t blockint8_moe_gemm_silu_quant_fp8(const uint8_t *xq, const float *xs, const int32_t *expert_offsets,
                                          const uint8_t *w13, const float *ws13, uint8_t *aq, float *as, int64_t R,
                                          int64_t I, int64_t K, int32_t E, int32_t block_n, int32_t block_k,
                                          void *stream) {
    static const char fn[] = "blockint8_moe_gemm_silu_quant_fp8";
    BI8_TRY(check_experts(fn, E));
    if (I <= 0 || I % 128 != 0 || I > kMaxRows / 2)
        return fail_status(BI8_ERR_SHAPE, "%s: I = %lld must be a positive multiple of 128", fn, (long long)I);
    BI8_TRY(check_gemm_sizes(fn, R, 2 * I, K, block_n, block_k));
    if (K % 16 != 0) return fail_status(BI8_ERR_ALIGN, "%s: K = %lld must be a multiple of 16", fn, (long long)K);
    if (R == 0) return done(fn);
    if (!expert_offsets || !w13 || !ws13) return null_pointer(fn);
    BI8_TRY(check_align(fn, "expert_offsets", expert_offsets, 4));
    BI8_TRY(check_codes(fn, xq, xs));
    BI8_TRY(check_codes(fn, aq, as));
    BI8_TRY(check_align(fn, "w13", w13, 16));
    BI8_TRY(check_align(fn, "ws13", ws13, 4));
    return bi8::call_status(fn, bi8::launch_moe_gemm_silu_quant_fp8(xq, xs, expert_offsets, w13, ws13, aq, as, R, I, K,
                                                                    E, false, static_cast<hipStream_t>(stream)));
}

int64_t blockint8_moe_gemm_fp8_workspace_size(int64_t R, int64_t N, int64_t K, int32_t E) {
    if (R <= 0 || R > kMaxRows || N <= 0 || N > kMaxRows || K <= 0 || K > BI8_MAX_K || K % 16 != 0 || E <= 0 ||
        E > 65536)
        return 0;
    return bi8::moe_gemm_fp8_workspace_bytes(R, N, K, E);
}

int64_t blockint8_moe_layer_fp8_workspace_size(int64_t T, int64_t H, int64_t I, int32_t E, int32_t k) {
    if (E < 1 || E > 1024 || k < 1 || k > 8 || k > E || T <= 0 || T > kMaxRows / k || H <= 0 || H > BI8_MAX_K ||
        H % 16 != 0 || I <= 0 || I > BI8_MAX_K || I % 16 != 0)
        return 0;
    return LayerPlan(T, H, I, E, k, BI8_GEMM_AUTO).bytes;
}

int32_t blockint8_moe_layer_fp8_select(int64_t T, int64_t H, int64_t I, int32_t E, int32_t k) {
    if (blockint8_moe_layer_fp8_workspace_size(T, H, I, E, k) == 0) return BI8_GEMM_AUTO;
    const LayerPlan p(T, H, I, E, k, BI8_GEMM_AUTO);
    if (p.w13 != bi8::Fp8Path::kAuto) return static_cast<int32_t>(p.w13);
    if (!p.gated && bi8::moe_gemm_fp8_workspace_bytes(T * k, 2 * I, H, E) > 0) return BI8_GEMM_TILE_128X64;
    return static_cast<int32_t>(bi8::select_moe_gemm_fp8_path(T * k, 2 * I, H, E));
}

int32_t blockint8_moe_layer_fp8(const uint16_t *x, int64_t ldx, const float *logits, const uint8_t *w13,
                                const float *ws13, const uint8_t *w2, const float *ws2, uint16_t *out, int64_t T,
                                int64_t H, int64_t I, int32_t E, int32_t k, int32_t renormalize, int32_t block_n,
                                int32_t block_k, void *workspace, int64_t workspace_bytes, void *stream) {
    return blockint8_moe_layer_fp8_variant(BI8_GEMM_AUTO, x, ldx, logits, w13, ws13, w2, ws2, out, T, H, I, E, k,
                                           renormalize, block_n, block_k, workspace, workspace_bytes, stream);
}

int32_t blockint8_moe_layer_fp8_variant(int32_t variant, const uint16_t *x, int64_t ldx, const float *logits,
                                        const uint8_t *w13, const float *ws13, const uint8_t *w2, const float *ws2,
                                        uint16_t *out, int64_t T, int64_t H, int64_t I, int32_t E, int32_t k,
                                        int32_t renormalize, int32_t block_n, int32_t block_k, void *workspace,
                                        int64_t workspace_bytes, void *stream) {
    static const char fn[] = "blockint8_moe_layer_fp8";
    if (variant != BI8_GEMM_AUTO && variant != BI8_GEMM_TILE_256X128_F16)
        return fail_status(BI8_ERR_SHAPE, "%s: variant %d is not one of the layer's", fn, variant);
    BI8_TRY(check_layer(fn, T, H, I, E, k));
    BI8_TRY(check_pitch(fn, "ldx", ldx, H));
    BI8_TRY(check_block(fn, block_n, block_k));
    if (T == 0) return done(fn);
    if (!x || !logits || !w13 || !ws13 || !w2 || !ws2 || !out || !workspace) return null_pointer(fn);
    BI8_TRY(check_align(fn, "x", x, 2));
    BI8_TRY(check_align(fn, "logits", logits, 4));
    BI8_TRY(check_align(fn, "w13", w13, 16));
    BI8_TRY(check_align(fn, "ws13", ws13, 4));
    BI8_TRY(check_align(fn, "w2", w2, 16));
    BI8_TRY(check_align(fn, "ws2", ws2, 4));
    BI8_TRY(check_align(fn, "out", out, 16));
    BI8_TRY(check_align(fn, "workspace", workspace, 256));
    const LayerPlan p(T, H, I, E, k, variant);
    if (workspace_bytes < p.bytes)
        return fail_status(BI8_ERR_SHAPE, "%s: workspace_bytes = %lld < %lld", fn, (long long)workspace_bytes,
                           (long long)p.bytes);
    char *const at = static_cast<char *>(workspace);
    auto i32 = [at](int64_t off) { return reinterpret_cast<int32_t *>(at + off); };
    auto f32 = [at](int64_t off) { return reinterpret_cast<float *>(at + off); };
    auto u8 = [at](int64_t off) { return reinterpret_cast<uint8_t *>(at + off); };
    uint16_t *const h = reinterpret_cast<uint16_t *>(at + p.h);
    float *const partial = p.partial_bytes ? f32(p.partial) : nullptr;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t R = T * k;
    hipError_t e = bi8::launch_moe_route(logits, T, E, k, renormalize, i32(p.ids), f32(p.weights), i32(p.sorted_token),
                                         i32(p.offsets), i32(p.row_of), st);
    if (e == hipSuccess)
        e = bi8::launch_quant_act_fp8(x, T, ldx, i32(p.sorted_token), R, H, u8(p.xq), f32(p.xs), st);
    if (p.gated) {
        if (e == hipSuccess)
            e = bi8::launch_moe_gemm_silu_quant_fp8(u8(p.xq), f32(p.xs), i32(p.offsets), w13, ws13, u8(p.aq), f32(p.as),
                                                    R, I, H, E, p.w13 == bi8::Fp8Path::kTile256x128F16, st);
    } else {
        if (e == hipSuccess)
            e = bi8::launch_moe_gemm_fp8(p.w13, u8(p.xq), f32(p.xs), i32(p.offsets), w13, ws13, h, R, 2 * I, H, E,
                                         partial, p.partial_bytes, st);
        if (e == hipSuccess) e = bi8::launch_silu_mul_quant_fp8(h, R, I, u8(p.aq), f32(p.as), nullptr, st);
    }
    if (e == hipSuccess)
        e = bi8::launch_moe_gemm_fp8(bi8::Fp8Path::kAuto, u8(p.aq), f32(p.as), i32(p.offsets), w2, ws2, h, R, H, I, E,
                                     partial, p.partial_bytes, st);
    if (e == hipSuccess) e = bi8::launch_moe_combine(h, R, i32(p.row_of), f32(p.weights), T, k, H, out, st);
    return bi8::call_status(fn, e);
}

int32_t blockint8_rmsnorm_quant(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                const uint16_t *weight, double eps, int64_t M, int64_t H, int32_t block_k, uint16_t *h,
                                int64_t ldh, uint16_t *y, int8_t *xq, float *xs, void *stream) {
    return rmsnorm_quant("blockint8_rmsnorm_quant", false, x, ldx, residual, ldr, weight, eps, M, H, block_k, h, ldh, y,
                         xq, xs, stream);
}

int32_t blockint8_rmsnorm_quant_fp8(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                    const uint16_t *weight, double eps, int64_t M, int64_t H, int32_t block_k,
                                    uint16_t *h, int64_t ldh, uint16_t *y, uint8_t *xq, float *xs, void *stream) {
    return rmsnorm_quant("blockint8_rmsnorm_quant_fp8", true, x, ldx, residual, ldr, weight, eps, M, H, block_k, h,
                         ldh, y, xq, xs, stream);
}

}  // extern "C"
