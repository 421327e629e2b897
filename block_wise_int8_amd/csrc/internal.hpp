// Host-side launchers of the block-wise INT8 kernels.  Arguments have been
// validated by the C ABI layer (abi.cpp) before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bi8 {

// A launch counts its threads along a dimension in 32 bits: one of 2^32 or more
// reports no error and runs the remainder modulo 2^32.
constexpr bool launch_fits(int64_t workgroups, int64_t threads) { return workgroups * threads <= 0xFFFFFFFFll; }

// Row-wise kernels of the e4m3 layer and the norm take their rows in bands of at
// most so many workgroups of 256 threads.
constexpr int64_t kBandWorkgroups = 1ll << 23;
static_assert(launch_fits(kBandWorkgroups, 256), "a band is one launch");

// GEMM kernels (the values are the BI8_GEMM_* variant ids of the C ABI).
enum class GemmPath : int { kAuto = 0, kSkinny = 1, kTile128x64 = 2, kTile256x128 = 3, kTile256x256 = 4 };

// Shape-based choice for the dense and the grouped GEMM (never kAuto).
GemmPath select_gemm_path(int64_t M, int64_t N, int64_t K);
GemmPath select_moe_gemm_path(int64_t R, int64_t N, int64_t K, int32_t E);

hipError_t launch_quant_act(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, int8_t *xq,
                            float *xs, hipStream_t stream);

// Gather form: output row m quantises row rows[m] of x ([src_rows, ldx]).
hipError_t launch_quant_act_gather(const uint16_t *x, int64_t src_rows, int64_t ldx, const int32_t *rows,
                                   int64_t M, int64_t K, int8_t *xq, float *xs, hipStream_t stream);

// Per-channel form (blocks of 1 x K): xs [M, 1], ws [N, 1], K <= 2^17.
hipError_t launch_gemm_per_channel(const int8_t *xq, const float *xs, const int8_t *w, const float *ws,
                                   const uint16_t *bias, uint16_t *y, int64_t M, int64_t N, int64_t K,
                                   hipStream_t stream);
// Per-token activation quantisation (one group of K per row).
hipError_t launch_quant_act_per_token(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, int8_t *xq,
                                      float *xs, hipStream_t stream);

// Offline block quantisation of a bf16 weight (128 x 128 blocks).
hipError_t launch_quant_weight(const uint16_t *w, int64_t N, int64_t K, int64_t ldw, int8_t *wq, float *ws,
                               hipStream_t stream);

// MoE steps around the grouped GEMM (E <= 1024, k <= 8).
hipError_t launch_moe_route(const float *logits, int64_t T, int32_t E, int32_t k, int32_t renorm,
                            int32_t *ids, float *weights, int32_t *sorted_token, int32_t *offsets,
                            int32_t *row_of, hipStream_t stream);
hipError_t launch_silu_mul_quant(const uint16_t *h, int64_t R, int64_t I, int8_t *aq, float *as,
                                 uint16_t *a_out, hipStream_t stream);
hipError_t launch_moe_combine(const uint16_t *y2, int64_t R, const int32_t *row_of, const float *w,
                              int64_t T, int32_t k, int64_t H, uint16_t *out, hipStream_t stream);

// Split K on a caller workspace for grids of few tiles (splits 1: no split).
int32_t splitk_splits(int64_t M, int64_t N, int64_t K);
int64_t splitk_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_ws(const int8_t *xq, const float *xs, const int8_t *w, const float *ws,
                          const uint16_t *bias, uint16_t *y, int64_t M, int64_t N, int64_t K, float *workspace,
                          int64_t workspace_bytes, hipStream_t stream);

hipError_t launch_gemm(GemmPath path, const int8_t *xq, const float *xs, const int8_t *w,
                       const float *ws, const uint16_t *bias, uint16_t *y, int64_t M, int64_t N,
                       int64_t K, hipStream_t stream);

// Host-side helpers of the C ABI layer (abi.cpp): the thread-local error
// message, the linear's argument checks and its two launches.
int32_t fail_status(int32_t status, const char *fmt, ...);
int32_t call_status(const char *fn, hipError_t e);
int32_t check_linear_args(const char *fn, const uint16_t *x, int64_t ldx, const int8_t *w, const float *ws,
                          const uint16_t *bias, const uint16_t *y, int64_t M, int64_t N, int64_t K,
                          int32_t block_n, int32_t block_k);
hipError_t launch_linear(const uint16_t *x, int64_t ldx, const int8_t *w, const float *ws, const uint16_t *bias,
                         uint16_t *y, int64_t M, int64_t N, int64_t K, int32_t block_n, int32_t block_k,
                         int8_t *xq, float *xs, hipStream_t st);

int64_t moe_gemm_workspace_bytes(int64_t R, int64_t N, int64_t K, int32_t E);
hipError_t launch_moe_gemm_ws(const int8_t *xq, const float *xs, const int32_t *offsets, const int8_t *w,
                              const float *ws, uint16_t *y, int64_t R, int64_t N, int64_t K, int32_t E,
                              float *workspace, int64_t workspace_bytes, hipStream_t stream);
hipError_t launch_moe_gemm_silu_quant(const int8_t *xq, const float *xs, const int32_t *offsets, const int8_t *w13,
                                      const float *ws13, int8_t *aq, float *as, int64_t R, int64_t I, int64_t K,
                                      int32_t E, hipStream_t stream);
hipError_t launch_moe_gemm(GemmPath path, const int8_t *xq, const float *xs, const int32_t *offsets,
                           const int8_t *w, const float *ws, uint16_t *y, int64_t R, int64_t N,
                           int64_t K, int32_t E, hipStream_t stream);

// The e4m3 layer (quant_fp8.hip, gemm_fp8.hip) and the normalising quantiser
// (norm.hip).  rows: the gather form of the quantiser (null: row m of x).
hipError_t launch_quant_act_fp8(const uint16_t *x, int64_t src_rows, int64_t ldx, const int32_t *rows, int64_t M,
                                int64_t K, uint8_t *xq, float *xs, hipStream_t stream);
hipError_t launch_silu_mul_quant_fp8(const uint16_t *h, int64_t R, int64_t I, uint8_t *aq, float *as,
                                     uint16_t *a_out, hipStream_t stream);
hipError_t launch_quant_weight_fp8(const uint16_t *w, int64_t N, int64_t K, int64_t ldw, uint8_t *wq, float *ws,
                                   hipStream_t stream);
enum class Fp8Path : int { kAuto = 0, kSkinny = 1, kTile128x64 = 2, kTile256x128 = 3, kTile256x256 = 4, kTile128x128 = 5,
                            kTile256x128F16 = 8 };
Fp8Path select_gemm_fp8_path(int64_t M, int64_t N, int64_t K);
Fp8Path select_moe_gemm_fp8_path(int64_t R, int64_t N, int64_t K, int32_t E);
Fp8Path select_layer_w13_path(int64_t R, int64_t N, int64_t K, int32_t E);
int64_t gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_fp8(Fp8Path path, const uint8_t *xq, const float *xs, const uint8_t *w, const float *ws,
                           const uint16_t *bias, uint16_t *y, int64_t M, int64_t N, int64_t K, float *workspace,
                           int64_t workspace_bytes, hipStream_t stream);
int64_t moe_gemm_fp8_workspace_bytes(int64_t R, int64_t N, int64_t K, int32_t E);
hipError_t launch_moe_gemm_silu_quant_fp8(const uint8_t *xq, const float *xs, const int32_t *offsets,
                                          const uint8_t *w13, const float *ws13, uint8_t *aq, float *as, int64_t R,
                                          int64_t I, int64_t K, int32_t E, bool f16, hipStream_t stream);
hipError_t launch_moe_gemm_fp8(Fp8Path path, const uint8_t *xq, const float *xs, const int32_t *offsets,
                               const uint8_t *w, const float *ws, uint16_t *y, int64_t R, int64_t N, int64_t K,
                               int32_t E, float *workspace, int64_t workspace_bytes, hipStream_t stream);
// h, ldr and ldh only with a residual; y may be null.
hipError_t launch_rmsnorm_quant(bool fp8, const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                const uint16_t *weight, double eps, int64_t M, int64_t H, uint16_t *h, int64_t ldh,
                                uint16_t *y, void *xq, float *xs, hipStream_t stream);

// Router with scores, a bias and groups (route.hip).
struct RouteArgs {
    const void *logits;   // [T, ldl], fp32 or bf16
    const float *bias;    // null: none
    int32_t *ids;
    float *weights;
    int32_t *sorted_token, *offsets, *row_of;
    int64_t ldl, T;
    double scale;
    int32_t bf16, E, k, score, groups, topk_groups, group_top, renormalize;
    // the launch's own: B tokens a workgroup, and on the workspace the counts
    // [workgroup, pitch], their sums over the workgroups before, the totals
    // (fours: lanes load their logits four at a time)
    int32_t block_tokens, log_groups, pitch, fours;
    uint8_t *counts;
    int32_t *before, *totals;
};
int64_t route_grouped_workspace_need(int64_t T, int32_t E);    // of a call
int64_t route_grouped_workspace_bytes(int64_t T, int32_t E);   // of any call of up to T tokens
hipError_t launch_moe_route_grouped(RouteArgs p, void *workspace, hipStream_t stream);

// Low-rank adapters beside a projection (lora.hip).
constexpr int kMaxParts = 4;
struct LoraArgs {
    const uint16_t *x, *a, *b;   // [M, ldx], [L, ranks, K], [L, N, R]
    const float *scales;         // null: 1
    const int32_t *adapter;
    uint16_t *y;
    float *t;                    // [splits, M, ranks]
    int64_t ldx, ldy, M, N, K;
    int32_t L, R, ranks;
    // the launch's own: blocks of rows; workgroups that share K, waves of one that
    // share the ranks; workgroups that share the adapters of a block of rows, in
    // either kernel, and how they do; rows 16 at a time; columns of y a workgroup, of K
    // a wave; first column and block of columns of each part, and behind the last
    int32_t blocks, splits, rank_waves, shrink_slots, slots, walk, candidates, by_adapter, narrow, columns;
    int64_t slice;
    int64_t part_first[kMaxParts + 1];
    int32_t part_blocks[kMaxParts + 1];
};
int64_t lora_workspace_need(int64_t M, int64_t K, int32_t ranks);    // of a call
int64_t lora_workspace_bytes(int64_t M, int64_t K, int32_t ranks);   // of any call of up to M rows
hipError_t launch_lora_add(LoraArgs p, const int64_t *part_columns, int32_t parts, hipStream_t stream);

// Norm and rotation of query and key heads (heads.hip).
constexpr int kMaxAxes = 4;
struct HeadsArgs {
    const uint16_t *q, *k;             // k: null with Hk = 0
    const uint16_t *q_weight, *k_weight;   // null: no norm
    uint16_t *q_out, *k_out;
    const float *table;                // [P, rot]
    const int32_t *positions;          // axis a at a * positions_axis
    int64_t q_token, q_head, k_token, k_head, q_out_token, q_out_head, k_out_token, k_out_head;
    int64_t P, positions_axis, T;
    double eps;
    int32_t Hq, Hk, D, rot, axes, interleaved;
    int32_t first[kMaxAxes];           // first pair of each axis (unused axes: past every pair)
    // the launch's own: lanes a head, groups of lanes a token and heads of each at
    // most, whether a chunk of pairs is one piece of the table, 1 / D
    int32_t log_lanes, q_groups, k_groups, each, table_chunks;
    double inverse;
};
hipError_t launch_qk_norm_rope(HeadsArgs p, hipStream_t stream);

}  // namespace bi8
