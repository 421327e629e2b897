// Shared by the block-scaled GEMM kernels of every element type (gfx950): the
// kernel arguments, range-checked operand loads, the order of the tiles
// (dense and grouped by expert), the split tail of a grouped GEMM and the
// reductions that add up the splits' fp32 partial sums.  Operands are bytes
// here; each kernel file gives them their meaning.
#pragma once

#include "common.hpp"
#include "internal.hpp"

namespace bi8 {

namespace {

struct GemmArgs {
    const int8_t *xq;
    const float *xs;
    const int8_t *w;
    const float *ws;
    const uint16_t *bias;
    uint16_t *y;
    const int32_t *offsets;   // MoE only: [E + 1] row offsets per expert
    int64_t M;                // rows (R for MoE)
    int64_t N;
    int64_t K;
    int64_t KB;               // ceil(K / 128)
    int64_t NB;               // ceil(N / 128)
    int64_t tiles_m;          // dense: ceil(M / BM); MoE: upper bound of m-tiles
    int64_t tiles_n;
    int32_t E;
    int32_t wide_store;       // y rows allow 8-byte stores (N % 4 == 0, y 8-byte aligned)
    float acc_bias;           // kAccBias, kept in a scalar register (see biased_acc_to_f32)
    float *partial;           // split K: fp32 partial sums [splits, M, N] (workspace)
    int64_t kb_per_split;     // split K: K blocks per split (the last split may hold fewer)
    int8_t *aq;               // gated MoE epilogue: 8-bit codes [M, I] of silu(gate) * up
    float *as;                // gated MoE epilogue: their scales [M, I / 128]
    int64_t I;                // gated MoE epilogue: intermediate size (N = 2 I)
};

__device__ __forceinline__ u32x4 buf_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
}

__device__ __forceinline__ float buf_load_f32(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
}

__device__ __forceinline__ i32x4 as_i32x4(u32x4 v) {
    return __builtin_bit_cast(i32x4, v);
}

// 16 bytes at any byte offset `off` of a buffer whose base is 4-byte aligned:
// five aligned 4-byte loads (each range-checked on its own, so a dword past
// the buffer's end reads as zero) and byte shifts.  For rows of a K that is
// not a multiple of 16, which start at any byte.
__device__ __forceinline__ u32x4 buf_load16_any(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    const uint32_t a = off & ~3u, sh = off & 3u;
    uint32_t d[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) d[i] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)(a + 4u * i), 0, 0);
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_alignbyte(d[i + 1], d[i], sh);
    return v;
}

// Keep the first n bytes of a 16-byte operand fragment (none for n <= 0, all
// for n >= 16): the part of a fragment that lies past the end of a row.
__device__ __forceinline__ i32x4 keep_bytes(i32x4 v, int64_t n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t b = n - 4 * i;
        v[i] = b >= 4 ? v[i] : (b <= 0 ? 0 : (int32_t)((uint32_t)v[i] & ((1u << (8 * b)) - 1u)));
    }
    return v;
}

// Buffer resource for bytes [p, p + n) of a tensor at any byte address: the
// base rounded down to 4 bytes (delta = p % 4 bytes before p) and the range
// rounded up to whole dwords (a dword holding a byte of the tensor lies on the
// same page, so reading all of it is safe).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc_any(const int8_t *p, int64_t n, uint32_t &delta) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    delta = (uint32_t)(a & 3u);
    return make_rsrc(reinterpret_cast<const void *>(a - delta), clamp_bytes((n + delta + 3) & ~(int64_t)3));
}

// Spread consecutive workgroup ids (dispatched round-robin over the 8 XCDs)
// so that each XCD receives a contiguous range of tiles and its L2 sees
// neighbouring tiles.  Bijective on [0, total).
__device__ __forceinline__ int64_t xcd_remap(int64_t bid, int64_t total) {
    const int64_t q = total >> 3, r = total & 7;
    const int64_t xcd = bid & 7, slot = bid >> 3;
    return xcd * q + (xcd < r ? xcd : r) + slot;
}

// m-tiles per group in the tile order: consecutive workgroups walk a group's
// m-tiles for one n-tile, then the next n-tile (measured: 8 for the 256 x 128
// tile, 4 for 256 x 256, where 8 was 15 % slower at 4096^3)
constexpr int64_t kGroupM = 8;

// Grouped GEMM: at most this many m-tiles of one expert advance together
// along n (the workload's experts hold 4-5 tiles of 256 rows and 8-9 of 128:
// each is one group).  Measured at the MoE size: 8 and 32 within 1 %.
constexpr int64_t kGroupMMoe = 16;

struct Tile {
    int64_t n0;    // first weight row / output column
    int64_t m0;    // first activation row (global row of xq, xs, y)
    int64_t rows;  // valid activation rows in this tile
    const int8_t *w;
    const float *ws;
    int32_t split = -1;   // grouped tail split: this unit's split of the tile (-1: the whole tile)
    int32_t nsplit = 1;   // grouped tail split: splits of the tile
    int64_t unit = 0;     // grouped tail split: the unit's partial-sum slot
};

// Split tail of a grouped GEMM (one workgroup per CU): the tiles that exist,
// T, fill F = 256 * floor(T / 256) whole rounds of the chip's CUs; the other
// T - F run split over K into S parts each, so that their units fill one more
// round.  S = min(256 / (T - F), KB, 16), trimmed so that no split is empty;
// S = 1 when splitting would not shorten the last round.
constexpr int64_t kTailRound = 256;
constexpr int64_t kTailMaxSplitsPlan = 16;   // at most this many splits per tail tile
struct TailPlan {
    int64_t full;     // F
    int64_t tail;     // T - F
    int32_t splits;   // S
    int64_t per;      // K blocks per split
};
__device__ __forceinline__ TailPlan tail_plan(int64_t total, int64_t KB) {
    static_assert((kTailRound & (kTailRound - 1)) == 0, "power of two");
    TailPlan t;
    t.full = total & ~(kTailRound - 1);
    t.tail = total - t.full;
    // (32-bit division: tail < 256 and KB <= 2^16, K being at most 2^23)
    uint32_t s = t.tail > 0 ? (uint32_t)kTailRound / (uint32_t)t.tail : 1u;
    s = s < KB ? s : (uint32_t)KB;
    s = s < kTailMaxSplitsPlan ? s : (uint32_t)kTailMaxSplitsPlan;
    s = s < 1 ? 1 : s;
    const uint32_t kb = (uint32_t)KB;
    t.per = (kb + s - 1) / s;
    t.splits = (int32_t)((kb + (uint32_t)t.per - 1) / (uint32_t)t.per);
    return t;
}

// The tiles that exist in a grouped GEMM with BM-row tiles: sum over the
// expert segments (offsets clamped to [0, R]) of ceil(rows / BM).
template <int BM>
__device__ __forceinline__ int64_t moe_tiles_m(const GemmArgs &p) {
    int64_t n = 0;
    for (int32_t e = 0; e < p.E; ++e) {
        int64_t a = p.offsets[e], b = p.offsets[e + 1];
        a = a < 0 ? 0 : (a > p.M ? p.M : a);
        b = b < a ? a : (b > p.M ? p.M : b);
        n += (b - a + BM - 1) / BM;
    }
    return n;
}

// Tile `tid` of the grouped order over tiles_m m-tiles: groups of GM m-tiles
// advance together along n, so the tiles that share a weight tile run side by
// side.  For the grouped GEMM the groups follow the expert segments: expert e's
// m-tiles (found by walking the segments) in groups of at most kGroupMMoe, so
// that no group mixes two experts' weights (groups across segment boundaries
// read both experts' weight tiles, and most of the weights twice).
template <int BN, int BM, bool MOE, int64_t GM>
__device__ __forceinline__ bool tile_at(const GemmArgs &p, int64_t tid, int64_t tiles_m, Tile &t) {
    // (32-bit division: tid < 2^31 and GM * tiles_n < 2^31, both launch limits)
    if constexpr (!MOE) {
        const uint32_t span = (uint32_t)(GM * p.tiles_n);
        const uint32_t group = (uint32_t)tid / span;
        const int64_t first_m = (int64_t)group * GM;
        const uint32_t gsize = (uint32_t)(tiles_m - first_m < GM ? tiles_m - first_m : GM);
        const uint32_t in = (uint32_t)tid - group * span;
        t.n0 = (int64_t)(in / gsize) * BN;
        t.m0 = (first_m + in % gsize) * BM;
        t.rows = p.M - t.m0 < BM ? p.M - t.m0 : BM;
        t.w = p.w;
        t.ws = p.ws;
        return true;
    } else {
        int64_t rem = tid;
        for (int32_t e = 0; e < p.E; ++e) {
            // clamp to [0, R] so that offsets breaking the precondition can
            // never address rows outside xq / y
            int64_t a = p.offsets[e], b = p.offsets[e + 1];
            a = a < 0 ? 0 : (a > p.M ? p.M : a);
            b = b < a ? a : (b > p.M ? p.M : b);
            const int64_t cnt = (b - a + BM - 1) / BM;
            const int64_t espan = cnt * p.tiles_n;
            if (rem < espan) {
                const uint32_t span = (uint32_t)(kGroupMMoe * p.tiles_n);
                const uint32_t group = (uint32_t)rem / span;
                const int64_t first_m = (int64_t)group * kGroupMMoe;
                const uint32_t gsize = (uint32_t)(cnt - first_m < kGroupMMoe ? cnt - first_m : kGroupMMoe);
                const uint32_t in = (uint32_t)rem - group * span;
                t.n0 = (int64_t)(in / gsize) * BN;
                t.m0 = a + (first_m + in % gsize) * BM;
                t.rows = b - t.m0 < BM ? b - t.m0 : BM;
                t.w = p.w + (int64_t)e * p.N * p.K;
                t.ws = p.ws + (int64_t)e * p.NB * p.KB;
                return true;
            }
            rem -= espan;
        }
        return false;
    }
}

template <int BN, int BM, bool MOE, int64_t GM = kGroupM, bool TAIL = false>
__device__ __forceinline__ bool decode_tile(const GemmArgs &p, Tile &t) {
    // MoE: the grid holds an upper bound of m-tiles (the segments' lengths are
    // only known on the device); the tiles that exist are counted here and
    // spread evenly over the XCDs, and the surplus workgroups exit.  (Mapped
    // over the whole grid instead, the missing tiles -- all at the end of the
    // order -- left the last XCD nearly idle: at R = 8192 over 8 experts the
    // w13 grid gave six XCDs 560 tiles each and one XCD 56.)
    // TAIL: workgroups [0, F) take the whole tiles of the full rounds (spread
    // over the XCDs as above), workgroup F + u split unit u of the tail: tile
    // F + u / S, split u % S.
    static_assert(!TAIL || MOE, "split tails are the grouped GEMM's");
    int64_t tiles_m = p.tiles_m;
    if constexpr (MOE) tiles_m = moe_tiles_m<BM>(p);
    const int64_t total = tiles_m * p.tiles_n;
    int64_t tid;
    if constexpr (MOE) {
        int64_t balanced = total;
        if constexpr (TAIL) {
            const TailPlan tp = tail_plan(total, p.KB);
            if (tp.splits > 1) {
                balanced = tp.full;
                if ((int64_t)blockIdx.x >= tp.full) {
                    const int64_t u = (int64_t)blockIdx.x - tp.full;
                    if (u >= tp.tail * tp.splits) return false;
                    tid = tp.full + u / tp.splits;
                    t.split = (int32_t)(u % tp.splits);
                    t.nsplit = tp.splits;
                    t.unit = u;
                    balanced = -1;
                }
            }
        }
        if (balanced >= 0) {
            const int64_t xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
            const int64_t q = balanced >> 3, r = balanced & 7;
            if (slot >= q + (xcd < r ? 1 : 0)) return false;
            tid = xcd * q + (xcd < r ? xcd : r) + slot;
        }
    } else {
        tid = xcd_remap(blockIdx.x, total);
    }
    return tile_at<BN, BM, MOE, GM>(p, tid, tiles_m, t);
}

// y[m, n] = bf16(sum over the splits, in split order, of partial[z, m, n]
// (+ bias[n])); four outputs of one row per thread when N % 4 == 0.
template <bool VEC>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float *__restrict__ partial, int32_t splits,
                                                            int64_t M, int64_t N, const uint16_t *__restrict__ bias,
                                                            uint16_t *__restrict__ y) {
    const int64_t MN = M * N;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * (VEC ? 4 : 1);
    if (i >= MN) return;
    if constexpr (VEC) {
        f32x4 acc = *reinterpret_cast<const f32x4 *>(partial + i);
        for (int32_t z = 1; z < splits; ++z) acc += *reinterpret_cast<const f32x4 *>(partial + z * MN + i);
        if (bias) {
            const int64_t n = i % N;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] += bf16_bits_to_f32(bias[n + e]);
        }
        *reinterpret_cast<uint2 *>(y + i) =
            make_uint2(f32x2_to_bf16x2_bits(acc[0], acc[1]), f32x2_to_bf16x2_bits(acc[2], acc[3]));
    } else {
        float acc = partial[i];
        for (int32_t z = 1; z < splits; ++z) acc += partial[z * MN + i];
        if (bias) acc += bf16_bits_to_f32(bias[i % N]);
        y[i] = (uint16_t)(f32x2_to_bf16x2_bits(acc, 0.0f) & 0xFFFFu);
    }
}

// Split tail of the grouped GEMM (BN x BM tiles): for each row r of each tail
// tile F + i, the S partial sums of its units added in split order and stored
// as bf16 -- the plan recomputed exactly as the GEMM's decoder computed it.
// A fixed grid (the tail's size is only known on the device); its waves take
// the (tile, row) pairs in turn, lane l columns
// [4l, 4l + 4) of every 256 columns, every split's load issued before the
// first add.
constexpr int kTailMaxSplits = 16;
static_assert(kTailMaxSplitsPlan <= kTailMaxSplits, "the reduce holds every split");
constexpr int kTailReduceWaves = 4;
// 1024 workgroups: at the MoE w2 size (32 tail tiles x 128 rows) one
// (tile, row) pair per wave, all loads in flight at once (256 workgroups:
// 17 us, four pairs per wave one after another)
#ifndef BI8_TAIL_REDUCE_BLOCKS
#define BI8_TAIL_REDUCE_BLOCKS 1024
#endif
constexpr int kTailReduceBlocks = BI8_TAIL_REDUCE_BLOCKS;
template <int BN, int BM>
__global__ __launch_bounds__(kTailReduceWaves * 64) void moe_tail_reduce_kernel(GemmArgs p) {
    const int64_t tiles_m = moe_tiles_m<BM>(p);
    const TailPlan tp = tail_plan(tiles_m * p.tiles_n, p.KB);
    if (tp.splits <= 1) return;
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * kTailReduceWaves + (threadIdx.x >> 6);
    const int64_t waves = (int64_t)gridDim.x * kTailReduceWaves;
    for (int64_t pair = wave; pair < tp.tail * BM; pair += waves) {
        const int64_t i = pair / BM;
        const int r = (int)(pair - i * BM);
        Tile t;
        if (!tile_at<BN, BM, true, kGroupM>(p, tp.full + i, tiles_m, t)) continue;
        if (r >= t.rows) continue;
        const float *slots = p.partial + i * tp.splits * (BM * BN) + (int64_t)r * BN;
        uint16_t *yrow = p.y + (t.m0 + r) * p.N;
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 256) {
            const int c = c0 + 4 * lane;
            const int64_t n = t.n0 + c;
            if (n >= p.N) continue;
            f32x4 part[kTailMaxSplits];
#pragma unroll
            for (int z = 0; z < kTailMaxSplits; ++z)
                if (z < tp.splits) part[z] = *reinterpret_cast<const f32x4 *>(slots + (int64_t)z * (BM * BN) + c);
            f32x4 acc = part[0];
#pragma unroll
            for (int z = 1; z < kTailMaxSplits; ++z)
                if (z < tp.splits) acc += part[z];
            if (p.wide_store && n + 4 <= p.N) {
                *reinterpret_cast<uint2 *>(yrow + n) =
                    make_uint2(f32x2_to_bf16x2_bits(acc[0], acc[1]), f32x2_to_bf16x2_bits(acc[2], acc[3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N) yrow[n + e] = (uint16_t)(f32x2_to_bf16x2_bits(acc[e], 0.0f) & 0xFFFFu);
            }
        }
    }
}

GemmArgs make_args(const int8_t *xq, const float *xs, const int8_t *w, const float *ws,
                   const uint16_t *bias, uint16_t *y, int64_t M, int64_t N, int64_t K) {
    GemmArgs p{};
    p.xq = xq;
    p.xs = xs;
    p.w = w;
    p.ws = ws;
    p.bias = bias;
    p.y = y;
    p.offsets = nullptr;
    p.M = M;
    p.N = N;
    p.K = K;
    p.KB = (K + kBlock - 1) / kBlock;
    p.NB = (N + kBlock - 1) / kBlock;
    p.E = 1;
    p.wide_store = (N % 4 == 0) && ((reinterpret_cast<uintptr_t>(y) & 7) == 0);
    p.acc_bias = kAccBias;
    return p;
}

}  // namespace

}  // namespace bi8
