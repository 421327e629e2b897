// Block-scaled e4m3 GEMM kernels for gfx950:
//   y[m, n] = bf16( sum_g (sum_{k in g} xq[m, k] w[n, k]) xs[m, g] ws[n / 128, g] (+ bias[n]) )
// dense, and grouped by expert.
//
// A K block of 128 codes is two v_mfma_f32_32x32x64_f8f6f4 in the tiled kernels:
// the block sum comes out of the matrix core in fp32 and enters the running sum by
// one fma with the block's scale.  Inside, the matrix core adds eight consecutive
// products at a time, aligned to the largest and cut 2^-13 below its leading bit
// (measured: beside 2^16 a product of 2^3 counts and one of 2^2 does not; the
// 16x16x128 form and the older 16x16x32 do the same), and those sums in fp32.  That
// is 7 2^-13 of the largest product of the eight at most, against the 2^-4 to which
// each code was rounded.  f16 MFMAs of the converted codes avoid it at half the
// rate: the streaming kernel, whose matrix core is idle most of the time, and the
// F16 variant of the 256 x 128 tiles run those.
//
// The weight rows are the A operand (rows of the result = output columns n) and
// the activation rows the B operand (columns = tokens m), so that a lane holds
// one token and columns of one 128-row weight block: the scale xs[m, g]
// ws[n / 128, g] is one factor a lane.
// K may be permuted inside a block as long as both operands agree, so a
// lane's 32 operand bytes are whichever two 16-byte pieces are cheapest to
// bring there.
//
// Scales and running sums are fp32; one rounding to bf16 at the store.
#include "codes.hpp"
#include "gemm_common.hpp"

namespace bi8 {

namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 join16(i32x4 a, i32x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Eight codes as f16, exactly (NaN stays NaN).
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f16x8 to_f16x8(int32_t lo, int32_t hi) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// ---------------------------------------------------------------------------
// Skinny path: few tokens, the weight streamed
// ---------------------------------------------------------------------------
//
// Bound by HBM: N K bytes of weight against 2 M N K operations.  `parts` of a
// workgroup's 8 waves split the K of 16 weight rows; with K short enough for
// fewer parts the other waves take further rows, so that every wave has U
// blocks (8 KB of weight) in flight.  At K = 4096 all 8 split it, and at
// N = 4096 each CU has one workgroup with its whole 64 KB share in flight.  A
// lane loads 32 bytes of weight per K block straight into registers, every
// load of U blocks is issued before the first MFMA, and the parts' sums meet
// in LDS.
//
// A K block is four v_mfma_f32_16x16x32_f16 of the codes as f16 values, whose sums
// binary32 holds (the one f8 MFMA that it could be took 0.3 us less of 7, 0 to 5 % of
// the longer times).
//
// Measured (weights from HBM): 1 x 131072 x 4096 91 us, 5.9 TB/s; 1 x 4096 x
// 4096 6.4 us, most of it one workgroup's latency; grouped, 8 experts of 28672 x
// 4096 (940 MB, read once by the counters) with a row each 156 us, 6.0 TB/s, with
// two each 169, 5.6; four of them with four rows each 89, 5.3.
// With 16 tokens or fewer two workgroups share a CU (128 registers at most: at
// 132, one a CU, 1 x 131072 x 4096 took 152 us).
//
// Rows [a, b) of the activations share the weight; they are taken 16 MT at a
// time.  Dense: [0, M), chunks over blockIdx.y.  MOE: one expert's segment, all
// of its chunks in turn (its weight rows then come from L2).
// ODD: K % 16 != 0, rows start at any byte (see buf_load16_any).
constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyUnroll = 4;
constexpr int skinny_unroll(int64_t mt) { return mt <= 3 ? kSkinnyUnroll : 2; }

// Host: 16-token groups of a chunk for so many rows, and waves that share a tile's K.
int64_t skinny_mt(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 48 ? 3 : 4; }
int32_t skinny_parts(int64_t KB) {
    int32_t parts = kSkinnyWaves;
    while (parts > 1 && KB <= parts / 2 * kSkinnyUnroll) parts /= 2;
    return parts;
}

// With fewer rows than experts the grid covers as many experts as there are rows,
// and e, the number of one among those that have rows, becomes its index, [a, b)
// its segment; false behind the last.  (With workgroups for every expert, most of
// them without rows, 8 rows over 40 experts of 10848 x 1152 took 35 us, now 30.)
__device__ __forceinline__ bool expert_with_rows(const GemmArgs &p, uint32_t &e, int64_t &a, int64_t &b) {
    const int lane = threadIdx.x & 63;
    uint32_t nth = e;
    for (int32_t e0 = 0; e0 < p.E; e0 += 64) {
        int32_t la = 0, lb = 0;
        if (e0 + lane < p.E) {
            la = p.offsets[e0 + lane];
            lb = p.offsets[e0 + lane + 1];
        }
        const bool any = lb > la && lb > 0 && la < p.M;
        const uint64_t with = __ballot(any);
        const uint32_t count = (uint32_t)__builtin_popcountll(with);
        if (nth < count) {
            const uint32_t below = __builtin_amdgcn_mbcnt_hi((uint32_t)(with >> 32),
                                                             __builtin_amdgcn_mbcnt_lo((uint32_t)with, 0u));
            const int l = __builtin_ctzll(__ballot(any && below == nth));
            e = (uint32_t)(e0 + l);
            a = __builtin_amdgcn_readlane(la, l);
            b = __builtin_amdgcn_readlane(lb, l);
            return true;
        }
        nth -= count;
    }
    return false;
}

template <int MT, bool ODD, bool MOE>
__global__ __launch_bounds__(kSkinnyWaves * 64)
    __attribute__((amdgpu_waves_per_eu(MT == 1 && !ODD ? 4 : 2))) void gemm_fp8_skinny_kernel(
        GemmArgs p, int32_t blocks_per_wave, int32_t parts) {
    constexpr int U = skinny_unroll(MT);
    constexpr int kRows = 16 * MT;
    __shared__ __attribute__((aligned(16))) float red[kSkinnyWaves][MT][64][4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = kSkinnyWaves / parts;   // weight tiles of this workgroup
    const int part = wave & (parts - 1);      // (parts is a power of two)
    const int mine = wave / parts;
    const int row = lane & 15;    // weight row in the tile, and token column
    const int quad = lane >> 4;   // 32-byte quarter of a K block
    const int K = (int)p.K, KB = (int)p.KB;   // (K <= 2^23: offsets inside 64 rows fit 32 bits)

    int64_t n0, a = 0, b = p.M;
    const int8_t *w = p.w;
    const float *ws = p.ws;
    if constexpr (MOE) {
        uint32_t e = blockIdx.x / (uint32_t)p.tiles_n;
        n0 = (int64_t)(blockIdx.x - e * (uint32_t)p.tiles_n) * 16 * tiles;
        if (p.M >= p.E) {
            a = p.offsets[e];
            b = p.offsets[e + 1];
        } else if (!expert_with_rows(p, e, a, b)) {
            return;
        }
        a = a < 0 ? 0 : (a > p.M ? p.M : a);
        b = b < a ? a : (b > p.M ? p.M : b);
        w += (int64_t)e * p.N * p.K;
        ws += (int64_t)e * p.NB * p.KB;
    } else {
        n0 = (int64_t)blockIdx.x * 16 * tiles;
    }
    const int64_t wg_n0 = n0;
    n0 += mine * 16;

    // (ranges of at most 2^31 bytes: 16 MT rows of K <= 2^23)
    const int wrows = p.N - n0 < 16 ? (p.N > n0 ? (int)(p.N - n0) : 0) : 16;   // (0: a wave without rows)
    if (wrows == 0) n0 = wg_n0;
    uint32_t wd = 0;
    const __amdgpu_buffer_rsrc_t wr =
        ODD ? make_rsrc_any(w + n0 * p.K, wrows * K, wd) : make_rsrc(w + n0 * p.K, (uint32_t)(wrows * K));
    const float *ws_row = ws + (n0 / kBlock) * p.KB;
    auto load = [&](__amdgpu_buffer_rsrc_t r, uint32_t off) __attribute__((always_inline)) {
        return as_i32x4(ODD ? buf_load16_any(r, off) : buf_load16(r, off));
    };
    const int b_begin = part * blocks_per_wave;
    const int b_end = b_begin + blocks_per_wave < KB ? b_begin + blocks_per_wave : KB;

    // Weight loads in whole 128-byte lines: load lane l reads piece l % 8 of
    // tile row l / 8 (and of row 8 + l / 8); the MFMA wants pieces 2q, 2q + 1 of
    // row i in lane (i, q), brought there by ds_bpermute.
    const int lrow = lane >> 3, lchunk = lane & 7;
    const int bp0 = ((lane & 7) * 8 + 2 * quad) * 4;
    const bool upper = row >= 8;

    auto chunk = [&](int64_t m0) __attribute__((always_inline)) {
        const int mrows = b - m0 < kRows ? (int)(b - m0) : kRows;
        uint32_t xd = 0;
        const __amdgpu_buffer_rsrc_t xr = ODD ? make_rsrc_any(p.xq + m0 * p.K, mrows * K, xd)
                                              : make_rsrc(p.xq + m0 * p.K, (uint32_t)(mrows * K));
        const __amdgpu_buffer_rsrc_t sr = make_rsrc(p.xs + m0 * p.KB, (uint32_t)(mrows * KB * 4));
        f32x4 yv[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) yv[mt] = f32x4{0.f, 0.f, 0.f, 0.f};

        for (int b0 = b_begin; b0 < b_end; b0 += U) {
            i32x4 wa[U][2];
            i32x4 xb[U][MT][2];
            float xsv[U][MT];
            float wsv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kb = b0 + u;
                const bool ok = kb < b_end;
                const int kk = kb * kBlock + quad * 32;
                const bool in0 = ok && kk < K, in1 = ok && kk + 16 < K;
                if constexpr (ODD) {
                    // (a weight byte past K would meet a zeroed activation
                    // byte, but NaN codes times zero are NaN: cleared too)
                    wa[u][0] = keep_bytes(load(wr, in0 ? (uint32_t)(wd + row * K + kk) : kOobOffset), K - kk);
                    wa[u][1] = keep_bytes(load(wr, in1 ? (uint32_t)(wd + row * K + kk + 16) : kOobOffset), K - kk - 16);
                } else {
                    const int kc = kb * kBlock + lchunk * 16;
                    const bool inl = ok && kc < K;
                    wa[u][0] = load(wr, inl ? (uint32_t)(lrow * K + kc) : kOobOffset);
                    wa[u][1] = load(wr, inl ? (uint32_t)((lrow + 8) * K + kc) : kOobOffset);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int tok = mt * 16 + row;   // relative to m0
                    xb[u][mt][0] = i32x4{0, 0, 0, 0};
                    xb[u][mt][1] = i32x4{0, 0, 0, 0};
                    xsv[u][mt] = 0.f;
                    if (tok < mrows) {   // lanes past the rows load nothing
                        xb[u][mt][0] = load(xr, in0 ? (uint32_t)(xd + tok * K + kk) : kOobOffset);
                        xb[u][mt][1] = load(xr, in1 ? (uint32_t)(xd + tok * K + kk + 16) : kOobOffset);
                        if constexpr (ODD) {
                            xb[u][mt][0] = keep_bytes(xb[u][mt][0], K - kk);
                            xb[u][mt][1] = keep_bytes(xb[u][mt][1], K - kk - 16);
                        }
                        xsv[u][mt] = buf_load_f32(sr, ok ? (uint32_t)((tok * KB + kb) * 4) : kOobOffset);
                    }
                }
                wsv[u] = ws_row[ok ? kb : KB - 1];
            }
            // every load above is in flight before the first MFMA
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool ok = b0 + u < b_end;
                i32x8 wf;
                if constexpr (ODD) {
                    wf = join16(wa[u][0], wa[u][1]);
                } else {
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int lo0 = __builtin_amdgcn_ds_bpermute(bp0, wa[u][0][d]);
                        const int hi0 = __builtin_amdgcn_ds_bpermute(bp0, wa[u][1][d]);
                        const int lo1 = __builtin_amdgcn_ds_bpermute(bp0 + 4, wa[u][0][d]);
                        const int hi1 = __builtin_amdgcn_ds_bpermute(bp0 + 4, wa[u][1][d]);
                        wf[d] = upper ? hi0 : lo0;
                        wf[4 + d] = upper ? hi1 : lo1;
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const i32x8 xf = join16(xb[u][mt][0], xb[u][mt][1]);
                    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_f16x8(wf[2 * c], wf[2 * c + 1]),
                                                                     to_f16x8(xf[2 * c], xf[2 * c + 1]), acc, 0, 0, 0);
                    const float t = ok ? xsv[u][mt] * wsv[u] : 0.f;   // (past the end: another block's scale)
#pragma unroll
                    for (int i = 0; i < 4; ++i) yv[mt][i] = fmaf(acc[i], t, yv[mt][i]);
                }
            }
        }

        // 16x16 result: lane -> token lane & 15, weight rows 4 (lane >> 4) + i.  A
        // thread adds a lane's four over the parts.
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) *reinterpret_cast<f32x4 *>(red[wave][mt][lane]) = yv[mt];
        __syncthreads();
        for (int t = threadIdx.x; t < tiles * MT * 64; t += kSkinnyWaves * 64) {
            const int tile = t / (MT * 64), mt = (t >> 6) % MT;
            f32x4 sum = *reinterpret_cast<const f32x4 *>(red[tile * parts][mt][lane]);
            for (int v = 1; v < parts; ++v) sum += *reinterpret_cast<const f32x4 *>(red[tile * parts + v][mt][lane]);
            const int64_t ml = mt * 16 + row, n = wg_n0 + tile * 16 + 4 * quad;
            if (ml >= mrows || n >= p.N) continue;
            if (p.bias) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < p.N) sum[i] += bf16_bits_to_f32(p.bias[n + i]);
            }
            uint16_t *dst = p.y + (m0 + ml) * p.N + n;
            const uint2 o = make_uint2(f32x2_to_bf16x2_bits(sum[0], sum[1]), f32x2_to_bf16x2_bits(sum[2], sum[3]));
            if (p.wide_store) {
                *reinterpret_cast<uint2 *>(dst) = o;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < p.N) dst[i] = (uint16_t)((i < 2 ? o.x : o.y) >> (16 * (i & 1)));
            }
        }
    };
    if constexpr (!MOE && MT < 4) {   // (all rows are one chunk)
        chunk(0);
    } else {
        for (int64_t m0 = a + (int64_t)blockIdx.y * kRows; m0 < b; m0 += (int64_t)gridDim.y * kRows) {
            chunk(m0);
            __syncthreads();   // (the next chunk writes the sums again)
        }
    }
}

// chunks: workgroups that share the rows of one weight tile (dense)
template <int MT, bool ODD, bool MOE>
hipError_t launch_skinny_mt(GemmArgs p, int64_t chunks, hipStream_t stream) {
    const int32_t parts = skinny_parts(p.KB);
    const int64_t rows = 16 * (kSkinnyWaves / parts);
    p.tiles_n = (p.N + rows - 1) / rows;
    const int64_t blocks = p.tiles_n * (MOE && p.M < p.E ? p.M : p.E);
    if (!launch_fits(blocks, kSkinnyWaves * 64)) return hipErrorInvalidValue;
    if (chunks > 65535) chunks = 65535;
    const int32_t bpw = (int32_t)((p.KB + parts - 1) / parts);
    hipLaunchKernelGGL((gemm_fp8_skinny_kernel<MT, ODD, MOE>), dim3((unsigned)blocks, (unsigned)chunks),
                       dim3(kSkinnyWaves * 64), 0, stream, p, bpw, parts);
    return hipGetLastError();
}

// rows: how many rows a weight tile is likely to meet (dense: M)
template <bool ODD, bool MOE>
hipError_t launch_skinny(const GemmArgs &p, int64_t rows, hipStream_t stream) {
    const int64_t mt = skinny_mt(rows);
    const int64_t chunks = MOE ? 1 : (p.M + 16 * mt - 1) / (16 * mt);
    switch (mt) {
        case 1: return launch_skinny_mt<1, ODD, MOE>(p, chunks, stream);
        case 2: return launch_skinny_mt<2, ODD, MOE>(p, chunks, stream);
        case 3: return launch_skinny_mt<3, ODD, MOE>(p, chunks, stream);
        default: return launch_skinny_mt<4, ODD, MOE>(p, chunks, stream);
    }
}

// ---------------------------------------------------------------------------
// Tile order
// ---------------------------------------------------------------------------
//
// Dense: gemm_common.hpp's.  Grouped: the same order (an expert's m-tiles
// advance together along n, only the tiles that exist are spread over the
// XCDs), with the experts' segments looked up by lanes, 64 experts a step,
// where a walk over them one by one takes longer than a tile of a few K blocks
// (64 experts of 2048 x 1024, a row each, 128 x 64 tiles: 89 us against 24).

// One lane's expert of the 64 from e0: its segment [a, b), clamped to [0, R],
// its m-tiles of BM rows, and the sum of the m-tiles up to and with its own.
struct Segment {
    int32_t a, b;
    uint32_t tiles, upto;
};
template <int BM>
__device__ __forceinline__ Segment lane_segment(const GemmArgs &p, int32_t e0) {
    const int lane = threadIdx.x & 63;
    const int32_t e = e0 + lane, R = (int32_t)p.M;
    Segment s = {0, 0, 0u, 0u};
    if (e < p.E) {
        s.a = p.offsets[e];
        s.b = p.offsets[e + 1];
        s.a = s.a < 0 ? 0 : (s.a > R ? R : s.a);
        s.b = s.b < s.a ? s.a : (s.b > R ? R : s.b);
        s.tiles = ((uint32_t)(s.b - s.a) + BM - 1) / BM;
    }
    s.upto = s.tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t v = __shfl_up(s.upto, d);
        if (lane >= d) s.upto += v;
    }
    return s;
}

// The m-tiles that exist.
template <int BM>
__device__ __forceinline__ int64_t count_tiles_m(const GemmArgs &p) {
    int64_t n = 0;
    for (int32_t e0 = 0; e0 < p.E; e0 += 64) n += __builtin_amdgcn_readlane((int)lane_segment<BM>(p, e0).upto, 63);
    return n;
}

// Tile tid of the grouped order (tid below the number of tiles that exist,
// itself below 2^31).
template <int BN, int BM>
__device__ __forceinline__ bool grouped_tile(const GemmArgs &p, int64_t tid, Tile &t) {
    uint32_t rem = (uint32_t)tid;
    const uint32_t tn = (uint32_t)p.tiles_n;
    for (int32_t e0 = 0; e0 < p.E; e0 += 64) {
        const Segment s = lane_segment<BM>(p, e0);
        const uint64_t past = __ballot(s.upto * tn > rem);
        if (past == 0) {
            rem -= (uint32_t)__builtin_amdgcn_readlane((int)s.upto, 63) * tn;
            continue;
        }
        const int l = __builtin_ctzll(past);
        const uint32_t cnt = (uint32_t)__builtin_amdgcn_readlane((int)s.tiles, l);
        rem -= ((uint32_t)__builtin_amdgcn_readlane((int)s.upto, l) - cnt) * tn;
        const int64_t a = __builtin_amdgcn_readlane(s.a, l), b = __builtin_amdgcn_readlane(s.b, l);
        const uint32_t span = (uint32_t)kGroupMMoe * tn;
        const uint32_t group = rem / span;
        const uint32_t first = group * (uint32_t)kGroupMMoe;
        const uint32_t size = cnt - first < (uint32_t)kGroupMMoe ? cnt - first : (uint32_t)kGroupMMoe;
        const uint32_t in = rem - group * span;
        t.n0 = (int64_t)(in / size) * BN;
        t.m0 = a + (int64_t)(first + in % size) * BM;
        t.rows = b - t.m0 < BM ? b - t.m0 : BM;
        t.w = p.w + (int64_t)(e0 + l) * p.N * p.K;
        t.ws = p.ws + (int64_t)(e0 + l) * p.NB * p.KB;
        return true;
    }
    return false;
}

// This workgroup's tile; false where it has none.  TAIL: the tiles of a partial
// last round are split over K (see tail_plan).
template <int BN, int BM, bool MOE, int64_t GM, bool TAIL = false>
__device__ __forceinline__ bool my_tile(const GemmArgs &p, Tile &t) {
    if constexpr (!MOE) {
        return decode_tile<BN, BM, false, GM>(p, t);
    } else {
        const int64_t total = count_tiles_m<BM>(p) * p.tiles_n;
        int64_t whole = total;   // tiles spread over the XCDs
        if constexpr (TAIL) {
            const TailPlan tp = tail_plan(total, p.KB);
            if (tp.splits > 1) {
                whole = tp.full;
                if ((int64_t)blockIdx.x >= tp.full) {
                    const int64_t u = (int64_t)blockIdx.x - tp.full;
                    if (u >= tp.tail * tp.splits) return false;
                    t.split = (int32_t)(u % tp.splits);
                    t.nsplit = tp.splits;
                    t.unit = u;
                    return grouped_tile<BN, BM>(p, tp.full + u / tp.splits, t);
                }
            }
        }
        const int64_t xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
        const int64_t q = whole >> 3, r = whole & 7;
        if (slot >= q + (xcd < r ? 1 : 0)) return false;
        return grouped_tile<BN, BM>(p, xcd * q + (xcd < r ? xcd : r) + slot, t);
    }
}

// The tiles that my_tile split: their units' partial sums added in split order
// and rounded to bf16.  A fixed grid (the tail's size is only known on the
// device) whose waves take (tile, row) pairs in turn, 4 columns a lane.
constexpr int kTailReduceGroups = 512;
template <int BN, int BM>
__global__ __launch_bounds__(256) void moe_fp8_tail_reduce_kernel(GemmArgs p) {
    const TailPlan tp = tail_plan(count_tiles_m<BM>(p) * p.tiles_n, p.KB);
    if (tp.splits <= 1) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t pair = (int64_t)blockIdx.x * 4 + wave; pair < tp.tail * BM; pair += (int64_t)kTailReduceGroups * 4) {
        const int64_t i = pair / BM;
        const int r = (int)(pair - i * BM);
        Tile t;
        if (!grouped_tile<BN, BM>(p, tp.full + i, t) || r >= t.rows) continue;
        const float *slots = p.partial + i * tp.splits * (BM * BN) + (int64_t)r * BN;
        uint16_t *yrow = p.y + (t.m0 + r) * p.N;
        const int c = 4 * lane;
        const int64_t n = t.n0 + c;
        if (c >= BN || n >= p.N) continue;
        f32x4 acc = *reinterpret_cast<const f32x4 *>(slots + c);
        for (int32_t z = 1; z < tp.splits; ++z)
            acc += *reinterpret_cast<const f32x4 *>(slots + (int64_t)z * (BM * BN) + c);
        if (p.wide_store) {
            *reinterpret_cast<uint2 *>(yrow + n) =
                make_uint2(f32x2_to_bf16x2_bits(acc[0], acc[1]), f32x2_to_bf16x2_bits(acc[2], acc[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N) yrow[n + e] = (uint16_t)(f32x2_to_bf16x2_bits(acc[e], 0.0f) & 0xFFFFu);
        }
    }
}

// Buffer-to-LDS fills, 16 or 4 bytes a lane: lane i's value lands at lds + 16 i
// (4 i).  Written out as instructions: a ring is refilled while other parts of
// it are read, in an order that the kernels' waits count, and the compiler's own
// tracking would drain every fill at the end of each turn of a loop.  They have
// no result register, and the memory clobber keeps LDS reads on their side.
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(const BI8_LDS void *)p;
}
// (the range check covers off + soff, and knows no wrap)
__device__ __forceinline__ void fill16(i32x4 rsrc, uint32_t lds, uint32_t off, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "memory", "m0");
}
__device__ __forceinline__ void fill4(i32x4 rsrc, uint32_t lds, uint32_t off, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "memory", "m0");
}
// The words of make_rsrc's buffer resource, wave-uniform.
__device__ __forceinline__ i32x4 rsrc_words(const void *base, uint32_t num_bytes) {
    const uint64_t a = reinterpret_cast<uintptr_t>(base);
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xFFFF);
    r[2] = __builtin_amdgcn_readfirstlane((int)num_bytes);
    r[3] = 0x00020000;
    return r;
}

// 16 bytes at any byte, of which the first n are a row's (zeros behind them).
struct __attribute__((packed, aligned(1))) AnyPiece {
    i32x4 v;
};
__device__ __forceinline__ i32x4 load_piece(const int8_t *p, int64_t n) {
    if (n >= 16) return reinterpret_cast<const AnyPiece *>(p)->v;
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) v[i / 4] |= (int32_t)((uint32_t)(uint8_t)p[i] << (8 * (i % 4)));
    return v;
}

// Where a row's scale of block b of a batch of 8 lies among the row's 8: 32 rows'
// scales of one block in 32 banks.
__device__ __forceinline__ int scale_slot(int b, int row) { return b ^ ((row >> 2) & 7); }

// Wait until at most N buffer-to-LDS fills are in flight (63: any number) and
// every LDS read has returned.
template <int N>
__device__ __forceinline__ void wait_lds() {
    __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0x0 << 8) | ((N >> 4) << 14));
}

// ---------------------------------------------------------------------------
// Tiled path
// ---------------------------------------------------------------------------
//
// A workgroup of WN x WM waves computes a BN x BM tile (weight rows x
// activation rows), each wave SA x SB sub-tiles of 32 x 32.  K advances one
// block a step through a ring of NS stages in LDS, filled by buffer-to-LDS
// loads: rows of 128 bytes, their 16-byte pieces XOR-swizzled so that the
// fragment reads do not conflict.  Rows past the tile and pieces past K read as
// zero through the buffer range check, on both sides (a NaN code times zero
// would be NaN).
//
// These tiles serve grids that leave a workgroup alone on its CU, where nothing
// else fills its waits.  So a step reads the fragments of block kb + 1 into a
// second set of registers while the matrix core works on block kb, whose stage is
// refilled at once with block kb + NS; a sub-tile's sum is rescaled behind the
// next one's MFMAs.  One barrier a block.
// The activation scales reach LDS eight blocks at a time; the weight scale of
// a wave's 128-row block is a scalar load a block ahead.
//
// Bound by two things, in us a block of 128 x 64 (128 x 128) tiles: 0.30 (0.48) is
// one workgroup's own time on an idle chip, with 757 cycles near the sum of its
// MFMAs (256 a SIMD), fragment reads (273 of the LDS) and fills (24 KB, 192 at 128
// bytes a cycle).  The rest comes with the number of busy CUs, at the same clock,
// and so from the path of the fills that they share: nothing up to 64 CUs, 0.41
// (0.62) with 256 that share operands, 0.56 (0.70) with weights of their own.
// Measured (us): 128 x 64 333 x 5000 x 4000 21.9, 512 x 4096 x 4096 18.1; 128 x 128
// 1024 x 4096 x 4096 25.5, grouped 512 x 4096 x 14336 over 8 experts 97.
template <int WN_, int WM_, int SA_, int SB_, int NS_>
struct Cfg {
    static constexpr int WN = WN_, WM = WM_, SA = SA_, SB = SB_, NS = NS_;
    static constexpr int kWaves = WN * WM;
    static constexpr int kThreads = kWaves * 64;
    static constexpr int kWaveN = 32 * SA;
    static constexpr int kWaveM = 32 * SB;
    static constexpr int kBN = kWaveN * WN;
    static constexpr int kBM = kWaveM * WM;
    static constexpr int kXOff = kBN * 128;
    static constexpr int kStageBytes = kXOff + kBM * 128;
    static constexpr int kWLoads = kBN / 8 / kWaves;   // 1 KB pieces a wave loads
    static constexpr int kXLoads = kBM / 8 / kWaves;
    static constexpr int kLoads = kWLoads + kXLoads;
    static constexpr int kSB = 8;                      // K blocks in a batch of scales
    static constexpr int kScaleLoads = kBM * kSB / 64 / kWaves;
    static_assert(kBN % (8 * kWaves) == 0 && kBM % (8 * kWaves) == 0, "load split");
    static_assert(128 % kWaveN == 0, "a wave's weight rows lie in one scale block");
    static_assert(kScaleLoads >= 1 && kBM * kSB % (64 * kWaves) == 0, "scale split");
    static_assert(kWaves % 2 == 0, "a lane's pieces share their parity");
    static_assert(NS >= 3 && NS <= 4, "ring depth");
};

// LDS accesses of the wave's lanes stay on their sides of this.
__device__ __forceinline__ void wave_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// Store a workgroup's tile as bf16, the bias added: BN columns from t.n0, of which a
// wave's sums start at column col0 and tile row ml0.  32x32 result: lane -> token
// lane & 31; element i -> weight row 8 (i / 4) + 4 (lane / 32) + i % 4, so a lane
// has 4 columns together.  Stored from there, 8 bytes to 32 rows an instruction,
// the tiles of 256 rows took 7 to 9 % longer; by way of LDS whole lines go out (and
// rows of any N by stores of 16 bytes: N = 5001 47 -> 34 us at 1000 x 5001 x 4096).
// buf: 2 BN BM bytes, free once every wave is here.
template <int SA, int SB, int BN, int BM>
__device__ __forceinline__ void store_lines(const GemmArgs &p, const Tile &t, const float (&y)[SA][SB][16], char *buf,
                                            int col0, int ml0, int lane, int wave) {
    constexpr int kPieces = BN / 8;   // 16-byte pieces of a token's values
    const int rr = lane & 31, hi = lane >> 5;
    __syncthreads();   // every wave is past its last fragment read
#pragma unroll
    for (int b = 0; b < SB; ++b)
#pragma unroll
        for (int a = 0; a < SA; ++a)
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = y[a][b][4 * i4 + e];
                    asm volatile("" : "+v"(v[e]));   // (or the sums would be held as pairs all along, and spill)
                }
                if (p.bias) {
                    const int64_t n = t.n0 + col0 + 32 * a + 8 * i4 + 4 * hi;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < p.N) v[e] += bf16_bits_to_f32(p.bias[n + e]);
                }
                const int tok = ml0 + 32 * b + rr, piece = col0 / 8 + 4 * a + i4;
                // (tokens 16 to 31 with the halves of a piece exchanged: the 8 bytes of
                // 32 tokens lie in 64 banks)
                *reinterpret_cast<uint2 *>(buf + (tok * kPieces + (piece ^ (tok & 15))) * 16 + 8 * (hi ^ ((rr >> 4) & 1))) =
                    make_uint2(f32x2_to_bf16x2_bits(v[0], v[1]), f32x2_to_bf16x2_bits(v[2], v[3]));
            }
    __syncthreads();
    const bool wide = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15u) == 0;
    constexpr int kTokens = 512 / kPieces;   // tokens that the workgroup stores at once
#pragma unroll 4
    for (int j = 0; j < BM / kTokens; ++j) {
        const int tok = kTokens * j + (64 * wave + lane) / kPieces, c = lane & (kPieces - 1);
        u32x4 v = *reinterpret_cast<const u32x4 *>(buf + (tok * kPieces + (c ^ (tok & 15))) * 16);
        if (tok & 16) v = u32x4{v[2], v[3], v[0], v[1]};
        const int64_t n = t.n0 + 8 * c;
        if (tok >= t.rows || n >= p.N) continue;
        uint16_t *dst = p.y + (t.m0 + tok) * p.N + n;
        if (wide)
            *reinterpret_cast<u32x4 *>(dst) = v;
        else
            store_bf16x8(dst, v, p.N - n);
    }
}

// Epilogue of the gated w13 projection: the tile's gate and up columns become the
// 128 columns t.n0 and on of a = bf16(silu(gate) up), one quantisation group, and
// leave as codes and scales; gate, up and a are rounded to bf16 where the two
// launches that this replaces round them, so the results are theirs bit for bit
// wherever the sums are.
//
// Columns [col0, col0 + 32 SA) of token sub-tiles 0 and 1 (tile rows from ml0) are
// the gate values of one wave and the up values of another, together pair `pair`
// of four.  Both leave all of theirs in LDS as bf16 (after that no register of the
// sums is needed, where the kernel has none to spare), then the gate wave
// finishes sub-tile 0 and the up wave sub-tile 1.  A token's columns lie in lanes
// l and l ^ 32, and with SA = 2 in those of pair ^ 1 too.
// buf: 32 SA KB, tops: 256 words, both free once every wave is here.
//
// Measured, 8 experts of 28672 x 4096 (the two launches / this one, us): 512 rows
// 195 + 10 / 197, 8192 rows 1046 + 113 / 1024.
template <int SA>
__device__ __forceinline__ void gate_store(const GemmArgs &p, const Tile &t, const float (&y)[SA][2][16], char *buf,
                                           uint32_t *tops, int pair, bool gate, int col0, int ml0, int lane) {
    constexpr int kSub = SA * 2048;     // a sub-tile's values of one wave
    constexpr int kPieces = SA * 2;     // 16-byte pieces of a token's 32 SA codes
    const int rr = lane & 31, hi = lane >> 5;
    __syncthreads();   // every wave is past its last fragment read
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int c = 0; c < 2 * SA; ++c) {
            float v[8];
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = y[c >> 1][b][8 * (c & 1) + i];
                asm volatile("" : "+v"(v[i]));   // (or the sums would be held as pairs all along, and spill)
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = f32x2_to_bf16x2_bits(v[2 * j], v[2 * j + 1]);
            *reinterpret_cast<u32x4 *>(buf + (4 * pair + (gate ? 0 : 2) + b) * kSub + c * 1024 + lane * 16) = o;
        }
    __syncthreads();
    const int b = gate ? 0 : 1;
    char *gates = buf + (4 * pair + b) * kSub;
    const char *ups = gates + 2 * kSub;
    u32x4 gv[2 * SA], av[2 * SA];
    float gmin = 0.0f;
#pragma unroll
    for (int c = 0; c < 2 * SA; ++c) {
        gv[c] = *reinterpret_cast<const u32x4 *>(gates + c * 1024 + lane * 16);
        av[c] = *reinterpret_cast<const u32x4 *>(ups + c * 1024 + lane * 16);
        float f[8];
        unpack_bf16x8(gv[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) gmin = fminf(gmin, f[i]);
    }
    // (silu_times takes another form for far negative gates: in a wave that has one)
    const bool far = __any(gmin < -80.0f);
    u32x4 top4 = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int c = 0; c < 2 * SA; ++c) {
        float g[8], u[8], a[8];
        unpack_bf16x8(gv[c], g);
        unpack_bf16x8(av[c], u);
        if (far) {
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = silu_times(g[i], u[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = silu_near(g[i], u[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            av[c][j] = f32x2_to_bf16x2_bits(a[2 * j], a[2 * j + 1]);
            top4[j] = umax<true>(top4[j], av[c][j] & 0x7FFF7FFFu);
        }
    }
    uint32_t top = umax<true>(umax<true>(top4[0], top4[1]), umax<true>(top4[2], top4[3]));
    top = umax<true>(top, (uint32_t)__shfl_xor((int)top, 32));
    if constexpr (SA == 2) {
        if (hi == 0) tops[(2 * pair + b) * 32 + rr] = top;
        __syncthreads();
        top = umax<true>(top, tops[(2 * (pair ^ 1) + b) * 32 + rr]);
    }
    const float sc = bf16_bits_to_f32(umax<false>(top & 0xFFFFu, top >> 16)) / E4m3Codes::kMax;
    // codes to LDS, over the gate values, a token a row of 32 SA bytes (pieces
    // swizzled by the token), and out in whole pieces; a wave's LDS accesses run in
    // order
    wave_order();
#pragma unroll
    for (int c = 0; c < 2 * SA; ++c) {
        float f[8];
        uint32_t lo, up;
        unpack_bf16x8(av[c], f);
        E4m3Codes::encode(f, sc, lo, up);
        char *row = gates + rr * (kPieces * 16) + (c ^ (rr & (kPieces - 1))) * 16 + 4 * hi;
        *reinterpret_cast<uint32_t *>(row) = lo;       // columns 16 c + 4 hi
        *reinterpret_cast<uint32_t *>(row + 8) = up;   // columns 16 c + 8 + 4 hi
    }
    wave_order();
    const int64_t ml = ml0 + 32 * b;
    if (hi == 0 && col0 == 0 && ml + rr < t.rows) p.as[(t.m0 + ml + rr) * (p.I / kBlock) + t.n0 / kBlock] = sc;
    constexpr int kTokens = 64 / kPieces;   // tokens that a store covers
#pragma unroll
    for (int j = 0; j < 32 / kTokens; ++j) {
        const int tok = kTokens * j + lane / kPieces, c = lane & (kPieces - 1);
        const i32x4 v =
            *reinterpret_cast<const i32x4 *>(gates + tok * (kPieces * 16) + (c ^ (tok & (kPieces - 1))) * 16);
        if (ml + tok < t.rows)
            *reinterpret_cast<i32x4 *>(p.aq + (t.m0 + ml + tok) * p.I + t.n0 + col0 + 16 * c) = v;
    }
}

// SPLIT: a workgroup sums only a run of K blocks and stores fp32 partial sums:
// dense, run blockIdx.y of kb_per_split blocks, in p.partial[blockIdx.y];
// grouped, the tiles of a partial last round (see tail_plan).
// ODD (dense, whole): K % 16 != 0, rows start at any byte.  Pieces then pass
// through registers, a block ahead of their stage, by loads at any byte; the
// piece that holds the end of a row is put together from its bytes.
template <class C, bool MOE, bool SPLIT, int64_t GM, bool ODD = false>
__global__ __launch_bounds__(C::kThreads) void gemm_fp8_tiled_kernel(GemmArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int SA = C::SA, SB = C::SB, NS = C::NS;
    __shared__ __attribute__((aligned(1024))) char lds[NS * C::kStageBytes];
    __shared__ float xsl[2][C::kBM * C::kSB];

    Tile t;
    if (!my_tile<C::kBN, C::kBM, MOE, GM, MOE && SPLIT>(p, t)) return;
    if (t.rows <= 0 || t.n0 >= p.N) return;   // (the latter: offsets that are not in order)

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t K = p.K;
    int64_t kb0 = 0, KB = p.KB;   // this workgroup's K blocks: [kb0, kb0 + KB)
    if constexpr (SPLIT && !MOE) {
        kb0 = (int64_t)blockIdx.y * p.kb_per_split;
        KB = p.KB - kb0 < p.kb_per_split ? p.KB - kb0 : p.kb_per_split;
    }
    if constexpr (SPLIT && MOE) {
        if (t.split >= 0) {
            const int64_t per = (p.KB + t.nsplit - 1) / t.nsplit;
            kb0 = (int64_t)t.split * per;
            KB = p.KB - kb0 < per ? p.KB - kb0 : per;
        }
    }

    // (ranges of at most 2^31 bytes: 256 rows of K <= 2^23)
    const int64_t wrows = p.N - t.n0 < C::kBN ? p.N - t.n0 : C::kBN;
    const i32x4 wr = rsrc_words(t.w + t.n0 * K, clamp_bytes(wrows * K));
    const i32x4 xr = rsrc_words(p.xq + t.m0 * K, clamp_bytes(t.rows * K));
    const i32x4 sr = rsrc_words(p.xs + t.m0 * p.KB, clamp_bytes(t.rows * p.KB * 4));

    // Piece q (1 KB) covers tile rows [8q, 8q + 8): lane i lands at row 8q + i/8,
    // 16-byte slot i % 8, which holds K piece slot ^ swz(row), swz(r) = (r & 7) ^
    // ((r >> 3) & 1).  A wave's pieces q = wave + j kWaves share their parity,
    // so a lane's K piece is the same in all of them.
    const int r_in = lane >> 3;
    const int chunk = 16 * ((lane & 7) ^ r_in ^ (wave & 1));
    const int nkb = (int)KB;
    uint32_t off = (uint32_t)((8 * wave + r_in) * K + kb0 * kBlock + chunk);
    const uint32_t piece_stride = (uint32_t)(8 * C::kWaves * K);
    // the lane's piece lies inside K and the run in blocks kb < kb_in
    const int kb_in = min((int)((K - chunk + kBlock - 1) / kBlock - kb0), nkb);
    const uint32_t wlds = lds_address(lds) + wave * 1024, xlds = wlds + C::kXOff;
    const uint32_t slds = lds_address(xsl) + wave * C::kScaleLoads * 256;
    // Entry (row, block) of a batch of scales at row * kSB + scale_slot(block, row);
    // entries past the last block are the next row's, or zero: unused.
    auto fill_scales = [&](int kb) __attribute__((always_inline)) {
        const uint32_t dst = slds + ((kb / C::kSB) & 1) * (C::kBM * C::kSB * 4);
        const int f = wave * C::kScaleLoads * 64 + lane;
        const int row = f / C::kSB, slot = f & (C::kSB - 1);
#pragma unroll
        for (int j = 0; j < C::kScaleLoads; ++j)
            fill4(sr, dst + j * 256, (uint32_t)((row * p.KB + kb0 + scale_slot(slot, row + 8 * j)) * 4),
                  (uint32_t)(kb * 4 + j * 8 * 4 * (int)p.KB));
    };
    i32x4 held[ODD ? C::kLoads : 1];   // ODD: the wave's pieces of the block that is next to be stored
    auto take = [&](int kb) __attribute__((always_inline)) {
        const int64_t k = (int64_t)kb * kBlock + chunk;
#pragma unroll
        for (int j = 0; j < C::kLoads; ++j) {
            const bool weight = j < C::kWLoads;
            const int row = 8 * (wave + (weight ? j : j - C::kWLoads) * C::kWaves) + r_in;
            const int8_t *src = (weight ? t.w + (t.n0 + row) * K : p.xq + (t.m0 + row) * K) + k;
            held[j] = load_piece(src, row < (weight ? wrows : t.rows) ? K - k : 0);
        }
    };
    auto keep = [&](const int st) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < C::kLoads; ++j) {
            const bool weight = j < C::kWLoads;
            const int q = wave + (weight ? j : j - C::kWLoads) * C::kWaves;
            *reinterpret_cast<i32x4 *>(lds + st * C::kStageBytes + (weight ? 0 : C::kXOff) + q * 1024 + lane * 16) =
                held[j];
        }
    };
    auto fill = [&](const int st, int kb) __attribute__((always_inline)) {
        if (__builtin_expect((kb & (C::kSB - 1)) == 0, 0)) fill_scales(kb);
        if constexpr (ODD) {
            keep(st);
            take(kb + 1);
            return;
        }
        off = kb < kb_in ? off : kOobOffset;   // out of range for good
#pragma unroll
        for (int j = 0; j < C::kWLoads; ++j)
            fill16(wr, wlds + st * C::kStageBytes + j * (C::kWaves * 1024), off, j * piece_stride + (uint32_t)kb * kBlock);
#pragma unroll
        for (int j = 0; j < C::kXLoads; ++j)
            fill16(xr, xlds + st * C::kStageBytes + j * (C::kWaves * 1024), off, j * piece_stride + (uint32_t)kb * kBlock);
    };

    const int wn = wave % C::WN, wm = wave / C::WN;
    const int rr = lane & 31, hi = lane >> 5;
    const int swz = (rr & 7) ^ ((rr >> 3) & 1);
    int wfrag[4], xfrag[4];   // fragment addresses of sub-tile 0, stage 0
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int piece = 16 * ((2 * s + hi) ^ swz);
        wfrag[s] = (wn * C::kWaveN + rr) * 128 + piece;
        xfrag[s] = C::kXOff + (wm * C::kWaveM + rr) * 128 + piece;
    }
    const int srow = (wm * C::kWaveM + rr) * C::kSB;

    int64_t nbw = (t.n0 + wn * C::kWaveN) / kBlock;
    if (nbw > p.NB - 1) nbw = p.NB - 1;
    const BI8_CONST float *ws_row =
        reinterpret_cast<const BI8_CONST float *>(reinterpret_cast<uintptr_t>(t.ws + nbw * p.KB + kb0));
    float ws_cur = ws_row[0];

    f32x16 zero16;
#pragma unroll
    for (int i = 0; i < 16; ++i) zero16[i] = 0.f;
    f32x16 acc[2];
    float y[SA][SB][16];   // (single registers: vectors of 16 would need room to be moved)
#pragma unroll
    for (int a = 0; a < SA; ++a)
#pragma unroll
        for (int b = 0; b < SB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) y[a][b][i] = 0.f;
    acc[0] = acc[1] = zero16;

    auto rescale = [&](const int j, float tb) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[j / SB][j % SB][i] = fmaf(acc[j & 1][i], tb, y[j / SB][j % SB][i]);
        // (a use here keeps the rescales where they are)
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("" ::"v"(y[j / SB][j % SB][i]));
    };

    // two sets of fragments and scales: blocks of even and of odd index
    i32x4 wf[2][SA][4], xf[2][SB][4];
    float xsv[2][SB], wsv[2], tlast = 0.f;
    auto read = [&](const int st, const int set, int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < SA; ++a)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                wf[set][a][s] = *reinterpret_cast<const i32x4 *>(lds + wfrag[s] + (st * C::kStageBytes + a * 4096));
#pragma unroll
        for (int b = 0; b < SB; ++b)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                xf[set][b][s] = *reinterpret_cast<const i32x4 *>(lds + xfrag[s] + (st * C::kStageBytes + b * 4096));
#pragma unroll
        for (int b = 0; b < SB; ++b)
            xsv[set][b] = xsl[(kb / C::kSB) & 1][srow + b * 32 * C::kSB + scale_slot(kb & (C::kSB - 1), rr)];
        wsv[set] = ws_cur;
        ws_cur = ws_row[kb + 1 < nkb ? kb + 1 : nkb - 1];
    };
    constexpr int kSub = SA * SB;
    // Block kb, whose fragments are in set `set` and whose stage is st.  Before
    // the barrier this wave's reads of the stage have returned and its fills of
    // block kb + 1 have landed (NS - 2 blocks may still be on their way; a batch
    // of scales among them only makes the wait stricter).
    auto step = [&](auto stc, auto setc, int kb) __attribute__((always_inline)) {
        constexpr int st = decltype(stc)::value, set = decltype(setc)::value;
        // (ODD: the block's pieces were stored a step ago or more, and the loads that
        // a store waits for are younger than a batch of scales before them)
        wait_lds<ODD ? 63 : (NS - 2) * C::kLoads>();
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        read((st + 1) % NS, set ^ 1, kb + 1);   // (past the last block: read and not used)
        fill(st, kb + NS);
        __builtin_amdgcn_sched_barrier(0);
        float tb[SB];
#pragma unroll
        for (int b = 0; b < SB; ++b) tb[b] = xsv[set][b] * wsv[set];
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
            const i32x4(&w)[4] = wf[set][j / SB], (&x)[4] = xf[set][j % SB];
            // (one sub-tile: two accumulators in turn from block to block)
            constexpr int flip = kSub == 1 ? set : 0;
            f32x16 &c = acc[(j + flip) & 1];
            c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(w[0], w[1]), join16(x[0], x[1]), zero16, 0, 0,
                                                                0, 0, 0, 0);
            c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(w[2], w[3]), join16(x[2], x[3]), c, 0, 0, 0, 0,
                                                                0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (kSub == 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i) y[0][0][i] = fmaf(acc[flip ^ 1][i], tlast, y[0][0][i]);
            } else if (j > 0) {
                rescale(j - 1, tb[(j - 1) % SB]);
            } else {
                rescale(kSub - 1, tlast);   // the previous block's last sub-tile
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        tlast = tb[SB - 1];
        asm volatile("" : "+v"(acc[0]), "+v"(acc[1]));
    };

    if constexpr (ODD) take(0);
#pragma unroll
    for (int i = 0; i < NS; ++i) fill(i, i);
    wait_lds<ODD ? 0 : (NS - 1) * C::kLoads>();
    lds_barrier();
    read(0, 0, 0);
    constexpr int kTurn = NS % 2 ? 2 * NS : NS;   // steps until stage and set are back
    int kb = 0;
    auto turn = [&](auto self, auto ic) __attribute__((always_inline)) -> void {
        constexpr int i = decltype(ic)::value;
        if constexpr (i < kTurn) {
            step(std::integral_constant<int, i % NS>{}, std::integral_constant<int, i % 2>{}, kb);
            if (++kb < nkb) self(self, std::integral_constant<int, i + 1>{});
        }
    };
    while (kb < nkb) turn(turn, std::integral_constant<int, 0>{});
    if constexpr (kSub == 1) {
        const int last = (nkb - 1) & 1;
#pragma unroll
        for (int i = 0; i < 16; ++i) y[0][0][i] = fmaf(last ? acc[1][i] : acc[0][i], tlast, y[0][0][i]);
    } else {
        rescale(kSub - 1, tlast);
    }
    wait_vmcnt<0>();   // no LDS fill may outlive the workgroup

    // Store.  32x32 result: lane -> token lane & 31; element i -> weight row
    // 8 (i / 4) + 4 hi + i % 4.
    if constexpr (SPLIT) {
        bool whole = false;
        float *rows;      // fp32 rows of this unit's partial sums, at tile row 0
        int64_t pitch, ncols, nrows;
        if constexpr (MOE) {
            whole = t.split < 0;
            rows = p.partial + t.unit * (int64_t)(C::kBM * C::kBN);
            pitch = C::kBN;
            ncols = C::kBN;
            nrows = C::kBM;
        } else {
            rows = p.partial + (int64_t)blockIdx.y * p.M * p.N + t.m0 * p.N + t.n0;
            pitch = p.N;
            ncols = p.N - t.n0;
            nrows = t.rows;
        }
        if (!whole) {
#pragma unroll
            for (int b = 0; b < SB; ++b) {
                const int64_t ml = wm * C::kWaveM + b * 32 + rr;
                if (ml >= nrows) continue;
#pragma unroll
                for (int a = 0; a < SA; ++a)
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) {
                        const int64_t c = wn * C::kWaveN + a * 32 + 8 * i4 + 4 * hi;
                        float *dst = rows + ml * pitch + c;
                        if (MOE || p.wide_store) {
                            if (c < ncols)
                                *reinterpret_cast<f32x4 *>(dst) = f32x4{y[a][b][4 * i4], y[a][b][4 * i4 + 1],
                                                                         y[a][b][4 * i4 + 2], y[a][b][4 * i4 + 3]};
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (c + e < ncols) dst[e] = y[a][b][4 * i4 + e];
                        }
                    }
            }
            return;
        }
    }
    store_lines<SA, SB, C::kBN, C::kBM>(p, t, y, lds, wn * C::kWaveN, wm * C::kWaveM, lane, wave);
#endif  // __HIP_DEVICE_COMPILE__
}

// ---------------------------------------------------------------------------
// Ping-pong path: 256 x 256 tile
// ---------------------------------------------------------------------------
//
// Eight waves of 128 weight rows x 64 activation rows.  Waves w and w + 4 share
// a SIMD and belong to two groups that run half a step apart: between two
// barriers one group issues the four MFMAs of a cluster (one 32-row weight
// sub-row against its two 32-row activation sub-rows), the other reads the
// fragments of its next cluster, issues fills and rescales its previous
// cluster.  A K block is four clusters, eight barriers.
//
// The two stages of 64 KB are refilled piecewise: the activation rows of block
// kb + 2 as soon as both groups have read those of kb into registers, the
// weight sub-rows a cluster or two after they were read, so that fills run
// between one and two blocks ahead and no wait drains them.
//
// Bound by the matrix core at the clock that the power cap leaves: 2048 x 28672 x
// 4096 227 us, 2120 TFLOP/s, the matrix core busy 68 % of the time at 1.8 GHz (of
// 2.4); 8192^3 445 us; grouped, 8192 rows over 8 experts of 28672 x 4096 971 us.
// Of a tile's 57 us at K = 4096 about 4 go on its first fills and 4 on its stores.
// (A workgroup that walked several tiles, filling the next one's first blocks
// during the last of the one before, lost more on the bookkeeping in its
// loop: 8192^3 488 us, 2048 x 28672 x 4096 245.)
struct PingPong {
    static constexpr int kThreads = 512;
    static constexpr int kBN = 256, kBM = 256, SA = 4, SB = 2;
    static constexpr int kSB = 8;
    static constexpr int kScaleLoads = kBM * kSB / 64 / 8;
};

// SILU: the grouped w13 projection with the gating and the quantisation as its
// epilogue (see gate_store): tile rows [0, 128) are gate rows t.n0 and on, [128,
// 256) the up rows of the same columns.
template <bool MOE, int64_t GM, bool SILU = false>
__global__ __launch_bounds__(512) void gemm_fp8_pingpong_kernel(GemmArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
    using C = PingPong;
    constexpr int SA = C::SA, SB = C::SB;
    // weight stages 0, 1 (row 128 g + 32 a + i: group g, sub-row a), then
    // activation stages 0, 1
    constexpr int kStage = 32768, kX = 2 * kStage;
    __shared__ __attribute__((aligned(1024))) char lds[4 * kStage];
    __shared__ float xsl[2][C::kBM * C::kSB];

    Tile t;
    static_assert(!SILU || MOE, "the gated epilogue is the grouped w13 projection's");
    if (!my_tile<SILU ? C::kBN / 2 : C::kBN, C::kBM, MOE, GM>(p, t)) return;
    if (t.rows <= 0 || t.n0 >= (SILU ? p.I : p.N)) return;   // (the latter: offsets that are not in order)

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave >> 2, wm = wave & 3;
    const int64_t K = p.K;
    const int nkb = (int)p.KB;

    // (SILU: of the wave's own half, the one whose rows it fills)
    const int64_t wrows = SILU ? C::kBN / 2 : (p.N - t.n0 < C::kBN ? p.N - t.n0 : C::kBN);
    const i32x4 wr = rsrc_words(t.w + (SILU ? wn * p.I + t.n0 : t.n0) * K, clamp_bytes(wrows * K));
    const i32x4 xr = rsrc_words(p.xq + t.m0 * K, clamp_bytes(t.rows * K));
    const i32x4 sr = rsrc_words(p.xs + t.m0 * p.KB, clamp_bytes(t.rows * p.KB * 4));

    // Pieces of 1 KB as in the tiled kernel.  A wave fills, of weight sub-row a,
    // rows 128 wn + 32 a + 8 wm + [0, 8), and activation rows 8 (wave + 8 j).
    const int r_in = lane >> 3;
    const int chunk = 16 * ((lane & 7) ^ r_in ^ (wave & 1));
    const uint32_t wgo = (uint32_t)(((SILU ? 0 : 128 * wn) + 8 * wm + r_in) * K + chunk);
    const uint32_t xgo = (uint32_t)((8 * wave + r_in) * K + chunk);
    const uint32_t wstride = (uint32_t)(32 * K), xstride = (uint32_t)(64 * K);
    const int kb_in = (int)((K - chunk + kBlock - 1) / kBlock);
    const uint32_t lds0 = lds_address(lds);
    const uint32_t wlds = lds0 + wn * 16384 + wm * 1024, xlds = lds0 + kX + wave * 1024;
    const uint32_t slds = lds_address(xsl) + wave * C::kScaleLoads * 256;
    // the lane's offsets: out of range for good once its piece lies past K
    uint32_t wv = wgo, xv = xgo;
    auto aim = [&](int kb) __attribute__((always_inline)) {
        wv = kb < kb_in ? wv : kOobOffset;
        xv = kb < kb_in ? xv : kOobOffset;
    };
    // (st: the stage, kb & 1; wv and xv aimed at kb)
    auto fill_w = [&](const int st, const int a, int kb) __attribute__((always_inline)) {
        fill16(wr, wlds + st * kStage + a * 4096, wv, a * wstride + (uint32_t)kb * kBlock);
    };
    auto fill_x = [&](const int st, const int j, int kb) __attribute__((always_inline)) {
        fill16(xr, xlds + st * kStage + j * 8192, xv, j * xstride + (uint32_t)kb * kBlock);
    };
    // Entry (row, block) of a batch at row * kSB + scale_slot(block, row); entries
    // past the last block are the next row's, or zero: unused.
    auto fill_scales = [&](int kb) __attribute__((always_inline)) {
        const uint32_t dst = slds + ((kb / C::kSB) & 1) * (C::kBM * C::kSB * 4);
        const int f = wave * C::kScaleLoads * 64 + lane;
        const int row = f / C::kSB, slot = f & (C::kSB - 1);
#pragma unroll
        for (int j = 0; j < C::kScaleLoads; ++j)
            fill4(sr, dst + j * 256, (uint32_t)((row * p.KB + scale_slot(slot, row + 8 * j)) * 4),
                  (uint32_t)(kb * 4 + j * 8 * 4 * (int)p.KB));
    };

    const int rr = lane & 31, hi = lane >> 5;
    const int swz = (rr & 7) ^ ((rr >> 3) & 1);
    int wfrag[4], xfrag[4];   // fragment addresses of sub-row 0, stage 0
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int piece = 16 * ((2 * s + hi) ^ swz);
        wfrag[s] = (wn * 128 + rr) * 128 + piece;
        xfrag[s] = kX + (wm * 64 + rr) * 128 + piece;
    }
    const int srow = (wm * 64 + rr) * C::kSB;

    int64_t nbw = (SILU ? t.n0 + wn * p.I : t.n0 + 128 * wn) / kBlock;
    if (nbw > p.NB - 1) nbw = p.NB - 1;
    const BI8_CONST float *ws_row =
        reinterpret_cast<const BI8_CONST float *>(reinterpret_cast<uintptr_t>(t.ws + nbw * p.KB));
    float ws_cur = ws_row[0];

    f32x16 zero16;
#pragma unroll
    for (int i = 0; i < 16; ++i) zero16[i] = 0.f;
    f32x16 acc[SB];
    float y[SA][SB][16];   // (single registers: vectors of 16 would need room to be moved)
    float tb[SB], xsv[SB], wsv = 0.f;
#pragma unroll
    for (int b = 0; b < SB; ++b) {
        acc[b] = zero16;
        tb[b] = 0.f;
#pragma unroll
        for (int a = 0; a < SA; ++a)
#pragma unroll
            for (int i = 0; i < 16; ++i) y[a][b][i] = 0.f;
    }
    // activation fragments: sub-row 0 of even and of odd blocks, sub-row 1
    i32x4 xf[3][4], wf[4];
    auto read_x = [&](i32x4 (&f)[4], const int st, const int b) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            f[s] = *reinterpret_cast<const i32x4 *>(lds + xfrag[s] + (st * kStage + b * 4096));
    };

    // elements [i0, i0 + n) of sub-tile (a, b)
    auto rescale = [&](const int a, const int b, const int i0, const int n) __attribute__((always_inline)) {
#pragma unroll
        for (int i = i0; i < i0 + n; ++i) y[a][b][i] = fmaf(acc[b][i], tb[b], y[a][b][i]);
#pragma unroll
        for (int i = i0; i < i0 + n; ++i) asm volatile("" ::"v"(y[a][b][i]));
    };
    // Memory phase of cluster a of block kb, in stage st.  It reads the weight
    // fragments of its cluster and, of the activations, sub-row 1 in a = 0 and
    // the next block's sub-row 0 in a = 3: 8, 4, 4, 8 reads.  Fills, in this order
    // from block to block:
    //   a = 1: activation pieces 0, 1 of kb + 2    a = 2: pieces 2, 3
    //   a = 3: weight sub-rows 0, 1 of kb + 2      a = 0: sub-rows 2, 3 of kb + 1
    // The waits leave the younger fills in flight (a batch of scales among
    // them only makes a wait stricter).
    auto memory = [&](auto ac, auto sc, int kb) __attribute__((always_inline)) {
        constexpr int a = decltype(ac)::value, st = decltype(sc)::value;
#pragma unroll
        for (int s = 0; s < 4; ++s) wf[s] = *reinterpret_cast<const i32x4 *>(lds + wfrag[s] + (st * kStage + a * 4096));
        if constexpr (a == 0) {
            read_x(xf[2], st, 1);
#pragma unroll
            for (int b = 0; b < SB; ++b)
                xsv[b] = xsl[(kb / C::kSB) & 1][srow + b * 32 * C::kSB + scale_slot(kb & (C::kSB - 1), rr)];
            wsv = ws_cur;
            ws_cur = ws_row[kb + 1 < nkb ? kb + 1 : nkb - 1];
            if (__builtin_expect(((kb + 2) & (C::kSB - 1)) == 0, 0)) fill_scales(kb + 2);
            fill_w(st ^ 1, 2, kb + 1);
            fill_w(st ^ 1, 3, kb + 1);
        } else if constexpr (a == 1) {
            aim(kb + 2);
            fill_x(st, 0, kb + 2);
            fill_x(st, 1, kb + 2);
        } else if constexpr (a == 2) {
            fill_x(st, 2, kb + 2);
            fill_x(st, 3, kb + 2);
        } else {
            read_x(xf[st ^ 1], st ^ 1, 0);
            fill_w(st, 0, kb + 2);
            fill_w(st, 1, kb + 2);
        }
        __builtin_amdgcn_sched_barrier(0);
        rescale((a + 3) % 4, 0, 0, 16);
        if constexpr (a == 1)
            wait_lds<10>();   // weight sub-rows 2, 3 of this block are in
        else if constexpr (a == 2)
            wait_lds<8>();    // the activation rows of the next block
        else if constexpr (a == 3)
            wait_lds<8>();    // weight sub-rows 0, 1 of the next block
        else
            wait_lds<63>();
        __builtin_amdgcn_sched_barrier(0);
    };
    // Math phase: the cluster's MFMAs, and between them the rescale of the
    // previous cluster's second sub-tile (that of the first runs in the memory
    // phase): each wave's vector work is spread over both phases, and neither
    // waits for an MFMA that has just been issued.
    auto math = [&](auto ac, auto sc) __attribute__((always_inline)) {
        constexpr int a = decltype(ac)::value, before = (a + 3) % 4, x0 = decltype(sc)::value;
        acc[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(wf[0], wf[1]), join16(xf[x0][0], xf[x0][1]),
                                                                 zero16, 0, 0, 0, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        rescale(before, 1, 0, 8);
        __builtin_amdgcn_sched_barrier(0);
        acc[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(wf[2], wf[3]), join16(xf[x0][2], xf[x0][3]),
                                                                 acc[0], 0, 0, 0, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        rescale(before, 1, 8, 8);
        if constexpr (a == 0) {
#pragma unroll
            for (int b = 0; b < SB; ++b) tb[b] = xsv[b] * wsv;
        }
        __builtin_amdgcn_sched_barrier(0);
        acc[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(wf[0], wf[1]), join16(xf[2][0], xf[2][1]),
                                                                 zero16, 0, 0, 0, 0, 0, 0);
        acc[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(wf[2], wf[3]), join16(xf[2][2], xf[2][3]),
                                                                 acc[1], 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int b = 0; b < SB; ++b) asm volatile("" : "+v"(acc[b]));
    };
    auto cluster = [&](auto ac, auto sc, int kb) __attribute__((always_inline)) {
        memory(ac, sc, kb);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        math(ac, sc);
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    auto block = [&](auto sc, int kb) __attribute__((always_inline)) {
        cluster(std::integral_constant<int, 0>{}, sc, kb);
        cluster(std::integral_constant<int, 1>{}, sc, kb);
        cluster(std::integral_constant<int, 2>{}, sc, kb);
        cluster(std::integral_constant<int, 3>{}, sc, kb);
    };
    fill_scales(0);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
        aim(st);
#pragma unroll
        for (int j = 0; j < 4; ++j) fill_x(st, j, st);
#pragma unroll
        for (int a = 0; a < (st ? 2 : 4); ++a) fill_w(st, a, st);
    }
    wait_lds<8>();
    lds_barrier();
    read_x(xf[0], 0, 0);
    if (wn == 1) lds_barrier();   // group 1 runs one phase behind
    for (int kb = 0;;) {
        block(std::integral_constant<int, 0>{}, kb);
        if (++kb >= nkb) break;
        block(std::integral_constant<int, 1>{}, kb);
        if (++kb >= nkb) break;
    }
    if (wn == 0) lds_barrier();
    rescale(3, 0, 0, 16);
    rescale(3, 1, 0, 16);
    wait_vmcnt<0>();   // no LDS fill may outlive the workgroup

    if constexpr (SILU)
        gate_store<SA>(p, t, y, lds, reinterpret_cast<uint32_t *>(xsl), wm, wn == 0, 0, wm * 64, lane);
    else
        store_lines<SA, SB, C::kBN, C::kBM>(p, t, y, lds, wn * 128, wm * 64, lane, wave);
#endif  // __HIP_DEVICE_COMPILE__
}

// The same for 256 x 128 tiles, where 256 x 256 would leave CUs without a tile or
// pad short segments: waves of 64 weight rows x 64 activation rows, group g
// owning activation rows 64 g, a block of two clusters, and three whole stages
// of 48 KB.  Measured: 2048 x 4096 x 14336 117 us, 2060 TFLOP/s; grouped, 512 rows
// over 8 experts of 28672 x 4096 192 us, there bound by the weight's stream (949 MB
// by the counters, 4.9 TB/s).
struct PingPong128 {
    static constexpr int kThreads = 512;
    static constexpr int kBN = 256, kBM = 128, SA = 2, SB = 2;
    static constexpr int kSB = 8;
    static constexpr int kScaleLoads = kBM * kSB / 64 / 8;
};

// WIDE: the codes converted to f16 (exactly: 4 significant bits, 2^-9 to 448) and
// multiplied by f16 MFMAs, whose sums of products binary32 holds without the cut, at
// half the matrix rate: for callers that quantise the result again, where a sum on
// the other side of a rounding moves a code by a whole step.  A cluster's weight
// fragment is converted chunk by chunk between its MFMAs, the activations once a
// block, in the memory phase, where the whole rescale then stands too.
// Bound by MFMAs (2048 cycles a block) and vector work that overlap in part, 1.4 us a
// block on an idle chip, and by the power cap with all CUs busy: 1.65 us, with or
// without the conversions.
// Measured (this / the f8 kernel, us): grouped, 8 experts of 28672 x 4096 with 12 to
// 24 rows 185 / 179, 25 to 45 196 / 185, 54 to 79 231 / 189, 1024 each 1705 / 1065;
// 2048 x 4096 x 14336 203 / 123.
template <bool MOE, int64_t GM, bool SILU = false, bool WIDE = false>
__global__ __launch_bounds__(512) void gemm_fp8_pingpong128_kernel(GemmArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
    using C = PingPong128;
    constexpr int SA = C::SA, SB = C::SB;
    // a stage: weight row 64 q + 32 a + i (quarter q, sub-row a), then activation rows
    constexpr int kStage = (C::kBN + C::kBM) * 128, kX = C::kBN * 128;
    __shared__ __attribute__((aligned(1024))) char lds[3 * kStage];
    __shared__ float xsl[2][C::kBM * C::kSB];

    Tile t;
    static_assert(!SILU || MOE, "the gated epilogue is the grouped w13 projection's");
    if (!my_tile<SILU ? C::kBN / 2 : C::kBN, C::kBM, MOE, GM>(p, t)) return;
    if (t.rows <= 0 || t.n0 >= (SILU ? p.I : p.N)) return;   // (the latter: offsets that are not in order)

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = wave >> 2, quarter = wave & 3;
    // WIDE, where the f16 MFMAs set the clock: none for sub-rows that have no rows (a
    // group without any only fills and keeps the barriers)
    const bool busy = 64 * group < t.rows, both = 64 * group + 32 < t.rows;
    const int64_t K = p.K;
    const int nkb = (int)p.KB;

    const int64_t wrows = SILU ? C::kBN / 2 : (p.N - t.n0 < C::kBN ? p.N - t.n0 : C::kBN);
    const i32x4 wr = rsrc_words(t.w + t.n0 * K, clamp_bytes(wrows * K));
    const i32x4 wr_up = SILU ? rsrc_words(t.w + (p.I + t.n0) * K, clamp_bytes(wrows * K)) : wr;
    const i32x4 xr = rsrc_words(p.xq + t.m0 * K, clamp_bytes(t.rows * K));
    const i32x4 sr = rsrc_words(p.xs + t.m0 * p.KB, clamp_bytes(t.rows * p.KB * 4));

    // Pieces of 1 KB as in the tiled kernel.  A wave fills, of weight sub-rows a,
    // rows 64 (wave / 4 + 2 j) + 32 a + 8 (wave % 4) + [0, 8) for j = 0, 1, and
    // activation rows 8 (wave + 8 j).
    const int r_in = lane >> 3;
    const int chunk = 16 * ((lane & 7) ^ r_in ^ (wave & 1));
    const int wrow = 64 * group + 8 * quarter;
    const uint32_t wgo = (uint32_t)((wrow + r_in) * K + chunk);
    const uint32_t xgo = (uint32_t)((8 * wave + r_in) * K + chunk);
    const uint32_t rows32 = (uint32_t)(32 * K);
    const int kb_in = (int)((K - chunk + kBlock - 1) / kBlock);
    const uint32_t lds0 = lds_address(lds);
    const uint32_t wlds = lds0 + wrow * 128, xlds = lds0 + kX + wave * 1024;
    const uint32_t slds = lds_address(xsl) + wave * C::kScaleLoads * 256;
    // the lane's offsets: out of range for good once its piece lies past K
    uint32_t wv = wgo, xv = xgo;
    auto aim = [&](int kb) __attribute__((always_inline)) {
        wv = kb < kb_in ? wv : kOobOffset;
        xv = kb < kb_in ? xv : kOobOffset;
    };
    // (st: the stage, kb % 3; wv and xv aimed at kb)
    auto fill_w = [&](const int st, const int a, const int j, int kb) __attribute__((always_inline)) {
        fill16(SILU && j ? wr_up : wr, wlds + st * kStage + (a + 4 * j) * 4096, wv,
               (SILU ? a : a + 4 * j) * rows32 + (uint32_t)kb * kBlock);
    };
    auto fill_x = [&](const int st, const int j, int kb) __attribute__((always_inline)) {
        fill16(xr, xlds + st * kStage + j * 8192, xv, 2 * j * rows32 + (uint32_t)kb * kBlock);
    };
    // Entry (row, block) of a batch at row * kSB + scale_slot(block, row); entries
    // past the last block are the next row's, or zero: unused.
    auto fill_scales = [&](int kb) __attribute__((always_inline)) {
        const uint32_t dst = slds + ((kb / C::kSB) & 1) * (C::kBM * C::kSB * 4);
        const int f = wave * C::kScaleLoads * 64 + lane;
        const int row = f / C::kSB, slot = f & (C::kSB - 1);
#pragma unroll
        for (int j = 0; j < C::kScaleLoads; ++j)
            fill4(sr, dst + j * 256, (uint32_t)((row * p.KB + scale_slot(slot, row + 8 * j)) * 4),
                  (uint32_t)(kb * 4 + j * 8 * 4 * (int)p.KB));
    };

    const int rr = lane & 31, hi = lane >> 5;
    const int swz = (rr & 7) ^ ((rr >> 3) & 1);
    int wfrag[4], xfrag[4];   // fragment addresses of sub-row 0, stage 0
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int piece = 16 * ((2 * s + hi) ^ swz);
        wfrag[s] = (quarter * 64 + rr) * 128 + piece;
        xfrag[s] = kX + (group * 64 + rr) * 128 + piece;
    }
    const int srow = (group * 64 + rr) * C::kSB;

    int64_t nbw = (SILU ? t.n0 + quarter / 2 * p.I : t.n0 + 64 * quarter) / kBlock;
    if (nbw > p.NB - 1) nbw = p.NB - 1;
    const BI8_CONST float *ws_row =
        reinterpret_cast<const BI8_CONST float *>(reinterpret_cast<uintptr_t>(t.ws + nbw * p.KB));
    float ws_cur = ws_row[0];

    f32x16 zero16;
#pragma unroll
    for (int i = 0; i < 16; ++i) zero16[i] = 0.f;
    f32x16 acc[SB];
    float y[SA][SB][16];   // (single registers: vectors of 16 would need room to be moved)
    float tb[SB], xsv[SB], wsv = 0.f;
#pragma unroll
    for (int b = 0; b < SB; ++b) {
        acc[b] = zero16;
        tb[b] = 0.f;
#pragma unroll
        for (int a = 0; a < SA; ++a)
#pragma unroll
            for (int i = 0; i < 16; ++i) y[a][b][i] = 0.f;
    }
    // activation fragments: sub-row 0 of even and of odd blocks, sub-row 1 (WIDE:
    // sub-row 0 of the next block, sub-row 1 of this one, and both of this one in f16)
    i32x4 xf[3][4], wf[4];
    f16x8 xh[SB][WIDE ? 8 : 1];
    auto read_x = [&](i32x4 (&f)[4], const int st, const int b) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            f[s] = *reinterpret_cast<const i32x4 *>(lds + xfrag[s] + (st * kStage + b * 4096));
    };

    // elements [i0, i0 + n) of sub-tile (a, b)
    auto rescale = [&](const int a, const int b, const int i0, const int n) __attribute__((always_inline)) {
#pragma unroll
        for (int i = i0; i < i0 + n; ++i) y[a][b][i] = fmaf(acc[b][i], tb[b], y[a][b][i]);
#pragma unroll
        for (int i = i0; i < i0 + n; ++i) asm volatile("" ::"v"(y[a][b][i]));
    };
    // Memory phase of cluster a of block kb, in stage st, set = kb % 2.  It reads
    // the weight fragments of its cluster and, of the activations, sub-row 1 in
    // a = 0 and the next block's sub-row 0 in a = 1: 8 reads each.  Fills of block
    // kb + 2, into the stage that block kb - 1 has left: the activation rows and
    // the first piece of the weight sub-rows 0 in a = 0, the others in a = 1.
    // The waits leave the younger fills in flight (a batch of scales among
    // them only makes a wait stricter).
    auto memory = [&](auto ac, auto stc, auto setc, int kb) __attribute__((always_inline)) {
        constexpr int a = decltype(ac)::value, st = decltype(stc)::value, set = decltype(setc)::value;
        constexpr int next = (st + 1) % 3, after = (st + 2) % 3;
#pragma unroll
        for (int s = 0; s < 4; ++s) wf[s] = *reinterpret_cast<const i32x4 *>(lds + wfrag[s] + (st * kStage + a * 4096));
        if constexpr (a == 0) {
            read_x(xf[2], st, 1);
#pragma unroll
            for (int b = 0; b < SB; ++b)
                xsv[b] = xsl[(kb / C::kSB) & 1][srow + b * 32 * C::kSB + scale_slot(kb & (C::kSB - 1), rr)];
            wsv = ws_cur;
            ws_cur = ws_row[kb + 1 < nkb ? kb + 1 : nkb - 1];
            if (__builtin_expect(((kb + 2) & (C::kSB - 1)) == 0, 0)) fill_scales(kb + 2);
            aim(kb + 2);
            fill_x(after, 0, kb + 2);
            fill_x(after, 1, kb + 2);
            fill_w(after, 0, 0, kb + 2);
        } else {
            read_x(xf[WIDE ? 0 : set ^ 1], next, 0);
            fill_w(after, 0, 1, kb + 2);
            fill_w(after, 1, 0, kb + 2);
            fill_w(after, 1, 1, kb + 2);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (!WIDE || busy) rescale(a ^ 1, 0, 0, 16);
        if constexpr (WIDE) {
            if (both) rescale(a ^ 1, 1, 0, 16);
        }
        if constexpr (a == 0)
            wait_lds<7>();   // weight sub-rows 1 of this block, the activation rows of the next
        else
            wait_lds<8>();   // weight sub-rows 0 of the next block
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (WIDE && a == 0) {
            auto widen = [&](const int b) __attribute__((always_inline)) {
                tb[b] = xsv[b] * wsv;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    xh[b][c] = to_f16x8(xf[2 * b][c / 2][2 * (c & 1)], xf[2 * b][c / 2][2 * (c & 1) + 1]);
            };
            if (busy) widen(0);
            if (both) widen(1);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Math phase, as in the 256 x 256 kernel.
    auto math = [&](auto ac, auto setc) __attribute__((always_inline)) {
        constexpr int a = decltype(ac)::value, before = a ^ 1, x0 = decltype(setc)::value;
        if constexpr (WIDE) {
            auto products = [&](auto sub_rows) __attribute__((always_inline)) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const f16x8 wh = to_f16x8(wf[c / 2][2 * (c & 1)], wf[c / 2][2 * (c & 1) + 1]);
#pragma unroll
                    for (int b = 0; b < decltype(sub_rows)::value; ++b)
                        acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(wh, xh[b][c], c ? acc[b] : zero16, 0, 0, 0);
                }
            };
            if (both)
                products(std::integral_constant<int, 2>{});
            else if (busy)
                products(std::integral_constant<int, 1>{});
#pragma unroll
            for (int b = 0; b < SB; ++b) asm volatile("" : "+v"(acc[b]));
            return;
        }
        acc[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(wf[0], wf[1]), join16(xf[x0][0], xf[x0][1]),
                                                                 zero16, 0, 0, 0, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        rescale(before, 1, 0, 8);
        __builtin_amdgcn_sched_barrier(0);
        acc[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(wf[2], wf[3]), join16(xf[x0][2], xf[x0][3]),
                                                                 acc[0], 0, 0, 0, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        rescale(before, 1, 8, 8);
        if constexpr (a == 0) {
#pragma unroll
            for (int b = 0; b < SB; ++b) tb[b] = xsv[b] * wsv;
        }
        __builtin_amdgcn_sched_barrier(0);
        acc[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(wf[0], wf[1]), join16(xf[2][0], xf[2][1]),
                                                                 zero16, 0, 0, 0, 0, 0, 0);
        acc[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join16(wf[2], wf[3]), join16(xf[2][2], xf[2][3]),
                                                                 acc[1], 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int b = 0; b < SB; ++b) asm volatile("" : "+v"(acc[b]));
    };
    auto cluster = [&](auto ac, auto stc, auto setc, int kb) __attribute__((always_inline)) {
        memory(ac, stc, setc, kb);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        math(ac, setc);
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    fill_scales(0);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
        aim(st);
        fill_x(st, 0, st);
        fill_x(st, 1, st);
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            fill_w(st, a, 0, st);
            fill_w(st, a, 1, st);
        }
    }
    wait_lds<8>();
    lds_barrier();
    read_x(xf[0], 0, 0);
    if (group == 1) lds_barrier();   // group 1 runs one phase behind
    int kb = 0;
    auto turn = [&](auto self, auto ic) __attribute__((always_inline)) -> void {
        constexpr int i = decltype(ic)::value;   // kb % 6
        if constexpr (i < 6) {
            cluster(std::integral_constant<int, 0>{}, std::integral_constant<int, i % 3>{},
                    std::integral_constant<int, i % 2>{}, kb);
            cluster(std::integral_constant<int, 1>{}, std::integral_constant<int, i % 3>{},
                    std::integral_constant<int, i % 2>{}, kb);
            if (++kb < nkb) self(self, std::integral_constant<int, i + 1>{});
        }
    };
    while (kb < nkb) turn(turn, std::integral_constant<int, 0>{});
    if (group == 0) lds_barrier();
    rescale(1, 0, 0, 16);
    rescale(1, 1, 0, 16);
    wait_vmcnt<0>();   // no LDS fill may outlive the workgroup

    if constexpr (SILU)
        gate_store<SA>(p, t, y, lds, reinterpret_cast<uint32_t *>(xsl), 2 * group + (quarter & 1), quarter < 2,
                       64 * (quarter & 1), group * 64, lane);
    else
        store_lines<SA, SB, C::kBN, C::kBM>(p, t, y, lds, quarter * 64, group * 64, lane, wave);
#endif  // __HIP_DEVICE_COMPILE__
}

typedef Cfg<4, 2, 1, 2, 4> Cfg128x128;   // weight rows x activation rows
typedef Cfg<4, 2, 1, 1, 4> Cfg128x64;

// (the host pass has to emit the launch stubs)
template __global__ void gemm_fp8_pingpong128_kernel<false, 8>(GemmArgs);
template __global__ void gemm_fp8_pingpong128_kernel<true, 8>(GemmArgs);
template __global__ void gemm_fp8_pingpong128_kernel<true, 8, true>(GemmArgs);
template __global__ void gemm_fp8_pingpong128_kernel<false, 8, false, true>(GemmArgs);
template __global__ void gemm_fp8_pingpong128_kernel<true, 8, false, true>(GemmArgs);
template __global__ void gemm_fp8_pingpong128_kernel<true, 8, true, true>(GemmArgs);
template __global__ void gemm_fp8_tiled_kernel<Cfg128x128, false, false, 8>(GemmArgs);
template __global__ void gemm_fp8_tiled_kernel<Cfg128x128, true, false, 8>(GemmArgs);
template __global__ void gemm_fp8_tiled_kernel<Cfg128x128, false, false, 8, true>(GemmArgs);
template __global__ void gemm_fp8_tiled_kernel<Cfg128x128, false, true, 8>(GemmArgs);
template __global__ void gemm_fp8_tiled_kernel<Cfg128x64, true, true, 8>(GemmArgs);
template __global__ void gemm_fp8_tiled_kernel<Cfg128x64, false, true, 8>(GemmArgs);
template __global__ void gemm_fp8_tiled_kernel<Cfg128x64, false, false, 8>(GemmArgs);
template __global__ void gemm_fp8_tiled_kernel<Cfg128x64, true, false, 8>(GemmArgs);

template __global__ void gemm_fp8_pingpong_kernel<false, 4>(GemmArgs);
template __global__ void gemm_fp8_pingpong_kernel<true, 4>(GemmArgs);
template __global__ void gemm_fp8_pingpong_kernel<true, 4, true>(GemmArgs);

// Grouped: at least the sum over experts of ceil(rows / bm), of which no more than
// p.M have rows.
template <bool MOE>
int64_t most_tiles_m(const GemmArgs &p, int64_t bm) {
    return (p.M + bm - 1) / bm + (MOE ? (p.M < p.E ? p.M : p.E) : 0);
}

template <class C, bool MOE, bool SILU = false, bool WIDE = false>
hipError_t launch_pingpong(GemmArgs p, hipStream_t stream) {
    p.tiles_m = most_tiles_m<MOE>(p, C::kBM);
    p.tiles_n = (p.N + C::kBN - 1) / C::kBN;   // (SILU: I / 128)
    const int64_t total = p.tiles_m * p.tiles_n;
    if (!launch_fits(total, C::kThreads)) return hipErrorInvalidValue;
    if constexpr (C::kBM == 256)
        hipLaunchKernelGGL((gemm_fp8_pingpong_kernel<MOE, 4, SILU>), dim3((unsigned)total), dim3(C::kThreads), 0, stream,
                           p);
    else
        hipLaunchKernelGGL((gemm_fp8_pingpong128_kernel<MOE, 8, SILU, WIDE>), dim3((unsigned)total), dim3(C::kThreads), 0,
                           stream, p);
    return hipGetLastError();
}

template <class C, bool MOE, bool SPLIT, int64_t GM, bool ODD = false>
hipError_t launch_tiled(GemmArgs p, hipStream_t stream, int64_t splits = 1) {
    p.tiles_m = most_tiles_m<MOE>(p, C::kBM);
    p.tiles_n = (p.N + C::kBN - 1) / C::kBN;
    const int64_t total = p.tiles_m * p.tiles_n + (MOE && SPLIT ? kTailRound : 0);
    if (!launch_fits(total, C::kThreads) || splits < 1 || splits > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gemm_fp8_tiled_kernel<C, MOE, SPLIT, GM, ODD>), dim3((unsigned)total, (unsigned)splits),
                       dim3(C::kThreads), 0, stream, p);
    return hipGetLastError();
}

template <bool MOE>
hipError_t launch_path(Fp8Path path, const GemmArgs &p, hipStream_t stream) {
    switch (path) {
        case Fp8Path::kSkinny: return launch_skinny<false, MOE>(p, MOE ? (p.M + p.E - 1) / p.E : p.M, stream);
        case Fp8Path::kTile128x64: return launch_tiled<Cfg128x64, MOE, false, 8>(p, stream);
        case Fp8Path::kTile128x128: return launch_tiled<Cfg128x128, MOE, false, 8>(p, stream);
        case Fp8Path::kTile256x128: return launch_pingpong<PingPong128, MOE>(p, stream);
        case Fp8Path::kTile256x256: return launch_pingpong<PingPong, MOE>(p, stream);
        case Fp8Path::kTile256x128F16: return launch_pingpong<PingPong128, MOE, false, true>(p, stream);
        default: return hipErrorInvalidValue;
    }
}

// ---------------------------------------------------------------------------
// Choice of the kernel
// ---------------------------------------------------------------------------
//
// A tile takes a time of its own (first fills, stores) and one per K block, with few
// tiles on the chip and with all 256 CUs taken (one workgroup a CU).  The estimate
// of a launch is its rounds of tiles, the last one's by how full it is, and the
// weight's stream beside them; split over K, a unit walks its share of the blocks,
// and the partial sums are written and read once.  The choice is the smallest
// estimate.  The constants are fitted to some 700 products of sizes drawn over 1 to 8192
// rows, 64 to 28672 columns, K 128 to 14336 and up to 64 experts
// (profiles/e4m3_gemm_choice.csv), where the chosen kernel takes 0.3 % (dense) and
// 0.9 % (grouped) longer than the fastest of the five on average; 0.7 % and 0.8 % on
// 500 others.
struct Tiling {
    Fp8Path path;
    int bn, bm;
    double light, full, tile;   // us a K block, us a tile
};
constexpr Tiling kTilings[] = {
    {Fp8Path::kTile128x64, 128, 64, 0.32, 0.56, 3.2},
    {Fp8Path::kTile128x128, 128, 128, 0.48, 0.73, 3.8},
    {Fp8Path::kTile256x128, 256, 128, 0.71, 1.27, 4.7},
    {Fp8Path::kTile256x256, 256, 256, 1.00, 1.60, 5.8},
};
constexpr double kCUs = 256;
constexpr int64_t kMaxPartialBytes = 64ll << 20;

struct Choice {
    Fp8Path path = Fp8Path::kSkinny;
    int32_t splits = 1;
    double us = 1e30;
};

double tiles_us(const Tiling &t, double tiles, int64_t blocks) {
    const double rounds = (double)(int64_t)(tiles / kCUs), rest = tiles - rounds * kCUs;
    const double last = rest > 0 ? t.tile + blocks * (t.light + (t.full - t.light) * rest / kCUs) : 0;
    return rounds * (t.tile + blocks * t.full) + last;
}

// The launch, the tiles' time and the weight's stream, which overlap, the
// shorter one not quite.
double overlapped_us(double tiles, double stream) {
    return 1.7 + (tiles < stream ? stream + 0.15 * tiles : tiles + 0.15 * stream);
}

// The streaming kernel: the weight's stream, longer where a wave's blocks leave
// loads of its last round unused and with more rows (`more`), and no less than the
// time of a chunk of so many rows.
double streaming_us(double stream, double rows, double more, double chunk, int64_t KB) {
    const int64_t mine = (KB + skinny_parts(KB) - 1) / skinny_parts(KB);
    const int64_t unroll = skinny_unroll(skinny_mt((int64_t)rows));
    const double waste = KB > 8 ? (double)((mine + unroll - 1) / unroll * unroll) / mine : 1;
    const double us = 4 + stream * waste * (1 + more), least = 4.2 + chunk * rows;
    return us < least ? least : us;
}

// Rows at any byte have two kernels: the streaming one, its loads made of
// dwords, in chunks of 64 tokens, and 128 x 128 tiles (streaming / tiles, us: M =
// 100, N = 4096, K = 1001 17.6 / 24.8; 2000 x 300 x 101 10.1 / 14.6; 64 x 20000 x
// 1001 33.8 / 25.5; 300 x 8192 x 2047 96 / 38; 4096 x 8192 x 1001 492 / 184).
bool odd_rows_streamed(int64_t M, int64_t N) { return N * (16 + M) <= 1000000; }

// partial: bytes of fp32 partial sums that may be used (0: no split).
// The streaming kernel reads the activations again for every 16 weight rows, and
// for more than 16 tokens a CU holds one workgroup, not two.  Measured (streaming /
// 128 x 64, us, weights from HBM, K = 4096): M = 1, N = 131072 91 / 116, M = 16, N =
// 28672 31.5 / 29.7, M = 32, N = 14336 31.1 / 19.0 (17.7 split over K), M = 64, N =
// 4096 16.1 / 18.4 (13.1 split), M = 64, N = K = 2048 15.4 / 9.8, M = 16, N = 8192, K =
// 28672 71 / 98 (47 split).
Choice choose_dense(int64_t M, int64_t N, int64_t K, int64_t partial) {
    Choice best;
    const double bytes = (double)N * (double)K;
    const int64_t KB = (K + kBlock - 1) / kBlock;
    if (M <= 64) best.us = streaming_us(bytes / 5.5e6, (double)M, (M - 1) * (M <= 16 ? 0.02 : 0.047), 0.2, KB);
    for (const Tiling &t : kTilings) {
        const double tiles = (double)((M + t.bm - 1) / t.bm) * (double)((N + t.bn - 1) / t.bn);
        const bool may_split = t.bn == 128;
        for (int32_t z = 1; z <= (may_split ? 8 : 1); ++z) {
            const int64_t per = (KB + z - 1) / z;
            if (z > 1 && (tiles * z > kCUs || per < 4 || z * M * N * 4 > partial || (KB + per - 1) / per != z)) continue;
            const double us = overlapped_us(tiles_us(t, tiles * z, per), bytes / 4.9e6) +
                              (z > 1 ? 3 + 8e-6 * z * M * N / 4 : 0);
            if (us < best.us) {
                best.path = t.path;
                best.splits = z;
                best.us = us;
            }
        }
    }
    return best;
}

// Segments are ragged and only the device knows them: R rows spread evenly over
// the experts, and half a tile more for each.  The weights of as many experts count
// as can have rows, at 5.5 TB/s for the tiled kernels and 6.35 for the streaming
// one: rates of the fit, whose segments are drawn, so that some experts have none
// and their weights are not read (where all have rows the streaming kernel reads
// 5.3 to 6.0 TB/s).  On 70 products whose experts all have rows the choice takes
// 1.2 % longer than the fastest of the five on average.
struct Grouped {
    double experts, mean, bytes;   // experts with rows, rows of each, bytes of their weights
    int64_t N, KB;
    Grouped(int64_t R, int64_t N_, int64_t K, int32_t E)
        : experts((double)(R < E ? R : E)), mean((double)R / experts), bytes(experts * (double)N_ * (double)K), N(N_),
          KB((K + kBlock - 1) / kBlock) {}
    double tiles(const Tiling &t) const {
        const double m = mean <= 1 ? 1 : mean / t.bm + 0.5 < 1 ? 1 : mean / t.bm + 0.5;
        return experts * m * (double)((N + t.bn - 1) / t.bn);
    }
    double us(double tiles) const { return overlapped_us(tiles, bytes / 5.5e6); }
};

double grouped_streaming_us(const Grouped &g) {
    return streaming_us(g.bytes / 6.35e6, g.mean, g.mean > 2 ? (g.mean - 2) / 12 : 0, 0.25, g.KB);
}

constexpr int64_t kGroupedPartialBytes = kTailRound * 128 * 64 * (int64_t)sizeof(float);   // a slot for each unit of a round

Choice choose_grouped(int64_t R, int64_t N, int64_t K, int32_t E, int64_t partial) {
    const Grouped g(R, N, K, E);
    Choice best;
    best.us = grouped_streaming_us(g);
    for (const Tiling &t : kTilings) {
        const double tiles = g.tiles(t);
        double us = tiles_us(t, tiles, g.KB);
        int32_t splits = 1;
        if (t.path == Fp8Path::kTile128x64 && partial >= kTailRound * t.bn * t.bm * 4 && tiles <= kCUs / 2) {
            const double most = (double)(int64_t)(kCUs / tiles), z = most < g.KB / 4.0 ? most : g.KB / 4.0;
            const double split_us = tiles_us(t, tiles * z, (int64_t)(g.KB / z) + 1) + 6;
            if (z >= 2 && split_us < us) {
                us = split_us;
                splits = 2;
            }
        }
        us = g.us(us);
        if (us < best.us) {
            best.path = t.path;
            best.splits = splits;
            best.us = us;
        }
    }
    return best;
}

// The F16 variant's tiles: as above, from its times alone on the chip and with all
// CUs busy.
constexpr Tiling kTilingF16 = {Fp8Path::kTile256x128F16, 256, 128, 1.27, 1.65, 5.0};

GemmArgs fp8_args(const uint8_t *xq, const float *xs, const uint8_t *w, const float *ws, const uint16_t *bias,
                  uint16_t *y, int64_t M, int64_t N, int64_t K) {
    return make_args(reinterpret_cast<const int8_t *>(xq), xs, reinterpret_cast<const int8_t *>(w), ws, bias, y, M, N,
                     K);
}

}  // namespace

Fp8Path select_gemm_fp8_path(int64_t M, int64_t N, int64_t K) {
    if (K % 16 != 0) return odd_rows_streamed(M, N) ? Fp8Path::kSkinny : Fp8Path::kTile128x128;
    return choose_dense(M, N, K, 0).path;
}

Fp8Path select_moe_gemm_fp8_path(int64_t R, int64_t N, int64_t K, int32_t E) {
    return choose_grouped(R, N, K, E, 0).path;
}

// The layer's w13 GEMM feeds a second quantiser, where a sum cut by the f8 matrix
// instruction moves codes by whole steps: the layer's output is then 0.0034 from the
// 64-bit evaluation, 0.0017 otherwise.  So it takes a kernel that holds its sums
// wherever the weights' stream leaves the matrix core most of that time: the
// streaming kernel, or the F16 tiles where they take little longer than the stream.
// Measured (layer of 8 experts, H 4096, I 14336, top 2, f8 / F16 tiles, us): 64
// tokens 285 / 300, 256 tokens 317 / 343; 1024 tokens, left to the f8 tiles, 518 /
// 730, and small layers, whose f8 tiles take half the time of F16 ones.
// kAuto: the grouped GEMM's own choice (whose streaming kernel holds them too).
Fp8Path select_layer_w13_path(int64_t R, int64_t N, int64_t K, int32_t E) {
    const Grouped g(R, N, K, E);
    const Choice c = choose_grouped(R, N, K, E, kGroupedPartialBytes);
    if (c.path == Fp8Path::kSkinny) return Fp8Path::kAuto;
    const double stream = g.bytes / 5.5e6, tiles = tiles_us(kTilingF16, g.tiles(kTilingF16), g.KB);
    const double streamed = grouped_streaming_us(g), tiled = tiles <= 1.35 * stream ? g.us(tiles) : 1e30;
    const double held = streamed < tiled ? streamed : tiled;
    if (held > 1.3 * c.us) return Fp8Path::kAuto;
    return streamed < tiled ? Fp8Path::kSkinny : Fp8Path::kTile256x128F16;
}

int64_t gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (K % 16 != 0) return 0;
    const Choice c = choose_dense(M, N, K, kMaxPartialBytes);
    return c.splits > 1 ? (int64_t)c.splits * M * N * 4 : 0;
}

hipError_t launch_gemm_fp8(Fp8Path path, const uint8_t *xq, const float *xs, const uint8_t *w, const float *ws,
                           const uint16_t *bias, uint16_t *y, int64_t M, int64_t N, int64_t K, float *workspace,
                           int64_t workspace_bytes, hipStream_t stream) {
    if (M == 0) return hipSuccess;
    GemmArgs p = fp8_args(xq, xs, w, ws, bias, y, M, N, K);
    if (K % 16 != 0)   // rows at any byte
        return odd_rows_streamed(M, N) ? launch_skinny<true, false>(p, M, stream)
                                       : launch_tiled<Cfg128x128, false, false, 8, true>(p, stream);
    if (path != Fp8Path::kAuto) return launch_path<false>(path, p, stream);
    const int64_t need = workspace ? gemm_fp8_workspace_bytes(M, N, K) : 0;
    if (need == 0 || workspace_bytes < need) return launch_path<false>(select_gemm_fp8_path(M, N, K), p, stream);
    const Choice c = choose_dense(M, N, K, kMaxPartialBytes);
    p.partial = workspace;
    p.kb_per_split = (p.KB + c.splits - 1) / c.splits;
    p.wide_store = N % 4 == 0;   // (the workspace is 16-byte aligned)
    const hipError_t e = c.path == Fp8Path::kTile128x64
                             ? launch_tiled<Cfg128x64, false, true, 8>(p, stream, c.splits)
                             : launch_tiled<Cfg128x128, false, true, 8>(p, stream, c.splits);
    if (e != hipSuccess) return e;
    const bool vec = N % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & 7) == 0;
    const int64_t blocks = ((vec ? M * N / 4 : M * N) + 255) / 256;
    if (!launch_fits(blocks, 256)) return hipErrorInvalidValue;
    if (vec)
        hipLaunchKernelGGL(splitk_reduce_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, stream, workspace,
                           c.splits, M, N, bias, y);
    else
        hipLaunchKernelGGL(splitk_reduce_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, stream, workspace,
                           c.splits, M, N, bias, y);
    return hipGetLastError();
}

int64_t moe_gemm_fp8_workspace_bytes(int64_t R, int64_t N, int64_t K, int32_t E) {
    return choose_grouped(R, N, K, E, kGroupedPartialBytes).splits > 1 ? kGroupedPartialBytes : 0;
}

hipError_t launch_moe_gemm_fp8(Fp8Path path, const uint8_t *xq, const float *xs, const int32_t *offsets,
                               const uint8_t *w, const float *ws, uint16_t *y, int64_t R, int64_t N, int64_t K,
                               int32_t E, float *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (R == 0) return hipSuccess;
    GemmArgs p = fp8_args(xq, xs, w, ws, nullptr, y, R, N, K);
    p.offsets = offsets;
    p.E = E;
    if (path != Fp8Path::kAuto) return launch_path<true>(path, p, stream);
    const int64_t need = workspace ? moe_gemm_fp8_workspace_bytes(R, N, K, E) : 0;
    if (need == 0 || workspace_bytes < need) return launch_path<true>(select_moe_gemm_fp8_path(R, N, K, E), p, stream);
    p.partial = workspace;
    hipError_t e = launch_tiled<Cfg128x64, true, true, 8>(p, stream);
    if (e != hipSuccess) return e;
    p.tiles_n = (N + 127) / 128;
    hipLaunchKernelGGL((moe_fp8_tail_reduce_kernel<128, 64>), dim3(kTailReduceGroups), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_moe_gemm_silu_quant_fp8(const uint8_t *xq, const float *xs, const int32_t *offsets,
                                          const uint8_t *w13, const float *ws13, uint8_t *aq, float *as, int64_t R,
                                          int64_t I, int64_t K, int32_t E, bool f16, hipStream_t stream) {
    if (R == 0) return hipSuccess;
    if (I % kBlock != 0) return hipErrorInvalidValue;
    GemmArgs p = fp8_args(xq, xs, w13, ws13, nullptr, nullptr, R, 2 * I, K);
    p.offsets = offsets;
    p.E = E;
    p.aq = reinterpret_cast<int8_t *>(aq);
    p.as = as;
    p.I = I;
    if (f16) return launch_pingpong<PingPong128, true, true, true>(p, stream);
    const Grouped g(R, 2 * I, K, E);
    const Tiling &small = kTilings[2], &large = kTilings[3];
    return g.us(tiles_us(small, g.tiles(small), g.KB)) <= g.us(tiles_us(large, g.tiles(large), g.KB))
               ? launch_pingpong<PingPong128, true, true>(p, stream)
               : launch_pingpong<PingPong, true, true>(p, stream);
}

}  // namespace bi8
