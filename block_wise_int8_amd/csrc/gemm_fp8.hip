// Block-scaled e4m3 GEMM kernels for gfx950:
//   y[m, n] = bf16( sum_g (sum_{k in g} xq[m, k] w[n, k]) xs[m, g] ws[n / 128, g] (+ bias[n]) )
// dense, and grouped by expert.
//
// A K block of 128 codes is one v_mfma_f32_16x16x128_f8f6f4 (or two of
// v_mfma_f32_32x32x64_f8f6f4): the block sum comes out of the matrix core in
// fp32 and enters the running sum by one fma with the block's scale.  Inside,
// the matrix core adds eight consecutive products at a time, aligned to the
// largest and cut 2^-13 below its leading bit (measured: beside 2^16 a product
// of 2^3 counts and one of 2^2 does not; the older 16x16x32 form does the
// same), and those sums in fp32.  That is 7 2^-13 of the largest product of the
// eight at most, against the 2^-4 to which each code was rounded; the bf16
// product of the converted codes would avoid it at half the rate.  The weight rows are the A operand (rows of
// the result = output columns n) and the activation rows the B operand
// (columns = tokens m), so that a lane holds one token and columns of one
// 128-row weight block: the scale xs[m, g] ws[n / 128, g] is one factor a lane.
// K may be permuted inside a block as long as both operands agree, so a
// lane's 32 operand bytes are whichever two 16-byte pieces are cheapest to
// bring there.
//
// Scales and running sums are fp32; one rounding to bf16 at the store.
#include "gemm_common.hpp"

namespace bi8 {

namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 join16(i32x4 a, i32x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// ---------------------------------------------------------------------------
// Skinny path: few tokens, the weight streamed
// ---------------------------------------------------------------------------
//
// Bound by HBM: N K bytes of weight against 2 M N K operations.  A workgroup
// owns 16 weight rows and its 8 waves split K, so that at N = 4096 each CU has
// one workgroup with its whole 64 KB share of the weight in flight.  A lane
// loads 32 bytes of weight per K block straight into registers, every load of
// U blocks is issued before the first MFMA, and the waves' partial sums meet in
// LDS.
//
// Rows [a, b) of the activations share the weight; they are taken 16 MT at a
// time.  Dense: [0, M), chunks over blockIdx.y.  MOE: one expert's segment, all
// of its chunks in turn (its weight rows then come from L2).
// ODD: K % 16 != 0, rows start at any byte (see buf_load16_any).
constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyUnroll = 4;

template <int MT, bool ODD, bool MOE>
__global__ __launch_bounds__(kSkinnyWaves * 64) void gemm_fp8_skinny_kernel(GemmArgs p, int32_t blocks_per_wave) {
    constexpr int U = MT <= 3 ? kSkinnyUnroll : 2;
    constexpr int kRows = 16 * MT;
    __shared__ float red[kSkinnyWaves][MT][64][4];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int row = lane & 15;    // weight row in the tile, and token column
    const int quad = lane >> 4;   // 32-byte quarter of a K block
    const int64_t K = p.K, KB = p.KB;

    int64_t n0, a = 0, b = p.M;
    const int8_t *w = p.w;
    const float *ws = p.ws;
    if constexpr (MOE) {
        const uint32_t e = blockIdx.x / (uint32_t)p.tiles_n;
        n0 = (int64_t)(blockIdx.x - e * (uint32_t)p.tiles_n) * 16;
        a = p.offsets[e];
        b = p.offsets[e + 1];
        a = a < 0 ? 0 : (a > p.M ? p.M : a);
        b = b < a ? a : (b > p.M ? p.M : b);
        w += (int64_t)e * p.N * K;
        ws += (int64_t)e * p.NB * KB;
    } else {
        n0 = (int64_t)blockIdx.x * 16;
    }

    // (ranges of at most 2^31 bytes: 16 MT rows of K <= 2^23)
    const int64_t wrows = p.N - n0 < 16 ? p.N - n0 : 16;
    uint32_t wd = 0;
    const __amdgpu_buffer_rsrc_t wr =
        ODD ? make_rsrc_any(w + n0 * K, wrows * K, wd) : make_rsrc(w + n0 * K, clamp_bytes(wrows * K));
    const float *ws_row = ws + (n0 / kBlock) * KB;
    auto load = [&](__amdgpu_buffer_rsrc_t r, uint32_t off) __attribute__((always_inline)) {
        return as_i32x4(ODD ? buf_load16_any(r, off) : buf_load16(r, off));
    };
    const int64_t b_begin = (int64_t)wave * blocks_per_wave;
    const int64_t b_end = b_begin + blocks_per_wave < KB ? b_begin + blocks_per_wave : KB;

    // Weight loads in whole 128-byte lines: load lane l reads piece l % 8 of
    // tile row l / 8 (and of row 8 + l / 8); the MFMA wants pieces 2q, 2q + 1 of
    // row i in lane (i, q), brought there by ds_bpermute.
    const int lrow = lane >> 3, lchunk = lane & 7;
    const int bp0 = ((lane & 7) * 8 + 2 * quad) * 4;
    const bool upper = row >= 8;

    for (int64_t m0 = a + (int64_t)blockIdx.y * kRows; m0 < b; m0 += (int64_t)gridDim.y * kRows) {
        const int64_t mrows = b - m0 < kRows ? b - m0 : kRows;
        uint32_t xd = 0;
        const __amdgpu_buffer_rsrc_t xr = ODD ? make_rsrc_any(p.xq + m0 * K, mrows * K, xd)
                                              : make_rsrc(p.xq + m0 * K, clamp_bytes(mrows * K));
        const __amdgpu_buffer_rsrc_t sr = make_rsrc(p.xs + m0 * KB, clamp_bytes(mrows * KB * 4));
        f32x4 yv[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) yv[mt] = f32x4{0.f, 0.f, 0.f, 0.f};

        for (int64_t b0 = b_begin; b0 < b_end; b0 += U) {
            i32x4 wa[U][2];
            i32x4 xb[U][MT][2];
            float xsv[U][MT];
            float wsv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t kb = b0 + u;
                const bool ok = kb < b_end;
                const int64_t kk = kb * kBlock + quad * 32;
                const bool in0 = ok && kk < K, in1 = ok && kk + 16 < K;
                if constexpr (ODD) {
                    // (a weight byte past K would meet a zeroed activation
                    // byte, but NaN codes times zero are NaN: cleared too)
                    wa[u][0] = keep_bytes(load(wr, in0 ? (uint32_t)(wd + row * K + kk) : kOobOffset), K - kk);
                    wa[u][1] = keep_bytes(load(wr, in1 ? (uint32_t)(wd + row * K + kk + 16) : kOobOffset), K - kk - 16);
                } else {
                    const int64_t kc = kb * kBlock + lchunk * 16;
                    const bool inl = ok && kc < K;
                    wa[u][0] = load(wr, inl ? (uint32_t)(lrow * K + kc) : kOobOffset);
                    wa[u][1] = load(wr, inl ? (uint32_t)((lrow + 8) * K + kc) : kOobOffset);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int64_t tok = mt * 16 + row;   // relative to m0
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
                if (b0 + u >= b_end) break;   // (the scale of a block past the end is another block's)
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
                    const f32x4 acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        wf, join16(xb[u][mt][0], xb[u][mt][1]), f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
                    const float t = xsv[u][mt] * wsv[u];
#pragma unroll
                    for (int i = 0; i < 4; ++i) yv[mt][i] = fmaf(acc[i], t, yv[mt][i]);
                }
            }
        }

        // 16x16 result: lane -> token lane & 15, weight rows 4 (lane >> 4) + i
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][mt][lane][i] = yv[mt][i];
        __syncthreads();
        for (int t = threadIdx.x; t < MT * 256; t += kSkinnyWaves * 64) {
            const int mt = t >> 8, c = (t >> 4) & 15, r = t & 15;
            const int src = c + 16 * (r >> 2), i = r & 3;
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < kSkinnyWaves; ++v) s += red[v][mt][src][i];
            const int64_t ml = mt * 16 + c, n = n0 + r;
            if (ml < mrows && n < p.N) {
                if (p.bias) s += bf16_bits_to_f32(p.bias[n]);
                p.y[(m0 + ml) * p.N + n] = (uint16_t)(f32x2_to_bf16x2_bits(s, 0.0f) & 0xFFFFu);
            }
        }
        __syncthreads();   // (the next chunk writes the sums again)
    }
}

// chunks: workgroups that share the rows of one weight tile (dense)
template <int MT, bool ODD, bool MOE>
hipError_t launch_skinny_mt(GemmArgs p, int64_t chunks, hipStream_t stream) {
    p.tiles_n = (p.N + 15) / 16;
    const int64_t blocks = p.tiles_n * p.E;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
    if (chunks > 65535) chunks = 65535;
    const int32_t bpw = (int32_t)((p.KB + kSkinnyWaves - 1) / kSkinnyWaves);
    hipLaunchKernelGGL((gemm_fp8_skinny_kernel<MT, ODD, MOE>), dim3((unsigned)blocks, (unsigned)chunks),
                       dim3(kSkinnyWaves * 64), 0, stream, p, bpw);
    return hipGetLastError();
}

// rows: how many rows a weight tile is likely to meet (dense: M)
template <bool ODD, bool MOE>
hipError_t launch_skinny(const GemmArgs &p, int64_t rows, hipStream_t stream) {
    const int64_t mt = rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 48 ? 3 : 4;
    const int64_t chunks = MOE ? 1 : (p.M + 16 * mt - 1) / (16 * mt);
    switch (mt) {
        case 1: return launch_skinny_mt<1, ODD, MOE>(p, chunks, stream);
        case 2: return launch_skinny_mt<2, ODD, MOE>(p, chunks, stream);
        case 3: return launch_skinny_mt<3, ODD, MOE>(p, chunks, stream);
        default: return launch_skinny_mt<4, ODD, MOE>(p, chunks, stream);
    }
}

GemmArgs fp8_args(const uint8_t *xq, const float *xs, const uint8_t *w, const float *ws, const uint16_t *bias,
                  uint16_t *y, int64_t M, int64_t N, int64_t K) {
    return make_args(reinterpret_cast<const int8_t *>(xq), xs, reinterpret_cast<const int8_t *>(w), ws, bias, y, M, N,
                     K);
}

}  // namespace

int64_t gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K) { return 0; }

hipError_t launch_gemm_fp8(const uint8_t *xq, const float *xs, const uint8_t *w, const float *ws, const uint16_t *bias,
                           uint16_t *y, int64_t M, int64_t N, int64_t K, float *workspace, int64_t workspace_bytes,
                           hipStream_t stream) {
    if (M == 0) return hipSuccess;
    const GemmArgs p = fp8_args(xq, xs, w, ws, bias, y, M, N, K);
    return K % 16 != 0 ? launch_skinny<true, false>(p, M, stream) : launch_skinny<false, false>(p, M, stream);
}

int64_t moe_gemm_fp8_workspace_bytes(int64_t R, int64_t N, int64_t K, int32_t E) { return 0; }

hipError_t launch_moe_gemm_fp8(const uint8_t *xq, const float *xs, const int32_t *offsets, const uint8_t *w,
                               const float *ws, uint16_t *y, int64_t R, int64_t N, int64_t K, int32_t E,
                               float *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (R == 0) return hipSuccess;
    GemmArgs p = fp8_args(xq, xs, w, ws, nullptr, y, R, N, K);
    p.offsets = offsets;
    p.E = E;
    return launch_skinny<false, true>(p, (R + E - 1) / E, stream);
}

}  // namespace bi8
