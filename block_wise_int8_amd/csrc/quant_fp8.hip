// e4m3 quantisers: activations (whole rows and gathered rows), the SiLU gating
// of a gate | up pair, and weights in 128 x 128 blocks.  One scale s = amax /
// 448 a group and codes rne(x / s); see codes.hpp.  Layouts as the int8
// quantisers': 16 lanes share a group of 128 columns, 8 bf16 (one 16-byte
// load) a lane.
//
// Each is one pass over its input and bound by HBM: 2 B read and 1 B written
// an element (the gating 4 and 1), 4 B a group.  Measured: activations 1 x 4096
// 2.1 us, 2048 x 14336 16.0 us (5.5 TB/s), 16384 x 4096 32 us (6.3); gating 8192 x
// 14336 106 us (5.5); weights, which are quantised once, 28672 x 4096 125 us (2.8
// TB/s: a load touches 64 lines, two threads a row).
#include "codes.hpp"
#include "internal.hpp"

namespace bi8 {

namespace {

constexpr int kQuantWaves = 4;   // waves per workgroup

// A lane's chunk `j` of row `m` covers 8 columns of group g0 + 4 j.  rows: the
// gather form (may be null); an index outside [0, src_rows) reads zeros.
// ODD: K % 8 != 0 or rows off the 16-byte grid (see load_bf16x8).
template <int kChunks, bool ODD>
__global__ __launch_bounds__(kQuantWaves * 64) void quant_act_fp8_kernel(
    const uint16_t *__restrict__ x, int64_t K, int64_t ldx, uint8_t *__restrict__ xq, float *__restrict__ xs,
    int64_t KB, int64_t waves_per_row, int64_t total_waves, const int32_t *__restrict__ rows, int64_t src_rows) {
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * kQuantWaves + (threadIdx.x >> 6);
    if (wave >= total_waves) return;
    const int64_t m = wave / waves_per_row;
    const int64_t g0 = (wave - m * waves_per_row) * 4 * kChunks + (lane >> 4);
    const int64_t src = rows ? (int64_t)rows[m] : m;
    const bool src_ok = src >= 0 && src < src_rows;
    u32x4 v[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        const int64_t g = g0 + 4 * j, k = g * kBlock + (lane & 15) * 8;
        v[j] = u32x4{0u, 0u, 0u, 0u};
        if (g < KB && k < K && src_ok)
            v[j] = ODD ? load_bf16x8(x + src * ldx + k, K - k)
                       : *reinterpret_cast<const u32x4 *>(x + src * ldx + k);
    }
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        const int64_t g = g0 + 4 * j, k = g * kBlock + (lane & 15) * 8;
        const float s = group_amax_bf16(v[j]) / E4m3Codes::kMax;
        if (g >= KB || k >= K) continue;
        float f[8];
        uint32_t lo, hi;
        unpack_bf16x8(v[j], f);
        E4m3Codes::encode(f, s, lo, hi);
        uint8_t *dst = xq + m * K + k;
        if constexpr (ODD)
            store_codes(dst, lo, hi, K - k);
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(lo, hi);
        if ((lane & 15) == 0) xs[m * KB + g] = s;
    }
}

// h = [gate | up] bf16 [R, 2 I] -> codes of a = bf16(silu(gate) up); a_out (may
// be null) receives a.  I % 16 == 0.
constexpr int kGateChunks = 2;
__global__ __launch_bounds__(kQuantWaves * 64) void silu_mul_quant_fp8_kernel(
    const uint16_t *__restrict__ h, int64_t I, uint8_t *__restrict__ aq, float *__restrict__ as,
    uint16_t *__restrict__ a_out, int64_t IB, int64_t waves_per_row, int64_t total_waves) {
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * kQuantWaves + (threadIdx.x >> 6);
    if (wave >= total_waves) return;
    const int64_t r = wave / waves_per_row;
    const int64_t g0 = (wave - r * waves_per_row) * 4 * kGateChunks + (lane >> 4);
    u32x4 gv[kGateChunks], uv[kGateChunks];
#pragma unroll
    for (int j = 0; j < kGateChunks; ++j) {
        const int64_t g = g0 + 4 * j, i = g * kBlock + (lane & 15) * 8;
        gv[j] = u32x4{0u, 0u, 0u, 0u};
        uv[j] = u32x4{0u, 0u, 0u, 0u};
        if (g < IB && i < I) {
            gv[j] = *reinterpret_cast<const u32x4 *>(h + r * 2 * I + i);
            uv[j] = *reinterpret_cast<const u32x4 *>(h + r * 2 * I + I + i);
        }
    }
#pragma unroll
    for (int j = 0; j < kGateChunks; ++j) {
        const int64_t g = g0 + 4 * j, i = g * kBlock + (lane & 15) * 8;
        float gf[8], uf[8], a[8];
        unpack_bf16x8(gv[j], gf);
        unpack_bf16x8(uv[j], uf);
        u32x4 ab;   // the bf16 activation: the value that is quantised
#pragma unroll
        for (int e = 0; e < 4; ++e)
            ab[e] = f32x2_to_bf16x2_bits(silu_times(gf[2 * e], uf[2 * e]), silu_times(gf[2 * e + 1], uf[2 * e + 1]));
        const float s = group_amax_bf16(ab) / E4m3Codes::kMax;
        if (g >= IB || i >= I) continue;
        uint32_t lo, hi;
        unpack_bf16x8(ab, a);
        E4m3Codes::encode(a, s, lo, hi);
        *reinterpret_cast<uint2 *>(aq + r * I + i) = make_uint2(lo, hi);
        if ((lane & 15) == 0) as[r * IB + g] = s;
        if (a_out) *reinterpret_cast<u32x4 *>(a_out + r * I + i) = ab;
    }
}

// One workgroup of 256 threads per 128 x 128 block: thread t takes half t % 2
// of row t / 2 (eight chunks).  Rows past N and columns past K read as zero
// and are not written.
template <bool ODD>
__global__ __launch_bounds__(256) void quant_weight_fp8_kernel(const uint16_t *__restrict__ w, int64_t N, int64_t K,
                                                               int64_t ldw, uint8_t *__restrict__ wq,
                                                               float *__restrict__ ws, int64_t KB) {
    __shared__ float wmax[16];
    const int t = threadIdx.x;
    const int64_t bn = blockIdx.y, bk = blockIdx.x;
    const int64_t n = bn * kBlock + (t >> 1);
    const int64_t k0 = bk * kBlock + (t & 1) * 64;
    u32x4 v[8];
    u32x4 top = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int64_t k = k0 + 8 * c;
        v[c] = u32x4{0u, 0u, 0u, 0u};
        if (n < N && k < K)
            v[c] = ODD ? load_bf16x8(w + n * ldw + k, K - k) : *reinterpret_cast<const u32x4 *>(w + n * ldw + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) top[j] = umax<true>(top[j], v[c][j] & 0x7FFF7FFFu);
    }
    const float g = group_amax_bf16(top);
    if ((t & 15) == 0) wmax[t >> 4] = g;
    __syncthreads();
    uint32_t m = 0u;   // (as bits: a NaN stays the largest)
#pragma unroll
    for (int i = 0; i < 16; ++i) m = umax<false>(m, __float_as_uint(wmax[i]));
    const float s = __uint_as_float(m) / E4m3Codes::kMax;
    if (t == 0) ws[bn * KB + bk] = s;
    if (n >= N) return;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int64_t k = k0 + 8 * c;
        if (k >= K) break;
        float f[8];
        uint32_t lo, hi;
        unpack_bf16x8(v[c], f);
        E4m3Codes::encode(f, s, lo, hi);
        uint8_t *dst = wq + n * K + k;
        if constexpr (ODD)
            store_codes(dst, lo, hi, K - k);
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(lo, hi);
    }
}

}  // namespace

hipError_t launch_quant_act_fp8(const uint16_t *x, int64_t src_rows, int64_t ldx, const int32_t *rows, int64_t M,
                                int64_t K, uint8_t *xq, float *xs, hipStream_t stream) {
    const int64_t KB = (K + kBlock - 1) / kBlock;
    const bool odd = K % 8 != 0 || ldx % 8 != 0 || (reinterpret_cast<uintptr_t>(x) & 15u) != 0;
    const bool two = M * KB >= 8192;   // enough groups to fill the chip with two per lane
    const int64_t gpw = two ? 8 : 4;           // groups per wave
    const int64_t waves_per_row = (KB + gpw - 1) / gpw;
    const int64_t band = kBandWorkgroups * kQuantWaves / waves_per_row;   // rows a launch (K <= 2^23: 2048 or more)
    for (int64_t m0 = 0; m0 < M; m0 += band) {
        const int64_t total_waves = (M - m0 < band ? M - m0 : band) * waves_per_row;
        const dim3 grid((unsigned)((total_waves + kQuantWaves - 1) / kQuantWaves)), block(kQuantWaves * 64);
        const uint16_t *src = rows ? x : x + m0 * ldx;
        const int32_t *idx = rows ? rows + m0 : nullptr;
        const int64_t nsrc = rows ? src_rows : src_rows - m0;
        uint8_t *q = xq + m0 * K;
        float *s = xs + m0 * KB;
        if (odd && two)
            hipLaunchKernelGGL((quant_act_fp8_kernel<2, true>), grid, block, 0, stream, src, K, ldx, q, s, KB,
                               waves_per_row, total_waves, idx, nsrc);
        else if (odd)
            hipLaunchKernelGGL((quant_act_fp8_kernel<1, true>), grid, block, 0, stream, src, K, ldx, q, s, KB,
                               waves_per_row, total_waves, idx, nsrc);
        else if (two)
            hipLaunchKernelGGL((quant_act_fp8_kernel<2, false>), grid, block, 0, stream, src, K, ldx, q, s, KB,
                               waves_per_row, total_waves, idx, nsrc);
        else
            hipLaunchKernelGGL((quant_act_fp8_kernel<1, false>), grid, block, 0, stream, src, K, ldx, q, s, KB,
                               waves_per_row, total_waves, idx, nsrc);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_silu_mul_quant_fp8(const uint16_t *h, int64_t R, int64_t I, uint8_t *aq, float *as,
                                     uint16_t *a_out, hipStream_t stream) {
    const int64_t IB = (I + kBlock - 1) / kBlock;
    const int64_t waves_per_row = (IB + 4 * kGateChunks - 1) / (4 * kGateChunks);
    const int64_t band = kBandWorkgroups * kQuantWaves / waves_per_row;
    for (int64_t r0 = 0; r0 < R; r0 += band) {
        const int64_t total_waves = (R - r0 < band ? R - r0 : band) * waves_per_row;
        hipLaunchKernelGGL(silu_mul_quant_fp8_kernel, dim3((unsigned)((total_waves + kQuantWaves - 1) / kQuantWaves)),
                           dim3(kQuantWaves * 64), 0, stream, h + r0 * 2 * I, I, aq + r0 * I, as + r0 * IB,
                           a_out ? a_out + r0 * I : nullptr, IB, waves_per_row, total_waves);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_quant_weight_fp8(const uint16_t *w, int64_t N, int64_t K, int64_t ldw, uint8_t *wq, float *ws,
                                   hipStream_t stream) {
    const int64_t NB = (N + kBlock - 1) / kBlock, KB = (K + kBlock - 1) / kBlock;
    if (NB == 0 || KB == 0) return hipSuccess;
    if (NB > 65535 || KB > 0x7FFFFFFFll) return hipErrorInvalidValue;
    const dim3 grid((unsigned)KB, (unsigned)NB), block(256);
    if (K % 8 != 0 || ldw % 8 != 0 || (reinterpret_cast<uintptr_t>(w) & 15u) != 0)
        hipLaunchKernelGGL(quant_weight_fp8_kernel<true>, grid, block, 0, stream, w, N, K, ldw, wq, ws, KB);
    else
        hipLaunchKernelGGL(quant_weight_fp8_kernel<false>, grid, block, 0, stream, w, N, K, ldw, wq, ws, KB);
    return hipGetLastError();
}

}  // namespace bi8
