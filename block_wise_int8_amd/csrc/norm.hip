// Root-mean-square norm with the residual's addition in front and the 8-bit
// quantisation behind it, one pass over a row:
//
//   h    = bf16(x + residual)                       (h = x without a residual)
//   rstd = fl32(1 / sqrt(mean(h^2) + eps))          (binary64 up to the rounding)
//   y    = fl32(fl32(h rstd) weight)
//   per 128 columns: s = max |y| / kMax, code = rne(y / s)      (codes.hpp)
//
// y is quantised from fp32, without the bf16 rounding that a norm and a
// quantiser in two launches put between them.  The sum of squares is held in
// binary64: squares of bf16 values are exact there and their sum all but
// exact, so rstd, and with it every code and scale, does not depend on the
// order of the addition, and the codes are reproducible bit for bit.
//
// Bound by HBM: 2 B read an element (4 with the residual) and 1 B written (2
// more for h, 2 more for the optional bf16 y), 4 B a group.  A row stays in
// registers as bf16 between the sum and the codes, so it is read once.
// Measured with a residual and e4m3 codes: 1 x 4096 3.2 us (a launch's latency),
// 4096 x 4096 22 us (5.3 TB/s), 16384 x 4096 82 us (5.7), 2048 x 20000, walked
// twice, 64 us. With int8 codes, whose encoding takes more vector work, 4096 x 4096
// 22 us and 16384 x 4096 85 us (5.6).
#include "codes.hpp"
#include "internal.hpp"

namespace bi8 {

namespace {

struct NormArgs {
    const uint16_t *x;
    const uint16_t *residual;   // null: none
    const uint16_t *weight;
    uint16_t *h;                // bf16(x + residual) (with a residual)
    uint16_t *y;                // null, or the normalised row in bf16
    int8_t *xq;
    float *xs;
    int64_t ldx, ldr, ldh;
    int64_t M, H, HB;
    double eps;
};

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// W waves share a row (1: four rows a workgroup, no barrier; 4: one row, the
// waves' sums meet in LDS).  C: chunks of 8 columns a lane, kept in registers;
// 0: any H, the row is walked twice.  ODD: H % 8 != 0 or a row off the 16-byte
// grid.
template <class Codes, int W, int C, bool ODD>
__global__ __launch_bounds__(256) void rmsnorm_quant_kernel(NormArgs p) {
    __shared__ double part[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = W == 1 ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x;
    if (W == 1 && m >= p.M) return;
    const int t = W == 1 ? lane : threadIdx.x;
    constexpr int64_t kStep = 64 * W * 8;   // columns a sweep covers
    const int64_t H = p.H;
    auto load = [&](const uint16_t *row, int64_t k) __attribute__((always_inline)) {
        if constexpr (ODD)
            return load_bf16x8(row + k, H - k);
        else
            return *reinterpret_cast<const u32x4 *>(row + k);
    };
    auto store = [&](uint16_t *row, int64_t k, const u32x4 &v) __attribute__((always_inline)) {
        if constexpr (ODD)
            store_bf16x8(row + k, v, H - k);
        else
            *reinterpret_cast<u32x4 *>(row + k) = v;
    };
    const uint16_t *xrow = p.x + m * p.ldx;
    const uint16_t *rrow = p.residual ? p.residual + m * p.ldr : nullptr;
    uint16_t *hrow = p.residual ? p.h + m * p.ldh : nullptr;
    auto add = [&](const u32x4 &a, const u32x4 &b) __attribute__((always_inline)) {
        float fa[8], fb[8];
        unpack_bf16x8(a, fa);
        unpack_bf16x8(b, fb);
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f32x2_to_bf16x2_bits(fa[2 * i] + fb[2 * i], fa[2 * i + 1] + fb[2 * i + 1]);
        return o;
    };
    double ss = 0.0;
    auto square = [&](const u32x4 &v) __attribute__((always_inline)) {
        float f[8];
        unpack_bf16x8(v, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma((double)f[i], (double)f[i], ss);
    };
    float rstd = 0.0f;
    auto finish_sum = [&]() __attribute__((always_inline)) {
        ss = wave_sum64(ss);
        if constexpr (W > 1) {
            if (lane == 0) part[wave] = ss;
            __syncthreads();
            ss = (part[0] + part[1]) + (part[2] + part[3]);
        }
        rstd = (float)(1.0 / sqrt(ss / (double)H + p.eps));
    };
    // columns [k, k + 8) of the row: every lane of a 16-lane group calls it
    // (the group maximum crosses lanes), those past the row with zeros
    auto emit = [&](const u32x4 &hv, const u32x4 &wv, int64_t k) __attribute__((always_inline)) {
        float hf[8], wf[8], yf[8];
        unpack_bf16x8(hv, hf);
        unpack_bf16x8(wv, wf);
#pragma unroll
        for (int i = 0; i < 8; ++i) yf[i] = (hf[i] * rstd) * wf[i];
        if constexpr (ODD) {   // (0 * rstd is not 0 for every rstd)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i >= H) yf[i] = 0.0f;
        } else {
            if (k >= H) {
#pragma unroll
                for (int i = 0; i < 8; ++i) yf[i] = 0.0f;
            }
        }
        const float s = group_amax_f32(yf) / Codes::kMax;
        if (k >= H) return;
        uint32_t lo, hi;
        Codes::encode(yf, s, lo, hi);
        int8_t *dst = p.xq + m * H + k;
        if constexpr (ODD)
            store_codes(dst, lo, hi, H - k);
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(lo, hi);
        if ((t & 15) == 0) p.xs[m * p.HB + k / kBlock] = s;
        if (p.y) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = f32x2_to_bf16x2_bits(yf[2 * i], yf[2 * i + 1]);
            store(p.y + m * H, k, o);
        }
    };

    const u32x4 zero = {0u, 0u, 0u, 0u};
    if constexpr (C > 0) {
        u32x4 v[C], g[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t k = 8 * t + kStep * c;
            v[c] = k < H ? load(xrow, k) : zero;
        }
        if (rrow) {
            u32x4 r[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t k = 8 * t + kStep * c;
                r[c] = k < H ? load(rrow, k) : zero;
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t k = 8 * t + kStep * c;
                v[c] = add(v[c], r[c]);
                if (k < H) store(hrow, k, v[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t k = 8 * t + kStep * c;
            g[c] = k < H ? load(p.weight, k) : zero;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) square(v[c]);
        finish_sum();
#pragma unroll
        for (int c = 0; c < C; ++c) emit(v[c], g[c], 8 * t + kStep * c);
    } else {
        for (int64_t k = 8 * t; k < H; k += kStep) {
            u32x4 v = load(xrow, k);
            if (rrow) {
                v = add(v, load(rrow, k));
                store(hrow, k, v);
            }
            square(v);
        }
        finish_sum();
        // h again, from where this thread wrote it (it may lie over x or the
        // residual, so the sum is not formed twice)
        const uint16_t *again = rrow ? hrow : xrow;
        for (int64_t k0 = 0; k0 < H; k0 += kStep) {
            const int64_t k = k0 + 8 * t;
            emit(k < H ? load(again, k) : zero, k < H ? load(p.weight, k) : zero, k);
        }
    }
}

template <class Codes, int W, int C, bool ODD>
hipError_t launch(NormArgs p, hipStream_t stream) {
    constexpr int64_t kRows = W == 1 ? 4 : 1;   // of a workgroup
    for (int64_t left = p.M; left > 0;) {
        p.M = left < kBandWorkgroups * kRows ? left : kBandWorkgroups * kRows;
        hipLaunchKernelGGL((rmsnorm_quant_kernel<Codes, W, C, ODD>), dim3((unsigned)((p.M + kRows - 1) / kRows)),
                           dim3(256), 0, stream, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        left -= p.M;
        p.x += p.M * p.ldx;
        if (p.residual) {
            p.residual += p.M * p.ldr;
            p.h += p.M * p.ldh;
        }
        if (p.y) p.y += p.M * p.H;
        p.xq += p.M * p.H;
        p.xs += p.M * p.HB;
    }
    return hipSuccess;
}

// four waves a row, by the sweeps of 2048 columns that it takes
template <class Codes, bool ODD>
hipError_t sweeps(const NormArgs &p, hipStream_t stream) {
    const int64_t n = (p.H + 2047) / 2048;
    if (n <= 1) return launch<Codes, 4, 1, ODD>(p, stream);
    if (n <= 2) return launch<Codes, 4, 2, ODD>(p, stream);
    if (n <= 4) return launch<Codes, 4, 4, ODD>(p, stream);
    if (n <= 8) return launch<Codes, 4, 8, ODD>(p, stream);
    return launch<Codes, 4, 0, ODD>(p, stream);
}

template <class Codes>
hipError_t choose(const NormArgs &p, hipStream_t stream) {
    auto off = [](const void *q) { return q && (reinterpret_cast<uintptr_t>(q) & 15u) != 0; };
    const bool odd = p.H % 8 != 0 || p.ldx % 8 != 0 || off(p.x) || off(p.weight) || off(p.y) ||
                     (p.residual && (p.ldr % 8 != 0 || p.ldh % 8 != 0 || off(p.residual) || off(p.h)));
    // A wave a row where the row is short and there are enough of them to fill
    // the chip (16384 x 512 16.8 us against 26.9 with four waves a row, 4096 x
    // 1024 10.3 against 11.4); else four (4096 x 2048 15.6 us against 16.2, 64 x
    // 1024 2.8 against 3.4, one row of 4096 3.3 against 5.8).
    if (p.M >= 1024 && p.H <= 1024 && !odd)
        return p.H <= 512 ? launch<Codes, 1, 1, false>(p, stream) : launch<Codes, 1, 2, false>(p, stream);
    return odd ? sweeps<Codes, true>(p, stream) : sweeps<Codes, false>(p, stream);
}

}  // namespace

hipError_t launch_rmsnorm_quant(bool fp8, const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                                const uint16_t *weight, double eps, int64_t M, int64_t H, uint16_t *h, int64_t ldh,
                                uint16_t *y, void *xq, float *xs, hipStream_t stream) {
    if (M == 0) return hipSuccess;
    const NormArgs p{x, residual, weight, h, y, static_cast<int8_t *>(xq), xs, ldx, ldr, ldh, M, H,
                     (H + kBlock - 1) / kBlock, eps};
    return fp8 ? choose<E4m3Codes>(p, stream) : choose<Int8Codes>(p, stream);
}

}  // namespace bi8
