// The two 8-bit encodings of a group of values with one fp32 scale, as used by
// the e4m3 quantisers and the normalising quantiser (gfx950 only).
//
// For a group with amax = max |x|:  s = amax / kMax (binary32),  code =
// rne(x / s) with x / s the correctly rounded binary32 quotient, clamped to
// [-kMax, kMax]; all codes are zero when s == 0.
//   Int8Codes  kMax = 127, integers
//   E4m3Codes  kMax = 448, OCP e4m3 (4 exponent bits, 3 mantissa bits, no
//              infinities, largest value 448)
#pragma once

#include "common.hpp"

namespace bi8 {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Largest of the 16 lanes of an aligned lane group, as unsigned words (see
// group_max16): each word one value, or (PACKED) two 16-bit values.
template <bool PACKED>
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) {
    if constexpr (PACKED)
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                      __builtin_bit_cast(u16x2, b)));
    else
        return a > b ? a : b;
}

template <int N>
__device__ __forceinline__ uint32_t row_ror_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}

template <bool PACKED>
__device__ __forceinline__ uint32_t group_umax16(uint32_t v) {
    v = umax<PACKED>(v, row_ror_u32<1>(v));
    v = umax<PACKED>(v, row_ror_u32<2>(v));
    v = umax<PACKED>(v, row_ror_u32<4>(v));
    v = umax<PACKED>(v, row_ror_u32<8>(v));
    return v;
}

// amax of a group of 128 bf16 values over 16 lanes, 8 per lane (two a word).
// With the sign bits cleared bf16 patterns order like the values they stand
// for, NaN above infinity, so one packed unsigned maximum serves two values
// and a NaN anywhere in the group becomes the group's amax (and scale).
__device__ __forceinline__ float group_amax_bf16(const u32x4 &v) {
    uint32_t m = umax<true>(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu);
    m = umax<true>(m, v[2] & 0x7FFF7FFFu);
    m = umax<true>(m, v[3] & 0x7FFF7FFFu);
    m = group_umax16<true>(m);
    const uint32_t lo = m & 0xFFFFu, hi = m >> 16;
    return bf16_bits_to_f32(lo > hi ? lo : hi);
}

// The same over fp32 values.
__device__ __forceinline__ float group_amax_f32(const float (&f)[8]) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax<false>(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return __uint_as_float(group_umax16<false>(m));
}

struct Int8Codes {
    static constexpr float kMax = 127.0f;
    // codes of 8 values (bytes of lo, hi in order)
    static __device__ __forceinline__ void encode(const float (&f)[8], float s, uint32_t &lo, uint32_t &hi) {
        lo = 0u;
        hi = 0u;
        if (s != 0.0f) {
            const float r = __builtin_amdgcn_rcpf(s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo |= ((uint32_t)quant_code(f[i], s, r) & 0xFFu) << (8 * i);
                hi |= ((uint32_t)quant_code(f[4 + i], s, r) & 0xFFu) << (8 * i);
            }
        }
    }
};

struct E4m3Codes {
    static constexpr float kMax = 448.0f;
    // The quotient q = x / s costs three operations: q0 = x r with r = fl(1/s)
    // (one division per group), the exact remainder e = q0 s - x, and
    // q = fl(q0 - e r), which is the correctly rounded quotient whenever q0 is
    // within an ulp of it and nothing underflows (Markstein); the signs are
    // placed so that a negative zero stays one.  bf16 inputs
    // often lie exactly half way between two codes, so an ulp of the quotient
    // decides codes; every bf16 significand against every bf16 group maximum
    // is checked against the division by a test.  |x| <= amax makes |q| at
    // most 448 (1 + 2^-22), which rounds to 448: no clamp.  Scales outside
    // (2^-80, 2^100), NaN among them, divide, and clamp (a subnormal scale
    // may lie far below amax / 448).  The hardware conversion rounds to
    // nearest even and keeps e4m3's subnormals.
    static __device__ __forceinline__ void encode(const float (&f)[8], float s, uint32_t &lo, uint32_t &hi) {
        float q[8];
        if (s > 0x1p-80f && s < 0x1p100f) {
            const float r = 1.0f / s;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q0 = f[i] * r;
                q[i] = fmaf(-fmaf(q0, s, -f[i]), r, q0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = f[i] / s;   // (NaN stays NaN: infinity over an infinite scale)
                q[i] = s == 0.0f ? 0.0f : v > kMax ? kMax : v < -kMax ? -kMax : v;
            }
        }
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], a, true);
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], b, true);
        lo = (uint32_t)a;
        hi = (uint32_t)b;
    }
};

// The 8 bf16 values of a 16-byte chunk as fp32.
__device__ __forceinline__ void unpack_bf16x8(const u32x4 &v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_bits_to_f32(v[i] & 0xFFFFu);
        f[2 * i + 1] = bf16_bits_to_f32(v[i] >> 16);
    }
}

// 16 bytes at any 2-byte, 8 bytes at any byte address: single instructions, the
// hardware takes global accesses at any byte.
struct __attribute__((packed, aligned(2))) Any16 {
    u32x4 v;
};
struct __attribute__((packed, aligned(1))) Any8 {
    uint32_t lo, hi;
};

// The first n of the 8 bf16 values at p, zeros behind them.
__device__ __forceinline__ u32x4 load_bf16x8(const uint16_t *p, int64_t n) {
    if (n >= 8) return reinterpret_cast<const Any16 *>(p)->v;
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) v[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
    return v;
}

// Store the first n of 8 bf16 values, of 8 codes.
__device__ __forceinline__ void store_bf16x8(uint16_t *p, const u32x4 &v, int64_t n) {
    if (n >= 8) {
        reinterpret_cast<Any16 *>(p)->v = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) p[j] = (uint16_t)((v[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
}

__device__ __forceinline__ void store_codes(void *p, uint32_t lo, uint32_t hi, int64_t n) {
    if (n >= 8) {
        *reinterpret_cast<Any8 *>(p) = Any8{lo, hi};
        return;
    }
    uint8_t *b = static_cast<uint8_t *>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) b[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
}

}  // namespace bi8
