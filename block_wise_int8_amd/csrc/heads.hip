// Root-mean-square norm of query and key heads and their rotation by position,
// one pass over the heads:
//
//   u = x rsqrt(mean(x^2) + eps) weight           (u = x without a weight)
//   (u1, u2) -> (u1 c - u2 s, u2 c + u1 s)        pair by pair, up to `rot`
//
// A group of G lanes (a power of two) holds a head: each lane has units of two
// chunks of CH values, which are the two halves of CH pairs, so that neither
// pairing moves a value between lanes; only the sum of squares crosses them.
// The sum is held in binary64, where squares of bf16 values are exact and do
// not overflow.  The cosines and sines of a token are read once for all the
// heads that the group takes.
//
// Bound by HBM: 2 B read and 2 B written a value, and rot * 4 B of the table a
// token.
#include "common.hpp"
#include "internal.hpp"

namespace bi8 {

namespace {

constexpr int kThreads = 256;

template <int CH>
__device__ __forceinline__ void load_chunk(const uint16_t *p, float *f) {
    if constexpr (CH == 8) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_bits_to_f32(v[i] & 0xFFFFu);
            f[2 * i + 1] = bf16_bits_to_f32(v[i] >> 16);
        }
    } else if constexpr (CH == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        f[0] = bf16_bits_to_f32(v.x & 0xFFFFu);
        f[1] = bf16_bits_to_f32(v.x >> 16);
        f[2] = bf16_bits_to_f32(v.y & 0xFFFFu);
        f[3] = bf16_bits_to_f32(v.y >> 16);
    } else {
        f[0] = bf16_bits_to_f32(*p);
    }
}

template <int CH>
__device__ __forceinline__ void store_chunk(uint16_t *p, const float *f) {
    if constexpr (CH == 8) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f32x2_to_bf16x2_bits(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<u32x4 *>(p) = v;
    } else if constexpr (CH == 4) {
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(f32x2_to_bf16x2_bits(f[0], f[1]), f32x2_to_bf16x2_bits(f[2], f[3]));
    } else {
        *p = (uint16_t)f32_to_bf16_bits(f[0]);
    }
}

// Unit u of a head is the chunks at columns c0 and c1 (c1 may lie past D: no
// chunk) and turns the pairs [CH u, CH u + CH) that are below rot / 2.
template <int CH>
__device__ __forceinline__ void unit_columns(const HeadsArgs &p, int u, int &c0, int &c1) {
    const int half = p.rot >> 1;
    if (p.interleaved) {
        c0 = 2 * CH * u;
        c1 = c0 + CH;
    } else if (CH * u < half) {   // half % CH == 0
        c0 = CH * u;
        c1 = c0 + half;
    } else {
        c0 = p.rot + 2 * (CH * u - half);
        c1 = c0 + CH;
    }
}

// LP: units a lane.  Group g of the grid has token g / p.share and the heads
// g % p.share, + p.share, ...: first the Hq query heads, then the Hk key heads.
template <int CH, int LP>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsArgs p) {
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t group = id >> p.log_lanes;
    const int64_t t = group / p.share;
    if (t >= p.T) return;   // whole groups: they are not split over the end of the grid
    const int lane = (int)(id & ((1 << p.log_lanes) - 1));
    const int half = p.rot >> 1;
    int64_t row[kMaxAxes];
    bool inside = true;
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) {
        row[a] = 0;
        if (a < p.axes) {
            row[a] = p.positions[a * p.positions_axis + t];
            inside &= row[a] >= 0 && row[a] < p.P;
            row[a] *= p.rot;
        }
    }
    if (!inside) return;

    float c[LP][CH], s[LP][CH];
#pragma unroll
    for (int l = 0; l < LP; ++l) {
        const int j0 = CH * (lane + (l << p.log_lanes));
        auto row_of = [&](int j) __attribute__((always_inline)) {
            int64_t r = row[0];
#pragma unroll
            for (int a = 1; a < kMaxAxes; ++a)
                if (j >= p.first[a]) r = row[a];
            return r;
        };
#pragma unroll
        for (int i = 0; i < CH; ++i) c[l][i] = 1.0f, s[l][i] = 0.0f;
        if (j0 >= half) continue;
        if (CH >= 4 && p.table_chunks) {   // a chunk's pairs have one axis and 16-byte aligned rows
            const float *r = p.table + row_of(j0) + j0;
#pragma unroll
            for (int i = 0; i < CH / 4; ++i) {
                const f32x4 cv = reinterpret_cast<const f32x4 *>(r)[i], sv = reinterpret_cast<const f32x4 *>(r + half)[i];
#pragma unroll
                for (int n = 0; n < 4; ++n) c[l][4 * i + n] = cv[n], s[l][4 * i + n] = sv[n];
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (j0 + i < half) {
                    const float *r = p.table + row_of(j0 + i) + j0 + i;
                    c[l][i] = r[0];
                    s[l][i] = r[half];
                }
        }
    }

    const int heads = p.Hq + p.Hk;
    for (int h = (int)(group - t * p.share); h < heads; h += p.share) {
        const bool key = h >= p.Hq;
        const uint16_t *x = key ? p.k + t * p.k_token + (h - p.Hq) * p.k_head : p.q + t * p.q_token + h * p.q_head;
        uint16_t *o = key ? p.k_out + t * p.k_out_token + (h - p.Hq) * p.k_out_head
                          : p.q_out + t * p.q_out_token + h * p.q_out_head;
        const uint16_t *w = key ? p.k_weight : p.q_weight;
        float u[LP][2 * CH];
#pragma unroll
        for (int l = 0; l < LP; ++l) {
            int c0, c1;
            unit_columns<CH>(p, lane + (l << p.log_lanes), c0, c1);
#pragma unroll
            for (int i = 0; i < 2 * CH; ++i) u[l][i] = 0.0f;
            if (c0 < p.D) load_chunk<CH>(x + c0, u[l]);
            if (c1 < p.D) load_chunk<CH>(x + c1, u[l] + CH);
        }
        if (w) {
            double ss = 0.0;
#pragma unroll
            for (int l = 0; l < LP; ++l)
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i) ss = fma((double)u[l][i], (double)u[l][i], ss);
            for (int d = 1; d < 1 << p.log_lanes; d <<= 1) ss += __shfl_xor(ss, d);
            const float rstd = (float)(1.0 / sqrt(ss / (double)p.D + p.eps));
#pragma unroll
            for (int l = 0; l < LP; ++l) {
                int c0, c1;
                unit_columns<CH>(p, lane + (l << p.log_lanes), c0, c1);
                float g[2 * CH];
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i) g[i] = 0.0f;
                if (c0 < p.D) load_chunk<CH>(w + c0, g);
                if (c1 < p.D) load_chunk<CH>(w + c1, g + CH);
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i) u[l][i] = (u[l][i] * rstd) * g[i];
            }
        }
#pragma unroll
        for (int l = 0; l < LP; ++l) {
            const int unit = lane + (l << p.log_lanes);
            int c0, c1;
            unit_columns<CH>(p, unit, c0, c1);
            float v[2 * CH];
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const float a = u[l][2 * i], b = u[l][2 * i + 1];
                    const bool turn = CH * unit + i < half;   // (a product with 0 is no copy: infinities)
                    v[2 * i] = turn ? fmaf(a, c[l][i], -(b * s[l][i])) : a;
                    v[2 * i + 1] = turn ? fmaf(b, c[l][i], a * s[l][i]) : b;
                }
            } else {
                const bool turn = CH * unit < half;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const float a = u[l][i], b = u[l][CH + i];
                    v[i] = turn ? fmaf(a, c[l][i], -(b * s[l][i])) : a;
                    v[CH + i] = turn ? fmaf(b, c[l][i], a * s[l][i]) : b;
                }
            }
            if (c0 < p.D) store_chunk<CH>(o + c0, v);
            if (c1 < p.D) store_chunk<CH>(o + c1, v + CH);
        }
    }
}

template <int CH, int LP>
hipError_t launch(HeadsArgs p, hipStream_t stream) {
    const int64_t token_threads = (int64_t)p.share << p.log_lanes;
    const int64_t band = kBandWorkgroups * kThreads / token_threads;   // tokens of one launch
    for (int64_t left = p.T; left > 0; left -= p.T) {
        p.T = left < band ? left : band;
        hipLaunchKernelGGL((heads_kernel<CH, LP>), dim3((unsigned)((p.T * token_threads + kThreads - 1) / kThreads)),
                           dim3(kThreads), 0, stream, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        p.q += p.T * p.q_token;
        p.q_out += p.T * p.q_out_token;
        if (p.Hk) {
            p.k += p.T * p.k_token;
            p.k_out += p.T * p.k_out_token;
        }
        p.positions += p.T;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_qk_norm_rope(HeadsArgs p, hipStream_t stream) {
    if (p.T == 0) return hipSuccess;
    const int half = p.rot / 2;
    // the widest chunk that every row, pair and weight allows
    auto fits = [&](int ch) {
        auto off = [ch](const void *q) { return q && (reinterpret_cast<uintptr_t>(q) & (uintptr_t)(2 * ch - 1)) != 0; };
        const int64_t strides = p.q_token | p.q_head | p.q_out_token | p.q_out_head |
                                (p.Hk ? p.k_token | p.k_head | p.k_out_token | p.k_out_head : 0);
        return p.D % ch == 0 && (p.interleaved || half % ch == 0) && (strides & (ch - 1)) == 0 && !off(p.q) &&
               !off(p.q_out) && !off(p.q_weight) && !off(p.k_weight) &&
               !(p.Hk && (off(p.k) || off(p.k_out)));
    };
    const int ch = fits(8) ? 8 : fits(4) ? 4 : 1;
    const int units = (p.D + 2 * ch - 1) / (2 * ch);   // rot % (2 ch) == 0 where halves are paired
    p.log_lanes = 0;
    while ((1 << p.log_lanes) < units && p.log_lanes < 6) ++p.log_lanes;
    const int lanes = 1 << p.log_lanes;
    p.table_chunks = ch >= 4 && half % ch == 0 && p.rot % 4 == 0 && (reinterpret_cast<uintptr_t>(p.table) & 15u) == 0;
    for (int a = 1; a < p.axes; ++a) p.table_chunks &= p.first[a] % ch == 0;
    // heads that share a group: one while the grid is small
    const int heads = p.Hq + p.Hk;
    int each = 1;
    while (each < 8 && (p.T * ((heads + 2 * each - 1) / (2 * each)) * lanes) / kThreads >= 2048) each *= 2;
    p.share = (heads + each - 1) / each;
    if (ch == 8) return launch<8, 1>(p, stream);
    if (ch == 4) return units <= 64 ? launch<4, 1>(p, stream) : launch<4, 2>(p, stream);
    if (units <= 64) return launch<1, 1>(p, stream);
    if (units <= 128) return launch<1, 2>(p, stream);
    if (units <= 256) return launch<1, 4>(p, stream);
    return launch<1, 8>(p, stream);
}

}  // namespace bi8
