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
// token.  4096 tokens of 32 + 8 heads of 128 with the norm 17.0 us (5.1 TB/s, the
// rate of a copy of as much), 8191 tokens of 28 + 4 heads without 26.4 us (5.2), 1
// token 2.5 us (a launch's latency).
#include "common.hpp"
#include "internal.hpp"

namespace bi8 {

namespace {

constexpr int kThreads = 256;

// A chunk of CH values as it lies in memory, two a word, at any 2-byte address
// (single instructions: the hardware takes global accesses at any byte).
template <int CH>
struct __attribute__((packed, aligned(2))) Chunk {
    uint32_t w[CH / 2];
};
template <>
struct Chunk<1> {
    uint16_t w[1];
};

template <int CH>
__device__ __forceinline__ void unpack(const Chunk<CH> &c, float *f) {
    if constexpr (CH == 1) {
        f[0] = bf16_bits_to_f32(c.w[0]);
    } else {
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
            const uint32_t w = c.w[i];
            f[2 * i] = __uint_as_float(w << 16);
            f[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
    }
}

template <int CH>
__device__ __forceinline__ Chunk<CH> pack(const float *f) {
    Chunk<CH> c;
    if constexpr (CH == 1) {
        c.w[0] = (uint16_t)f32_to_bf16_bits(f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) c.w[i] = f32x2_to_bf16x2_bits(f[2 * i], f[2 * i + 1]);
    }
    return c;
}

template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xF, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xF, 0xF, false);
    return v + __hiloint2double(hi, lo);
}

// The sum over the 2^log_lanes lanes of an aligned group, in each of them: pairs,
// quads, then mirrored halves (whose quads hold one value each).
__device__ __forceinline__ double group_sum(double v, int log_lanes) {
    if (log_lanes >= 1) v = add_dpp<0xB1>(v);    // quad_perm [1, 0, 3, 2]
    if (log_lanes >= 2) v = add_dpp<0x4E>(v);    // quad_perm [2, 3, 0, 1]
    if (log_lanes >= 3) v = add_dpp<0x141>(v);   // row_half_mirror
    if (log_lanes >= 4) v = add_dpp<0x140>(v);   // row_mirror
    if (log_lanes >= 5) v += __shfl_xor(v, 16);
    if (log_lanes >= 6) v += __shfl_xor(v, 32);
    return v;
}

// 1 / sqrt(m) to well below 2^-24: the hardware's estimate, corrected once.
__device__ __forceinline__ float rsqrt64(double m) {
    const double y = __builtin_amdgcn_rsq(m);
    if (!(m > 0.0 && m < INFINITY)) return (float)y;
    return (float)(y * fma(-0.5 * m, y * y, 1.5));
}

// Unit u of a head is the chunks at columns c0 and c1 (past D: no chunk) and
// turns the pairs [CH u, CH u + CH) that are below rot / 2.
template <int CH, bool INTERLEAVED>
__device__ __forceinline__ void unit_columns(const HeadsArgs &p, int u, int &c0, int &c1) {
    const int half = p.rot >> 1;
    if (INTERLEAVED) {
        c0 = 2 * CH * u;
        c1 = c0 + CH;
    } else {   // half % CH == 0
        const bool turned = CH * u < half;
        c0 = turned ? CH * u : p.rot + 2 * (CH * u - half);
        c1 = c0 + (turned ? half : CH);
    }
}

// LP: units a lane.  A token has p.q_groups groups of lanes for its query heads
// and p.k_groups for its key heads; group w of n takes the heads w, w + n, ...,
// p.each at most.  FULL: every lane has two whole chunks and turns them.  NORM:
// heads of both kinds have a weight (else none has).
//
// The loads of a group's first head, of its positions and weight and then of its
// table row are issued without a branch between them, those of lanes, heads and
// tokens that are not there at addresses that are; each further head is on its way
// while the one before is worked on and stored.
template <int CH, int LP, bool INTERLEAVED, bool FULL, bool NORM>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsArgs p) {
    const uint32_t id = blockIdx.x * kThreads + threadIdx.x;   // (a launch has fewer than 2^32 threads)
    const uint32_t group = id >> p.log_lanes, groups = p.q_groups + p.k_groups, token = group / groups;
    const int64_t t = token < p.T ? token : p.T - 1;
    const int lane = (int)(id & ((1u << p.log_lanes) - 1));
    const int half = p.rot >> 1;
    int first = (int)(group - token * groups);
    const bool key = first >= p.q_groups;
    first -= key ? p.q_groups : 0;
    const int step = pick(key, p.k_groups, p.q_groups), heads = pick(key, p.Hk, p.Hq);
    const int64_t pitch = pick(key, p.k_head, p.q_head), out_pitch = pick(key, p.k_out_head, p.q_out_head);
    const uint16_t *const in = pick(key, p.k, p.q) + t * pick(key, p.k_token, p.q_token);
    uint16_t *const out = pick(key, p.k_out, p.q_out) + t * pick(key, p.k_out_token, p.q_out_token);

    struct Unit {
        Chunk<CH> a, b;
    };
    int c0[LP], c1[LP];
    bool in0[LP], in1[LP];
#pragma unroll
    for (int l = 0; l < LP; ++l) {
        unit_columns<CH, INTERLEAVED>(p, lane + (l << p.log_lanes), c0[l], c1[l]);
        in0[l] = FULL || c0[l] < p.D;
        in1[l] = FULL || c1[l] < p.D;
    }
    auto load = [&](const uint16_t *row, Unit (&u)[LP]) __attribute__((always_inline)) {
#pragma unroll
        for (int l = 0; l < LP; ++l) {
            u[l].a = *reinterpret_cast<const Chunk<CH> *>(row + (in0[l] ? c0[l] : 0));
            u[l].b = *reinterpret_cast<const Chunk<CH> *>(row + (in1[l] ? c1[l] : 0));
        }
    };
    Unit next[LP], weight[LP];
    load(in + first * pitch, next);
    static_assert(kMaxAxes == 4, "axes by name");
    const int32_t *at = p.positions + t;   // (axes that are not there: the first again)
    const int32_t at0 = at[0], at1 = at[p.axes > 1 ? p.positions_axis : 0],
                  at2 = at[p.axes > 2 ? 2 * p.positions_axis : 0], at3 = at[p.axes > 3 ? 3 * p.positions_axis : 0];
    if constexpr (NORM) load(pick(key, p.k_weight, p.q_weight), weight);

    const int first1 = p.first[1], first2 = p.first[2], first3 = p.first[3], rot = p.rot;
    const int64_t P = p.P;
    auto fits = [=](int32_t i) { return i >= 0 && i < P; };
    const bool inside = token < p.T && fits(at0) && fits(at1) && fits(at2) && fits(at3);
    auto row_of = [=](int j) __attribute__((always_inline)) {
        int32_t i = pick(j >= first1, at1, at0);
        i = pick(j >= first2, at2, i);
        i = pick(j >= first3, at3, i);
        return (int64_t)(inside ? i : 0) * rot;
    };
    float c[LP][CH], s[LP][CH];
#pragma unroll
    for (int l = 0; l < LP; ++l) {
        const int j0 = CH * (lane + (l << p.log_lanes));
        if (CH >= 4 && p.table_chunks) {   // a chunk's pairs have one axis and 16-byte aligned rows
            const int j = j0 < half ? j0 : 0;
            const float *r = p.table + row_of(j) + j;
#pragma unroll
            for (int i = 0; i < CH / 4; ++i) {
                const f32x4 cv = reinterpret_cast<const f32x4 *>(r)[i], sv = reinterpret_cast<const f32x4 *>(r + half)[i];
#pragma unroll
                for (int n = 0; n < 4; ++n) c[l][4 * i + n] = cv[n], s[l][4 * i + n] = sv[n];
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int j = j0 + i < half ? j0 + i : 0;
                const float *r = p.table + row_of(j) + j;
                c[l][i] = r[0];
                s[l][i] = r[half];
            }
        }
    }
    float g[LP][2 * CH];
    if constexpr (NORM) {
#pragma unroll
        for (int l = 0; l < LP; ++l) {
            unpack<CH>(weight[l].a, g[l]);
            unpack<CH>(weight[l].b, g[l] + CH);
        }
    }

    for (int i = 0; i < p.each; ++i) {
        const int h = first + i * step;
        float u[LP][2 * CH];
#pragma unroll
        for (int l = 0; l < LP; ++l) {
            unpack<CH>(next[l].a, u[l]);
            unpack<CH>(next[l].b, u[l] + CH);
            if (!FULL) {
#pragma unroll
                for (int n = 0; n < 2 * CH; ++n) u[l][n] = (n < CH ? in0[l] : in1[l]) ? u[l][n] : 0.0f;
            }
        }
        load(in + min(h + step, heads - 1) * pitch, next);
        if constexpr (NORM) {
            double ss = 0.0;
#pragma unroll
            for (int l = 0; l < LP; ++l)
#pragma unroll
                for (int n = 0; n < 2 * CH; ++n) ss = fma((double)u[l][n], (double)u[l][n], ss);
            const float rstd = rsqrt64(fma(group_sum(ss, p.log_lanes), p.inverse, p.eps));
#pragma unroll
            for (int l = 0; l < LP; ++l)
#pragma unroll
                for (int n = 0; n < 2 * CH; ++n) u[l][n] = (u[l][n] * rstd) * g[l][n];
        }
        uint16_t *const o = out + h * out_pitch;
        const bool there = inside && h < heads;
#pragma unroll
        for (int l = 0; l < LP; ++l) {
            const int unit = lane + (l << p.log_lanes);
            float v[2 * CH];
#pragma unroll
            for (int n = 0; n < CH; ++n) {
                const int one = INTERLEAVED ? 2 * n : n, two = INTERLEAVED ? 2 * n + 1 : CH + n;
                const float a = u[l][one], b = u[l][two];
                const bool turn = FULL || (INTERLEAVED ? CH * unit + n : CH * unit) < half;   // (a product with 0 is no copy)
                v[one] = turn ? fmaf(a, c[l][n], -(b * s[l][n])) : a;
                v[two] = turn ? fmaf(b, c[l][n], a * s[l][n]) : b;
            }
            if (there && in0[l]) *reinterpret_cast<Chunk<CH> *>(o + c0[l]) = pack<CH>(v);
            if (there && in1[l]) *reinterpret_cast<Chunk<CH> *>(o + c1[l]) = pack<CH>(v + CH);
        }
    }
}

template <int CH, int LP, bool INTERLEAVED, bool FULL, bool NORM>
hipError_t launch(HeadsArgs p, hipStream_t stream) {
    const int64_t token_threads = (int64_t)(p.q_groups + p.k_groups) << p.log_lanes;
    const int64_t band = kBandWorkgroups * kThreads / token_threads;   // tokens of one launch
    for (int64_t left = p.T; left > 0; left -= p.T) {
        p.T = left < band ? left : band;
        hipLaunchKernelGGL((heads_kernel<CH, LP, INTERLEAVED, FULL, NORM>),
                           dim3((unsigned)((p.T * token_threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream,
                           p);
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

template <bool INTERLEAVED, bool NORM>
hipError_t by_chunks(const HeadsArgs &p, int ch, int units, hipStream_t stream) {
    if (ch == 8)
        return p.D % 16 == 0 && p.rot == p.D && units == 1 << p.log_lanes
                   ? launch<8, 1, INTERLEAVED, true, NORM>(p, stream)
                   : launch<8, 1, INTERLEAVED, false, NORM>(p, stream);
    if (ch == 4)
        return units <= 64 ? launch<4, 1, INTERLEAVED, false, NORM>(p, stream)
                           : launch<4, 2, INTERLEAVED, false, NORM>(p, stream);
    if (units <= 64) return launch<1, 1, INTERLEAVED, false, NORM>(p, stream);
    if (units <= 128) return launch<1, 2, INTERLEAVED, false, NORM>(p, stream);
    if (units <= 256) return launch<1, 4, INTERLEAVED, false, NORM>(p, stream);
    return launch<1, 8, INTERLEAVED, false, NORM>(p, stream);
}

}  // namespace

hipError_t launch_qk_norm_rope(HeadsArgs p, hipStream_t stream) {
    if (p.T == 0) return hipSuccess;
    if (p.Hk == 0) p.k_weight = p.q_weight;
    if (!p.q_weight != !p.k_weight) {   // a norm of one kind of heads: a launch each
        HeadsArgs k = p;
        k.q = p.k, k.q_weight = p.k_weight, k.q_out = p.k_out, k.Hq = p.Hk;
        k.q_token = p.k_token, k.q_head = p.k_head, k.q_out_token = p.k_out_token, k.q_out_head = p.k_out_head;
        p.Hk = k.Hk = 0;
        const hipError_t e = launch_qk_norm_rope(p, stream);
        return e == hipSuccess ? launch_qk_norm_rope(k, stream) : e;
    }
    const int half = p.rot / 2;
    // the widest chunk that heads and pairs allow; rows and weights lie anywhere
    auto fits = [&](int ch) { return p.D % ch == 0 && (p.interleaved || half % ch == 0); };
    const int ch = fits(8) ? 8 : fits(4) ? 4 : 1;
    const int units = (p.D + 2 * ch - 1) / (2 * ch);   // rot % (2 ch) == 0 where halves are paired
    p.inverse = 1.0 / p.D;
    p.log_lanes = 0;
    while ((1 << p.log_lanes) < units && p.log_lanes < 6) ++p.log_lanes;
    p.table_chunks = ch >= 4 && half % ch == 0 && p.rot % 4 == 0 && (reinterpret_cast<uintptr_t>(p.table) & 15u) == 0;
    for (int a = 1; a < p.axes; ++a) p.table_chunks &= p.first[a] % ch == 0;
    // Heads of a group.  One while the grid is small (1 x 40 heads 2.5 us, 2.9 with
    // two); in larger ones more where there is a norm, whose weight is unpacked once
    // for them (4096 tokens of 40 heads of 128: 19.0 us with one, 17.3 two, 17.0 four,
    // 17.8 eight; 2047 of 40 of 80: 9.4, 8.2, 9.0).  Without a norm one stays best
    // (8191 tokens of 32 heads: 26.4, 26.9 with two, 28.1 four).
    const int64_t all = (p.T * (p.Hq + p.Hk) << p.log_lanes) / kThreads;   // workgroups with one each
    p.each = !p.q_weight || all < 2048 ? 1 : all < 4096 ? 2 : 4;
    p.q_groups = (p.Hq + p.each - 1) / p.each;
    p.k_groups = (p.Hk + p.each - 1) / p.each;
    if (p.q_weight)
        return p.interleaved ? by_chunks<true, true>(p, ch, units, stream) : by_chunks<false, true>(p, ch, units, stream);
    return p.interleaved ? by_chunks<true, false>(p, ch, units, stream) : by_chunks<false, false>(p, ch, units, stream);
}

}  // namespace bi8
