// Router of a mixture of experts with scores, a bias for balance and groups, and
// the dispatch order of its tokens (gfx950).
//
//  * route_kernel   a group of G lanes holds a token's logits, V a lane, and takes
//                   the k largest by k reductions over the lanes, of the value and
//                   then of the index of those that have it.  A workgroup has
//                   B <= 64 tokens; a token picks an expert once at most, so one
//                   64-bit word an expert in LDS, with a bit a token, is its
//                   histogram and, below a token's bit, that token's place among
//                   the workgroup's.
//  * place_kernel   a workgroup for the same B tokens: sums the counts of all
//                   workgroups (an expert's start) and of those before it, and
//                   writes the rows.  One workgroup's tokens are placed by
//                   route_kernel itself.
//  * column_kernel  past kSumBlocks workgroups: those sums, once for all.
//
// Bound by the instructions of the picks, and by the latency of their chain where
// tokens are few: 1 token of 256 experts in 8 groups, top 8, 6.3 us, 64 of 128 8.0,
// 4096 of 256 14.7 (11 and 5 of the second kernel), 16381 of 160 21.6 (18 and 5).  The
// logits would take 0.8 and 1.1.
//
// Lanes and groups: the experts of a group lie on G / 2^ceil(log2 groups)
// neighbouring lanes, so that a group's value is a reduction over those.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "common.hpp"
#include "internal.hpp"

namespace bi8 {

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 32;
constexpr int kPlaceThreads = 1024;
constexpr int kSumBlocks = 256;  // workgroups whose counts every workgroup sums by itself

// v of the lane that CTRL names (DPP).  ROWS: the rows of 16 lanes that take it, the
// others keep v.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int dpp(int v) {
    if constexpr (ROWS == 0xF) return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
    return __builtin_amdgcn_update_dpp(v, v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(dpp<CTRL, ROWS>(__float_as_int(v)));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp(double v) {
    return __hiloint2double(dpp<CTRL, ROWS>(__double2hiint(v)), dpp<CTRL, ROWS>(__double2loint(v)));
}
__device__ __forceinline__ int lane_of(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float lane_of(float v, int lane) { return __int_as_float(lane_of(__float_as_int(v), lane)); }
__device__ __forceinline__ double lane_of(double v, int lane) {
    return __hiloint2double(lane_of(__double2hiint(v), lane), lane_of(__double2loint(v), lane));
}

// v of the last lane of the G (16, 32, 64) that this one belongs to, for all of them.
template <int G, class T>
__device__ __forceinline__ T from_last(T v) {
    if constexpr (G == 64) return lane_of(v, 63);
    if constexpr (G == 32) {
        const T a = lane_of(v, 31), b = lane_of(v, 63);
        return pick((threadIdx.x & 32) != 0, b, a);
    }
    return v;   // (every lane of a row of 16 has it)
}

constexpr int kRor1 = 0x121, kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128;   // rotations of a row of 16 lanes
constexpr int kBcast15 = 0x142, kBcast31 = 0x143;   // a row's last lane to the next, lane 31 to the upper half

// op over the G lanes of an aligned group, in every lane of it; op is idempotent,
// so four rotations of a row of 16 lanes cover it.
template <int G, class T, class Op>
__device__ __forceinline__ T reduce(T v, Op op) {
    v = op(v, dpp<kRor1>(v));
    v = op(v, dpp<kRor2>(v));
    v = op(v, dpp<kRor4>(v));
    v = op(v, dpp<kRor8>(v));
    if constexpr (G >= 32) v = op(v, dpp<kBcast15, 0xA>(v));
    if constexpr (G >= 64) v = op(v, dpp<kBcast31, 0xC>(v));
    return from_last<G>(v);
}

// The sum over the G lanes, in every lane of them: the same order for all.
template <int G>
__device__ __forceinline__ double sum(double v) {
    v += dpp<0xB1>(v);    // quad_perm [1, 0, 3, 2]
    v += dpp<0x4E>(v);    // quad_perm [2, 3, 0, 1]
    v += dpp<0x141>(v);   // row_half_mirror
    v += dpp<0x140>(v);   // row_mirror
    if constexpr (G == 32) {
        const double a = lane_of(v, 0) + lane_of(v, 16), b = lane_of(v, 32) + lane_of(v, 48);
        return pick((threadIdx.x & 32) != 0, b, a);
    }
    if constexpr (G == 64) return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
    return v;
}

template <class T>
__device__ __forceinline__ T larger(T a, T b) {
    return pick(a > b, a, b);
}
template <>
__device__ __forceinline__ double larger(double a, double b) {
    return fmax(a, b);
}
template <class T>
__device__ __forceinline__ T smaller(T a, T b) {
    return pick(a < b, a, b);
}

// A logit's place in the order, as a signed word: -infinity and NaN the lowest,
// +infinity as the largest finite value, both zeros alike; kTaken is below all.
constexpr int32_t kTaken = INT_MIN;
__device__ __forceinline__ int32_t order_of(float l) {
    const float f = pick(l > -INFINITY, fminf(l, FLT_MAX), -INFINITY) + 0.0f;
    const int32_t s = __float_as_int(f);
    return s ^ ((s >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float logit_of(int32_t order) {
    return __int_as_float(order ^ ((order >> 31) & 0x7FFFFFFF));
}

// exp(l - m); 0 for NaN and -infinity.
__device__ __forceinline__ double softmax_score(float l, float m) {
    const double e = exp((double)fminf(l, FLT_MAX) - (double)m);
    return pick(l > -INFINITY, e, 0.0);
}

// 1 / (1 + exp(-l)), as t / (1 + t) with t = exp(l) where l is negative: t is at most
// 1, so nothing overflows and the quotient needs no more than the hardware's
// reciprocal of a value in [1, 2], corrected twice.  0 for NaN and -infinity.
__device__ __forceinline__ double sigmoid_score(float l) {
    const double t = exp(-(double)fminf(fabsf(l), FLT_MAX)), d = 1.0 + t;
    double r = __builtin_amdgcn_rcp(d);
    r = fma(fma(-d, r, 1.0), r, r);
    r = fma(fma(-d, r, 1.0), r, r);
    return pick(l > -INFINITY, pick(l >= 0.0f, r, t * r), 0.0);
}
__device__ __forceinline__ double score_of(float l, float m, bool sigmoid) {
    return sigmoid ? sigmoid_score(l) : softmax_score(l, m);
}

// Four logits from a place that is aligned to them.
__device__ __forceinline__ void load_logits4(const RouteArgs &p, const void *row, int e, float *l) {
    if (p.bf16) {
        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(row) + e);
        l[0] = bf16_bits_to_f32(v.x & 0xFFFFu), l[1] = bf16_bits_to_f32(v.x >> 16);
        l[2] = bf16_bits_to_f32(v.y & 0xFFFFu), l[3] = bf16_bits_to_f32(v.y >> 16);
    } else {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(row) + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) l[i] = v[i];
    }
}
// Exclusive prefix of counts[0 .. E) over the workgroup into starts, and the
// total: E <= the number of threads.  All threads call it.
__device__ __forceinline__ void scan_experts(int32_t count, int32_t E, int32_t *starts, int32_t *wave_sums,
                                             int32_t *offsets) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t x = wave_incl_scan(count);
    if (lane == 63) wave_sums[wave] = x;
    __syncthreads();
    int32_t before = 0;
    for (int w = 0; w < wave; ++w) before += wave_sums[w];
    if (tid < E) {
        starts[tid] = before + x - count;
        if (offsets) {
            offsets[tid] = before + x - count;
            if (tid == E - 1) offsets[E] = before + x;
        }
    }
    __syncthreads();
}

// One token on G lanes.  lane's experts: e0 + [0, count).
template <int G, int V, bool BIAS>
__device__ __forceinline__ void route_token(const RouteArgs &p, int64_t t, int t_local, int lane, uint64_t *mask,
                                            uint16_t *picks, float *pick_logits) {
    using Val = typename std::conditional<BIAS, double, int32_t>::type;
    constexpr int kNone = INT_MAX;
    const Val taken = BIAS ? (Val)-INFINITY : (Val)kTaken;   // below every choice
    const int n = p.E / p.groups;
    const int lanes = G >> p.log_groups;   // of a group of experts, a power of two
    const int g = lane / lanes, sub = lane & (lanes - 1);
    const int each = (n + lanes - 1) / lanes;
    const int e0 = g * n + sub * each;
    const int count = g < p.groups ? min(each, n - sub * each) : 0;
    const void *row = p.bf16 ? static_cast<const void *>(static_cast<const uint16_t *>(p.logits) + t * p.ldl)
                             : static_cast<const void *>(static_cast<const float *>(p.logits) + t * p.ldl);
    // all loads at once, those of experts that are not there from one that is
    float l[V], bias[BIAS ? V : 1];
    auto at = [=](int v) { return min(e0 + max(min(v, count - 1), 0), p.E - 1); };
    if (V >= 4 && p.fours) {   // count is 0 or a multiple of 4
#pragma unroll
        for (int v = 0; v < V; v += 4) load_logits4(p, row, at(v & ~3) & ~3, l + v);
    } else if (p.bf16) {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = bf16_bits_to_f32(static_cast<const uint16_t *>(row)[at(v)]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = static_cast<const float *>(row)[at(v)];
    }
    if constexpr (BIAS) {
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = p.bias[at(v)];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = v < count ? l[v] : -INFINITY;

    // the largest logit that counts, and the sum of the exponentials where it is used
    const bool sigmoid = p.score != 0;
    float m = -INFINITY;
    double total = 1.0;
    if (!sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) m = fmaxf(m, l[v]);   // (fmaxf drops NaN)
        m = reduce<G>(m, [](float a, float b) { return fmaxf(a, b); });
        m = fminf(m, FLT_MAX);
    }

    // the choices; those taken and those of groups that are not kept: `taken`
    Val c[V];
    if constexpr (BIAS) {
        if (sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] = sigmoid_score(l[v]);
        } else {
            double part = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                c[v] = softmax_score(l[v], m);
                part += c[v];
            }
            total = sum<G>(part);
            total = pick(total > 0.0, total, 1.0);
            const double inverse = 1.0 / total;
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] *= inverse;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double w = c[v] + (double)bias[v];
            c[v] = pick(v < count, pick(w > -DBL_MAX, fmin(w, DBL_MAX), -DBL_MAX), taken);   // (NaN: the lowest)
        }
    } else {
        if (!sigmoid && !p.renormalize) {   // (exponentials in binary32: 2 of 22 us less, up to 12 units of 2^-24 off)
            double part = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) part += softmax_score(l[v], m);
            total = sum<G>(part);
            total = pick(total > 0.0, total, 1.0);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = pick(v < count, order_of(l[v]), taken);
    }

    if (p.topk_groups < p.groups) {
        Val one = taken, two = taken;   // the group's two largest
#pragma unroll
        for (int v = 0; v < V; ++v) {
            two = larger(two, smaller(one, c[v]));
            one = larger(one, c[v]);
        }
        for (int d = 1; d < lanes; d <<= 1) {
            const Val o1 = __shfl_xor(one, d), o2 = __shfl_xor(two, d);
            two = larger(smaller(one, o1), larger(two, o2));
            one = larger(one, o1);
        }
        double value = (double)one;
        if (p.group_top == 2) {
            if constexpr (BIAS) {
                if (two > taken) value = fmax(value + (double)two, -DBL_MAX);
            } else {
                value = score_of(logit_of(one), m, sigmoid);
                if (two > taken) value += score_of(logit_of(two), m, sigmoid);
            }
        }
        int rank = 0;
        const int base = (threadIdx.x & 63) & ~(G - 1);
#pragma unroll 4
        for (int o = 0; o < p.groups; ++o) {
            const double other = G == 64 ? lane_of(value, o * lanes) : __shfl(value, base + o * lanes);
            rank += other > value || (other == value && o < g) ? 1 : 0;
        }
        if (rank >= p.topk_groups) {
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] = taken;
        }
    }

    // k times the largest choice, then the lowest expert that has it; its lane leaves
    // both the expert and its logit in LDS
    picks += t_local * p.k;
    pick_logits += t_local * p.k;
    for (int j = 0; j < p.k; ++j) {
        Val most = c[0];
#pragma unroll
        for (int v = 1; v < V; ++v) most = larger(most, c[v]);
        most = reduce<G>(most, [](Val a, Val b) { return larger(a, b); });
        int mine = kNone;
#pragma unroll
        for (int v = V - 1; v >= 0; --v) mine = pick(c[v] == most, e0 + v, mine);
        const int expert = reduce<G>(mine, [](int a, int b) { return min(a, b); });
        float logit = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            c[v] = pick(e0 + v == expert, taken, c[v]);
            if constexpr (BIAS) logit = pick(e0 + v == expert, l[v], logit);
        }
        if (mine == expert) {
            if constexpr (!BIAS) logit = logit_of(most);
            picks[j] = (uint16_t)expert;
            pick_logits[j] = logit;
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // read by other lanes of the wave
    __builtin_amdgcn_wave_barrier();
    int id[2] = {0, 0};
    double w[2], all = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = lane + i * G;
        w[i] = 0.0;
        if (j < p.k) {
            id[i] = picks[j];
            w[i] = score_of(pick_logits[j], m, sigmoid);
        }
        all += w[i];
    }
    double factor = p.scale / total;
    if (p.renormalize) {
        all = sum<G>(all);
        factor = all > 0.0 ? p.scale / all : 0.0;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = lane + i * G;
        if (j < p.k) {
            p.ids[t * p.k + j] = id[i];
            p.weights[t * p.k + j] = (float)(w[i] * factor);
            atomicOr(reinterpret_cast<unsigned long long *>(mask + id[i]), 1ull << t_local);
        }
    }
}

__device__ __forceinline__ int below(uint64_t mask, int t) { return __popcll(mask & ((1ull << t) - 1)); }

// A workgroup of THREADS / G tokens at a time; ceil(T / B) of them, or SINGLE one,
// which places its rows too (T = 0 included).
template <int G, int V, bool BIAS, int THREADS, bool SINGLE>
__global__ __launch_bounds__(THREADS) void route_kernel(RouteArgs p) {
    constexpr int kThreads = THREADS;
    __shared__ uint64_t mask[kThreads];   // E <= G V <= kThreads
    __shared__ uint16_t picks[64 * kMaxTop];
    __shared__ float pick_logits[64 * kMaxTop];
    __shared__ int32_t starts[SINGLE ? kThreads : 1];
    __shared__ int32_t wave_sums[16];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * p.block_tokens;
    mask[tid] = 0;
    __syncthreads();
    for (int i = tid / G; i < p.block_tokens; i += kThreads / G)
        if (t0 + i < p.T) route_token<G, V, BIAS>(p, t0 + i, i, tid & (G - 1), mask, picks, pick_logits);
    __syncthreads();
    const int32_t count = tid < p.E ? __popcll(mask[tid]) : 0;
    if constexpr (SINGLE) {
        scan_experts(count, p.E, starts, wave_sums, p.offsets);
        for (int i = tid; i < (int)p.T * p.k; i += kThreads) {
            const int t = i / p.k, e = picks[i];
            const int32_t r = starts[e] + below(mask[e], t);
            p.row_of[i] = r;
            p.sorted_token[r] = t;
        }
    } else {
        if (tid < p.pitch) p.counts[(int64_t)blockIdx.x * p.pitch + tid] = (uint8_t)count;
    }
}

// Counts of four experts of every workgroup -> the sums over the workgroups
// before each, and the totals.  One workgroup a word of four experts.
__global__ __launch_bounds__(256) void column_kernel(RouteArgs p, int64_t blocks) {
    __shared__ int32_t part[256][4];
    const int tid = threadIdx.x, words = p.pitch / 4, col = blockIdx.x;
    const uint32_t *counts = reinterpret_cast<const uint32_t *>(p.counts);
    const int64_t each = (blocks + 255) / 256, b0 = tid * each, b1 = min(b0 + each, blocks);
    int32_t s[4] = {0, 0, 0, 0};
    for (int64_t b = b0; b < b1; ++b) {
        const uint32_t w = counts[b * words + col];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += (w >> (8 * i)) & 0xFF;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[tid][i] = s[i];
    __syncthreads();
    if (tid < 4) {
        int32_t run = 0;
        for (int i = 0; i < 256; ++i) {
            const int32_t x = part[i][tid];
            part[i][tid] = run;
            run += x;
        }
        p.totals[4 * col + tid] = run;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = part[tid][i];
    for (int64_t b = b0; b < b1; ++b) {
        const uint32_t w = counts[b * words + col];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p.before[b * p.pitch + 4 * col + i] = s[i];
            s[i] += (w >> (8 * i)) & 0xFF;
        }
    }
}

__global__ __launch_bounds__(kPlaceThreads) void place_kernel(RouteArgs p, int blocks) {
    __shared__ uint64_t mask[kMaxExperts];
    __shared__ int32_t total[kMaxExperts], starts[kMaxExperts], before[kMaxExperts];
    __shared__ int32_t wave_sums[16];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * p.block_tokens;
    const int entries = (int)(min((int64_t)p.block_tokens, p.T - t0) * p.k);
    mask[tid] = 0;
    if (p.before) {
        total[tid] = tid < p.E ? p.totals[tid] : 0;
        before[tid] = tid < p.E ? p.before[(int64_t)blockIdx.x * p.pitch + tid] : 0;
    } else {
        total[tid] = 0;
        before[tid] = 0;
    }
    __syncthreads();
    const int32_t *ids = p.ids + t0 * p.k;
    for (int i = tid; i < entries; i += kPlaceThreads)
        atomicOr(reinterpret_cast<unsigned long long *>(mask + ids[i]), 1ull << (i / p.k));
    if (!p.before) {
        // thread: four experts of every slices-th workgroup, summed two to a word
        // (at most kSumBlocks / 4 counts of at most 64 in 16 bits)
        const int words = p.pitch / 4, slices = kPlaceThreads / words, col = tid % words, slice = tid / words;
        const uint32_t *counts = reinterpret_cast<const uint32_t *>(p.counts);
        uint32_t even = 0, odd = 0, even_before = 0, odd_before = 0;
        if (slice < slices && slice < blocks) {
            constexpr int kBatch = 8;   // in flight; past the last: the last, not counted
            for (int b0 = slice; b0 < blocks; b0 += kBatch * slices) {
                uint32_t w[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) w[i] = counts[min(b0 + i * slices, blocks - 1) * words + col];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int b = b0 + i * slices;
                    if (b >= blocks) w[i] = 0;
                    even += w[i] & 0x00FF00FFu;
                    odd += (w[i] >> 8) & 0x00FF00FFu;
                    if (b < (int)blockIdx.x) {
                        even_before += w[i] & 0x00FF00FFu;
                        odd_before += (w[i] >> 8) & 0x00FF00FFu;
                    }
                }
            }
            const int e = 4 * col;
            atomicAdd(&total[e], (int)(even & 0xFFFFu));
            atomicAdd(&total[e + 1], (int)(odd & 0xFFFFu));
            atomicAdd(&total[e + 2], (int)(even >> 16));
            atomicAdd(&total[e + 3], (int)(odd >> 16));
            atomicAdd(&before[e], (int)(even_before & 0xFFFFu));
            atomicAdd(&before[e + 1], (int)(odd_before & 0xFFFFu));
            atomicAdd(&before[e + 2], (int)(even_before >> 16));
            atomicAdd(&before[e + 3], (int)(odd_before >> 16));
        }
    }
    __syncthreads();
    scan_experts(tid < p.E ? total[tid] : 0, p.E, starts, wave_sums, blockIdx.x == 0 ? p.offsets : nullptr);
    for (int i = tid; i < entries; i += kPlaceThreads) {
        const int t = i / p.k, e = ids[i];
        const int32_t r = starts[e] + before[e] + below(mask[e], t);
        p.row_of[t0 * p.k + i] = r;
        p.sorted_token[r] = (int32_t)(t0 + t);
    }
}

int block_tokens(int64_t T) { return T <= kSumBlocks * 16 ? 16 : T <= kSumBlocks * 32 ? 32 : 64; }

// Lanes a token, values a lane, and whether one workgroup does it all.
struct RoutePlan {
    int G, V;
    bool single;
};

RoutePlan route_plan(int64_t T, int32_t E, int32_t groups, int log_groups) {
    const int n = E / groups;
    auto values = [&](int G) { return G >> log_groups ? (n + (G >> log_groups) - 1) / (G >> log_groups) : 1 << 20; };
    auto plan = [&](int G, bool single) {
        const int v = values(G);
        return RoutePlan{G, v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : v <= 8 ? 8 : v <= 16 ? 16 : 32, single};
    };
    // One workgroup of 1024 threads while all its tokens go at once and the values
    // stay in 128 registers (64 tokens, 128 experts: 7.6 us with 16 lanes a token,
    // 11.2 with 32 and 17.0 with 64, tokens in turn; 10.9 as two launches).
    if (T <= 16) return plan(64, true);
    if (T <= 32 && values(32) <= 8) return plan(32, true);
    if (T <= 64 && values(16) <= 8) return plan(16, true);
    // Else few tokens take many lanes, for the time of one; many take few, for fewer
    // instructions (4096 tokens, 256 experts: 11.3 us with 16, 11.7 32, 12.7 64).
    for (int G : {16, 32, 64})
        if ((T > 1024 || G == 64) && (values(G) <= 16 || G == 64)) return plan(G, false);
    return plan(64, false);
}

template <int G, int V, bool BIAS>
hipError_t launch_route(const RouteArgs &p, bool single, int64_t blocks, hipStream_t stream) {
    // 32 tokens at once where a workgroup has as many, for two waves a SIMD (16381
    // tokens, 160 experts: 15.4 us against 21.0)
    constexpr int kWide = G == 16 ? 512 : 16 * G;
    if (single)
        hipLaunchKernelGGL((route_kernel<G, V, BIAS, 1024, true>), dim3(1), dim3(1024), 0, stream, p);
    else if (p.block_tokens == 16)
        hipLaunchKernelGGL((route_kernel<G, V, BIAS, 16 * G, false>), dim3((unsigned)blocks), dim3(16 * G), 0, stream, p);
    else
        hipLaunchKernelGGL((route_kernel<G, V, BIAS, kWide, false>), dim3((unsigned)blocks), dim3(kWide), 0, stream, p);
    return hipGetLastError();
}

template <int G, bool BIAS>
hipError_t by_values(const RoutePlan &plan, const RouteArgs &p, int64_t blocks, hipStream_t stream) {
    switch (plan.V) {
        case 1: return launch_route<G, 1, BIAS>(p, plan.single, blocks, stream);
        case 2: return launch_route<G, 2, BIAS>(p, plan.single, blocks, stream);
        case 4: return launch_route<G, 4, BIAS>(p, plan.single, blocks, stream);
        case 8: return launch_route<G, 8, BIAS>(p, plan.single, blocks, stream);
        case 16: return launch_route<G, 16, BIAS>(p, plan.single, blocks, stream);
        default:   // up to 1024 experts in a number of groups that is no power of two
            if constexpr (G == 64) return launch_route<64, 32, BIAS>(p, plan.single, blocks, stream);
            return hipErrorInvalidValue;
    }
}

int64_t pad16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

int64_t route_grouped_workspace_need(int64_t T, int32_t E) {
    const int64_t blocks = (T + block_tokens(T) - 1) / block_tokens(T), pitch = (E + 3) / 4 * 4;
    if (blocks <= 1) return 0;
    const int64_t counts = pad16(blocks * pitch);
    return blocks <= kSumBlocks ? counts : counts + pad16(4 * pitch) + 4 * blocks * pitch;
}

// The most that a batch of up to T tokens needs: workgroups have twice the tokens past
// 2^12 and 2^13, and are half as many.
int64_t route_grouped_workspace_bytes(int64_t T, int32_t E) {
    const int64_t most = route_grouped_workspace_need(T, E);
    return T > kSumBlocks * 16 ? std::max(most, route_grouped_workspace_need(kSumBlocks * 16, E)) : most;
}

hipError_t launch_moe_route_grouped(RouteArgs p, void *workspace, hipStream_t stream) {
    p.log_groups = 0;
    while ((1 << p.log_groups) < p.groups) ++p.log_groups;
    p.pitch = (p.E + 3) / 4 * 4;
    const RoutePlan plan = route_plan(p.T, p.E, p.groups, p.log_groups);
    p.block_tokens = plan.single ? 64 : block_tokens(p.T);
    const int64_t blocks = (p.T + p.block_tokens - 1) / p.block_tokens;
    if (!launch_fits(blocks, kPlaceThreads)) return hipErrorInvalidValue;
    const int n = p.E / p.groups, lanes = plan.G >> p.log_groups, each = (n + lanes - 1) / lanes;
    p.fours = each % 4 == 0 && n % each == 0 && p.ldl % 4 == 0 &&
              (reinterpret_cast<uintptr_t>(p.logits) & (p.bf16 ? 7u : 15u)) == 0;
    p.counts = static_cast<uint8_t *>(workspace);
    if (blocks > kSumBlocks) {
        p.totals = reinterpret_cast<int32_t *>(p.counts + pad16(blocks * p.pitch));
        p.before = reinterpret_cast<int32_t *>(p.counts + pad16(blocks * p.pitch) + pad16(4 * p.pitch));
    }
    hipError_t e;
    if (p.bias)
        e = plan.G == 16   ? by_values<16, true>(plan, p, blocks, stream)
            : plan.G == 32 ? by_values<32, true>(plan, p, blocks, stream)
                           : by_values<64, true>(plan, p, blocks, stream);
    else
        e = plan.G == 16   ? by_values<16, false>(plan, p, blocks, stream)
            : plan.G == 32 ? by_values<32, false>(plan, p, blocks, stream)
                           : by_values<64, false>(plan, p, blocks, stream);
    if (e != hipSuccess || plan.single) return e;
    if (p.before) {
        hipLaunchKernelGGL(column_kernel, dim3((unsigned)(p.pitch / 4)), dim3(256), 0, stream, p, blocks);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(place_kernel, dim3((unsigned)blocks), dim3(kPlaceThreads), 0, stream, p, (int)blocks);
    return hipGetLastError();
}

}  // namespace bi8
