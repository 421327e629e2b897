// Router of a mixture of experts with scores, a bias for balance and groups, and
// the dispatch order of its tokens (gfx950).
//
//  * route_kernel   a group of G lanes holds a token's logits, V a lane, and takes
//                   the k largest by k reductions of (value, index) over the
//                   lanes.  A workgroup has B <= 64 tokens; a token picks an
//                   expert once at most, so one 64-bit word an expert in LDS,
//                   with a bit a token, is its histogram and, below a token's
//                   bit, that token's place among the workgroup's.
//  * place_kernel   a workgroup for the same B tokens: sums the counts of all
//                   workgroups (an expert's start) and of those before it, and
//                   writes the rows.  One workgroup's tokens are placed by
//                   route_kernel itself.
//  * column_kernel  past kSumBlocks workgroups: those sums, once for all.
//
// Lanes and groups: the experts of a group lie on G / 2^ceil(log2 groups)
// neighbouring lanes, so that a group's value is a reduction over those.
#include <cfloat>
#include <climits>
#include <type_traits>

#include "common.hpp"
#include "internal.hpp"

namespace bi8 {

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 32;
constexpr int kTokens = 16;      // of a workgroup at a time
constexpr int kPlaceThreads = 1024;
constexpr int kSumBlocks = 256;  // workgroups whose counts every workgroup sums by itself

template <int N>
__device__ __forceinline__ int ror(int v) {
    return __builtin_amdgcn_update_dpp(0, v, 0x120 + N, 0xF, 0xF, false);
}
template <int N>
__device__ __forceinline__ float ror(float v) {
    return __int_as_float(ror<N>(__float_as_int(v)));
}
template <int N>
__device__ __forceinline__ double ror(double v) {
    return __hiloint2double(ror<N>(__double2hiint(v)), ror<N>(__double2loint(v)));
}

// op over the G lanes of an aligned group, in every lane of it; op is
// idempotent, so four rotations of a row of 16 lanes cover it.
template <int G, class T, class Op>
__device__ __forceinline__ T reduce(T v, Op op) {
    v = op(v, ror<1>(v));
    v = op(v, ror<2>(v));
    v = op(v, ror<4>(v));
    v = op(v, ror<8>(v));
    if constexpr (G >= 32) v = op(v, __shfl_xor(v, 16));
    if constexpr (G >= 64) v = op(v, __shfl_xor(v, 32));
    return v;
}

template <int G>
__device__ __forceinline__ double sum(double v) {
#pragma unroll
    for (int d = 1; d < G; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// Takes (ov, oi) if it is larger, or equal with a lower index.
template <class T>
__device__ __forceinline__ void take(T &v, int &i, T ov, int oi) {
    const bool better = ov > v || (ov == v && oi < i);
    v = better ? ov : v;
    i = better ? oi : i;
}

template <class T>
__device__ __forceinline__ T larger(T a, T b) {
    return a > b ? a : b;
}
template <class T>
__device__ __forceinline__ T smaller(T a, T b) {
    return a < b ? a : b;
}

// The largest value and its index over the G lanes, in every lane of them.
template <int G, class T>
__device__ __forceinline__ void best_of(T &v, int &i) {
    take(v, i, ror<1>(v), ror<1>(i));
    take(v, i, ror<2>(v), ror<2>(i));
    take(v, i, ror<4>(v), ror<4>(i));
    take(v, i, ror<8>(v), ror<8>(i));
    if constexpr (G >= 32) take(v, i, __shfl_xor(v, 16), __shfl_xor(i, 16));
    if constexpr (G >= 64) take(v, i, __shfl_xor(v, 32), __shfl_xor(i, 32));
}

// A logit's place in the order, as a signed word: -infinity and NaN the lowest,
// +infinity as the largest finite value, both zeros alike; kTaken is below all.
constexpr int32_t kTaken = INT_MIN;
__device__ __forceinline__ int32_t order_of(float l) {
    const float f = (l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY) + 0.0f;
    const int32_t s = __float_as_int(f);
    return s ^ ((s >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float logit_of(int32_t order) {
    return __int_as_float(order ^ ((order >> 31) & 0x7FFFFFFF));
}

// exp(l - m), or 1 / (1 + exp(-l)); 0 for NaN and -infinity.
__device__ __forceinline__ double score_of(float l, float m, bool sigmoid) {
    if (!(l > -INFINITY)) return 0.0;
    const double x = (double)fminf(l, FLT_MAX);
    return sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)m);
}

__device__ __forceinline__ float load_logit(const RouteArgs &p, const void *row, int e) {
    return p.bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(row)[e]) : static_cast<const float *>(row)[e];
}

// Exclusive prefix of counts[0 .. E) over the workgroup into starts, and the
// total: E <= the number of threads.  All threads call it.
__device__ __forceinline__ void scan_experts(int32_t count, int32_t E, int32_t *starts, int32_t *wave_sums,
                                             int32_t *offsets) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int32_t x = count;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t y = __shfl_up(x, d);
        x += lane >= d ? y : 0;
    }
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
                                            uint16_t *picks) {
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
    float l[V];
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = v < count ? load_logit(p, row, e0 + v) : -INFINITY;

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
        double part = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            c[v] = v < count ? score_of(l[v], m, sigmoid) : 0.0;
            part += c[v];
        }
        if (!sigmoid) {
            total = sum<G>(part);
            if (!(total > 0.0)) total = 1.0;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (v < count) {
                const double b = (double)p.bias[e0 + v];
                const double w = (sigmoid ? c[v] : c[v] / total) + b;
                c[v] = w > -DBL_MAX ? fmin(w, DBL_MAX) : -DBL_MAX;   // (NaN: the lowest)
            } else {
                c[v] = taken;
            }
        }
    } else {
        if (!sigmoid && !p.renormalize) {
            double part = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) part += v < count && l[v] > -INFINITY ? (double)expf(fminf(l[v], FLT_MAX) - m) : 0.0;
            total = sum<G>(part);
            if (!(total > 0.0)) total = 1.0;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = v < count ? order_of(l[v]) : taken;
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
        for (int o = 0; o < p.groups; ++o) {
            const double other = __shfl(value, base + o * lanes);
            rank += other > value || (other == value && o < g) ? 1 : 0;
        }
        if (rank >= p.topk_groups) {
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] = taken;
        }
    }

    int id[2] = {0, 0};   // lane j % G keeps pick j
    int last = kNone;
    for (int j = 0; j < p.k; ++j) {
        Val bv = taken;
        int bi = kNone;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            c[v] = e0 + v == last ? taken : c[v];
            const bool better = c[v] > bv;
            bv = better ? c[v] : bv;
            bi = better ? e0 + v : bi;
        }
        best_of<G>(bv, bi);
        last = bi;
        if (lane == (j & (G - 1))) {
            if (j < G)
                id[0] = bi;
            else
                id[1] = bi;
        }
    }
    double w[2], all = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = 0.0;
        if (lane + i * G < p.k) w[i] = score_of(load_logit(p, row, id[i]), m, sigmoid);
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
            picks[t_local * p.k + j] = (uint16_t)id[i];
        }
    }
}

__device__ __forceinline__ int below(uint64_t mask, int t) { return __popcll(mask & ((1ull << t) - 1)); }

// ceil(T / B) workgroups of kTokens groups; SINGLE: one, which places its rows
// too (T = 0 included).
template <int G, int V, bool BIAS, bool SINGLE>
__global__ __launch_bounds__(kTokens *G) void route_kernel(RouteArgs p) {
    __shared__ uint64_t mask[G * kTokens];   // E <= G V <= the number of threads
    __shared__ uint16_t picks[64 * kMaxTop];
    __shared__ int32_t starts[SINGLE ? G * kTokens : 1];
    __shared__ int32_t wave_sums[16];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * p.block_tokens;
    mask[tid] = 0;
    __syncthreads();
    for (int i = tid / G; i < p.block_tokens; i += kTokens)
        if (t0 + i < p.T) route_token<G, V, BIAS>(p, t0 + i, i, tid & (G - 1), mask, picks);
    __syncthreads();
    const int32_t count = tid < p.E ? __popcll(mask[tid]) : 0;
    if constexpr (SINGLE) {
        scan_experts(count, p.E, starts, wave_sums, p.offsets);
        for (int i = tid; i < (int)p.T * p.k; i += kTokens * G) {
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
            for (int b = slice; b < blocks; b += slices) {
                const uint32_t w = counts[b * words + col];
                even += w & 0x00FF00FFu;
                odd += (w >> 8) & 0x00FF00FFu;
                if (b < (int)blockIdx.x) {
                    even_before += w & 0x00FF00FFu;
                    odd_before += (w >> 8) & 0x00FF00FFu;
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

// Lanes a token and values a lane.
struct RouteShape {
    int G, V;
};

RouteShape route_shape(int64_t T, int32_t E, int32_t groups, int log_groups) {
    const int n = E / groups;
    auto values = [&](int G) { return G >> log_groups ? (n + (G >> log_groups) - 1) / (G >> log_groups) : 1 << 20; };
    for (int G : {16, 32, 64}) {
        if (T <= 1024 && G < 64) continue;
        const int v = values(G);
        if (G == 64 && v > 16) return {64, 32};   // 1024 experts in a number of groups that is no power of two
        if (v <= 16) return {G, v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : v <= 8 ? 8 : 16};
    }
    return {0, 0};
}

template <int G, int V, bool BIAS>
hipError_t launch_route(const RouteArgs &p, int64_t blocks, hipStream_t stream) {
    if (blocks <= 1)
        hipLaunchKernelGGL((route_kernel<G, V, BIAS, true>), dim3(1), dim3(kTokens * G), 0, stream, p);
    else
        hipLaunchKernelGGL((route_kernel<G, V, BIAS, false>), dim3((unsigned)blocks), dim3(kTokens * G), 0, stream, p);
    return hipGetLastError();
}

template <int G, bool BIAS>
hipError_t by_values(int V, const RouteArgs &p, int64_t blocks, hipStream_t stream) {
    switch (V) {
        case 1: return launch_route<G, 1, BIAS>(p, blocks, stream);
        case 2: return launch_route<G, 2, BIAS>(p, blocks, stream);
        case 4: return launch_route<G, 4, BIAS>(p, blocks, stream);
        case 8: return launch_route<G, 8, BIAS>(p, blocks, stream);
        case 16: return launch_route<G, 16, BIAS>(p, blocks, stream);
        default:
            if constexpr (G == 64) return launch_route<64, 32, BIAS>(p, blocks, stream);
            return hipErrorInvalidValue;
    }
}

int block_tokens(int64_t T) {
    if (T <= 16) return 16;
    return T <= kSumBlocks * 16 ? 16 : T <= kSumBlocks * 32 ? 32 : 64;
}

int64_t pad16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

int64_t route_grouped_workspace_bytes(int64_t T, int32_t E) {
    const int64_t blocks = (T + block_tokens(T) - 1) / block_tokens(T), pitch = (E + 3) / 4 * 4;
    if (blocks <= 1) return 0;
    const int64_t counts = pad16(blocks * pitch);
    return blocks <= kSumBlocks ? counts : counts + pad16(4 * pitch) + 4 * blocks * pitch;
}

hipError_t launch_moe_route_grouped(RouteArgs p, void *workspace, hipStream_t stream) {
    p.block_tokens = block_tokens(p.T);
    p.log_groups = 0;
    while ((1 << p.log_groups) < p.groups) ++p.log_groups;
    p.pitch = (p.E + 3) / 4 * 4;
    const int64_t blocks = (p.T + p.block_tokens - 1) / p.block_tokens;
    const RouteShape s = route_shape(p.T, p.E, p.groups, p.log_groups);
    if (s.G == 0 || !launch_fits(blocks, kPlaceThreads)) return hipErrorInvalidValue;
    p.counts = static_cast<uint8_t *>(workspace);
    if (blocks > kSumBlocks) {
        p.totals = reinterpret_cast<int32_t *>(p.counts + pad16(blocks * p.pitch));
        p.before = reinterpret_cast<int32_t *>(p.counts + pad16(blocks * p.pitch) + pad16(4 * p.pitch));
    }
    hipError_t e;
    if (p.bias)
        e = s.G == 16   ? by_values<16, true>(s.V, p, blocks, stream)
            : s.G == 32 ? by_values<32, true>(s.V, p, blocks, stream)
                        : by_values<64, true>(s.V, p, blocks, stream);
    else
        e = s.G == 16   ? by_values<16, false>(s.V, p, blocks, stream)
            : s.G == 32 ? by_values<32, false>(s.V, p, blocks, stream)
                        : by_values<64, false>(s.V, p, blocks, stream);
    if (e != hipSuccess || blocks <= 1) return e;
    if (p.before) {
        hipLaunchKernelGGL(column_kernel, dim3((unsigned)(p.pitch / 4)), dim3(256), 0, stream, p, blocks);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(place_kernel, dim3((unsigned)blocks), dim3(kPlaceThreads), 0, stream, p, (int)blocks);
    return hipGetLastError();
}

}  // namespace bi8
