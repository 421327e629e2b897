// Low-rank adapters of many requests beside a shared projection (gfx950):
//
//   t[m, r]  = scales[e] sum_k x[m, k] a[e, r, k]             e = adapter[m]
//   y[m, n] += sum_j t[m, p R + j] b[e, n, j]                 p the part of n
//
//  * lora_shrink_kernel  t, split over K between waves (whose sums meet in LDS)
//                        and workgroups (whose sums meet in the second kernel);
//  * lora_expand_kernel  y, a workgroup for a block of its columns.
//
// Rows and adapters.  Both take 64 rows at a time, one a lane.  The rows of an
// adapter are a ballot of the lanes that hold it, and belong to the first of
// them: a workgroup visits the lanes s, s + slots, ... and does the work of those
// that are the first of their adapter, its rows pushed together to tiles of 16.
// No row is sorted and nothing is kept between calls; rows of one adapter that lie
// next to each other make full tiles.
//
// Matrix core: 16x16x32 bf16 with t's side transposed in both (ranks, then
// columns of y, are rows of the result), so that a lane ends up with neighbouring
// ranks or columns of one row.  t has no bf16 rounding: it is split into hi + lo,
// two bf16 values that hold 16 bits of it, which take the two halves of a longer
// sum over the ranks, each against the same b.
//
// Bound by HBM: x read once, y read and written once, the adapters in use once.
#include "codes.hpp"
#include "internal.hpp"

namespace bi8 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 64;   // of a block of rows: one a lane
constexpr int kShrinkWaves = 8;
constexpr int kExpandWaves = 4;
constexpr int kColumns = 32;   // of a wave at a time

__device__ __forceinline__ f32x4 mfma(const u32x4 &a, const u32x4 &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// The adapter of a block's row on each lane, -1 for none.
__device__ __forceinline__ int adapter_of(const LoraArgs &p, int64_t m0, int lane) {
    const int e = m0 + lane < p.M ? p.adapter[m0 + lane] : -1;
    return e >= 0 && e < p.L ? e : -1;
}

// Whether lane i is the first of its adapter; then its adapter and the lanes that
// hold it, as a list: entry l of `rows` for l < count.  Uniform over the wave.
struct Rows {
    int adapter, count, list;   // list: this lane's entry
};
__device__ __forceinline__ bool rows_of(int mine, int i, int lane, Rows &r) {
    r.adapter = __builtin_amdgcn_readlane(mine, i);
    if (r.adapter < 0) return false;
    const uint64_t members = __ballot(mine == r.adapter);
    if (__ffsll((unsigned long long)members) - 1 != i) return false;
    r.count = __popcll(members);
    const uint64_t lower = (1ull << lane) - 1;
    const bool in = (members >> lane) & 1;
    const int to = in ? __popcll(members & lower) : r.count + __popcll(~members & lower);
    r.list = __builtin_amdgcn_ds_permute(to << 2, lane);
    return true;
}

template <bool ODD>
__device__ __forceinline__ u32x4 load_k(const uint16_t *row, int64_t k, int64_t K) {
    if (k >= K) return u32x4{0u, 0u, 0u, 0u};
    if constexpr (ODD)
        return load_bf16x8(row + k, K - k);
    else
        return *reinterpret_cast<const u32x4 *>(row + k);
}

// J tiles of 16 rows times the NR tiles of 16 ranks from rank0 on, over this
// wave's part of K; the waves' sums meet in LDS, tile by tile.
template <int J, int NR, bool ODD>
__device__ __forceinline__ void shrink_rows(const LoraArgs &p, const Rows &r, int64_t m0, int split, int rank0,
                                            f32x4 *meet) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, at = lane & 15, g = lane >> 4;
    const uint16_t *xrow[J], *arow[NR];
#pragma unroll
    for (int j = 0; j < J; ++j)
        xrow[j] = p.x + (m0 + __shfl(r.list, min(16 * j + at, r.count - 1))) * p.ldx + 8 * g;
#pragma unroll
    for (int f = 0; f < NR; ++f)
        arow[f] = p.a + ((int64_t)r.adapter * p.ranks + min(rank0 + 16 * f + at, p.ranks - 1)) * p.K + 8 * g;
    f32x4 acc[J][NR];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int f = 0; f < NR; ++f) acc[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t first = (int64_t)(split * kShrinkWaves + wave) * p.slice, last = min(first + p.slice, p.K);
    const int64_t end = p.K - 8 * g;   // of this lane's columns
    for (int64_t k = first; k < last; k += 64) {
        u32x4 xv[J][2], av[NR][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < J; ++j) xv[j][h] = load_k<ODD>(xrow[j], k + 32 * h, end);
#pragma unroll
            for (int f = 0; f < NR; ++f) av[f][h] = load_k<ODD>(arow[f], k + 32 * h, end);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int f = 0; f < NR; ++f) acc[j][f] = mfma(av[f][h], xv[j][h], acc[j][f]);
    }
    // meet[wave][row][4 NR quads of ranks], the quads of a row turned against bank conflicts
    constexpr int kQuads = 4 * NR, kTurn = (kQuads < 8 ? kQuads : 8) - 1;
    const float scale = p.scales ? p.scales[r.adapter] : 1.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (16 * j >= r.count) break;
        __syncthreads();
#pragma unroll
        for (int f = 0; f < NR; ++f) meet[(wave * 16 + at) * kQuads + ((4 * f + g) ^ (at & kTurn))] = acc[j][f];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * kQuads; i += 64 * kShrinkWaves) {
            const int row = i / kQuads, quad = i % kQuads;
            const int turned = row * kQuads + (quad ^ (row & kTurn));
            f32x4 s = meet[turned];
#pragma unroll
            for (int w = 1; w < kShrinkWaves; ++w) s += meet[w * 16 * kQuads + turned];
            const int from = __shfl(r.list, 16 * j + row);
            if (16 * j + row < r.count && rank0 + 4 * quad < p.ranks)
                *reinterpret_cast<f32x4 *>(p.t + ((int64_t)split * p.M + m0 + from) * p.ranks + rank0 + 4 * quad) =
                    s * scale;
        }
    }
}

// Workgroup x: slot x % slots of block x / slots; y: split of K; z: 16 NR ranks.
template <int NR, bool ODD>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(LoraArgs p) {
    __shared__ f32x4 meet[kShrinkWaves * 16 * 4 * NR];
    const int lane = threadIdx.x & 63;
    const int64_t m0 = (int64_t)(blockIdx.x / p.slots) * kRows;
    const int mine = adapter_of(p, m0, lane);
    const int rank0 = blockIdx.z * 16 * NR;
    for (int i = blockIdx.x % p.slots; i < kRows; i += p.slots) {
        Rows r;
        if (!rows_of(mine, i, lane, r)) continue;
        if (r.count <= 16)
            shrink_rows<1, NR, ODD>(p, r, m0, blockIdx.y, rank0, meet);
        else if (r.count <= 32)
            shrink_rows<2, NR, ODD>(p, r, m0, blockIdx.y, rank0, meet);
        else
            shrink_rows<4, NR, ODD>(p, r, m0, blockIdx.y, rank0, meet);
    }
}

// The NM matrix products over the ranks of one part: 4 NM chunks of 8, of which
// the first R / 8 are hi, the next R / 8 lo, the rest zero.  TWICE: there is no
// rest, and lo meets the registers of b that hi did.
template <int J, int NM, bool TWICE, bool ODD>
__device__ __forceinline__ void expand_rows(const LoraArgs &p, const Rows &r, int64_t m0, int row0, int64_t n0,
                                            int64_t end, const u32x4 *tile) {
    constexpr int kPitch = 4 * NM + 1;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, at = lane & 15, g = lane >> 4;
    const int chunks = p.R / 8;
    uint16_t *yrow[J];
    bool have[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int i = row0 + 16 * j + at;
        have[j] = i < r.count;
        yrow[j] = p.y + (m0 + __shfl(r.list, min(i, r.count - 1))) * p.ldy;
    }
    const uint16_t *b = p.b + (int64_t)r.adapter * p.N * p.R;
    for (int64_t n = n0 + kColumns * wave; n < end; n += kColumns * kExpandWaves) {
        if (n >= n0 + p.columns) break;
        // result row i of the products x and y: column n + 8 (i / 4) + i % 4, and 4 on
        const int64_t col = n + 8 * g, bx = n + 8 * (at >> 2) + (at & 3);
        const uint16_t *brow[2] = {b + min(bx, end - 1) * p.R, b + min(bx + 4, end - 1) * p.R};
        u32x4 yv[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            yv[j] = u32x4{0u, 0u, 0u, 0u};
            if (have[j] && col < end) {
                if constexpr (ODD)
                    yv[j] = load_bf16x8(yrow[j] + col, end - col);
                else
                    yv[j] = *reinterpret_cast<const u32x4 *>(yrow[j] + col);
            }
        }
        f32x4 acc[J][2];
#pragma unroll
        for (int j = 0; j < J; ++j) acc[j][0] = acc[j][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        u32x4 bv[NM][2];
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            const int q = 4 * i + g, c = q < chunks ? q : q - chunks;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (TWICE && i >= NM / 2)
                    bv[i][h] = bv[i - NM / 2][h];
                else
                    bv[i][h] = c < chunks ? *reinterpret_cast<const u32x4 *>(brow[h] + 8 * c) : u32x4{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int i = 0; i < NM; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const u32x4 tv = tile[(16 * j + at) * kPitch + 4 * i + g];
                acc[j][0] = mfma(bv[i][0], tv, acc[j][0]);
                acc[j][1] = mfma(bv[i][1], tv, acc[j][1]);
            }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (!have[j] || col >= end) continue;
            float f[8];
            unpack_bf16x8(yv[j], f);
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = 2 * i;
                o[i] = f32x2_to_bf16x2_bits(f[e] + acc[j][e >> 2][e & 3], f[e + 1] + acc[j][e >> 2][(e & 3) + 1]);
            }
            if constexpr (ODD)
                store_bf16x8(yrow[j] + col, o, end - col);
            else
                *reinterpret_cast<u32x4 *>(yrow[j] + col) = o;
        }
    }
}

// Workgroup: block of columns, fastest; then slot; then block of rows.
template <int NM, bool TWICE, bool ODD>
__global__ __launch_bounds__(64 * kExpandWaves) void lora_expand_kernel(LoraArgs p) {
    constexpr int kTile = NM > 8 ? 32 : kRows;   // rows of t in LDS at a time
    constexpr int kChunks = 4 * NM, kPitch = kChunks + 1;
    __shared__ u32x4 tile[kTile * kPitch];
    const int lane = threadIdx.x & 63;
    const int column_blocks = p.part_blocks[kMaxParts];
    const int64_t rest = blockIdx.x / column_blocks;
    int cb = blockIdx.x - (int)rest * column_blocks, part = 0;
#pragma unroll
    for (int i = 1; i < kMaxParts; ++i)
        if (cb >= p.part_blocks[i]) part = i;   // (parts that are not there begin past all blocks)
    const int64_t n0 = p.part_first[part] + (int64_t)(cb - p.part_blocks[part]) * p.columns;
    const int64_t end = p.part_first[part + 1];
    const int64_t m0 = rest / p.slots * kRows;
    const int mine = adapter_of(p, m0, lane);
    const int chunks = p.R / 8;
    for (int i = (int)(rest % p.slots); i < kRows; i += p.slots) {
        Rows r;
        if (!rows_of(mine, i, lane, r)) continue;
        for (int row0 = 0; row0 < r.count; row0 += kTile) {
            const int count = min(r.count - row0, kTile);
            __syncthreads();   // the last tile is read
            for (int base = 0; base < count * kChunks; base += 64 * kExpandWaves) {
                const int idx = base + threadIdx.x, row = idx / kChunks, q = idx % kChunks;
                const int from = __shfl(r.list, (row0 + row) & 63);
                if (row >= count) continue;
                if (q < chunks) {
                    const float *t = p.t + (m0 + from) * p.ranks + part * p.R + 8 * q;
                    f32x4 s0 = reinterpret_cast<const f32x4 *>(t)[0], s1 = reinterpret_cast<const f32x4 *>(t)[1];
                    for (int s = 1; s < p.splits; ++s) {
                        t += p.M * p.ranks;
                        s0 += reinterpret_cast<const f32x4 *>(t)[0];
                        s1 += reinterpret_cast<const f32x4 *>(t)[1];
                    }
                    u32x4 hi, lo;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float v0 = w < 2 ? s0[2 * w] : s1[2 * w - 4], v1 = w < 2 ? s0[2 * w + 1] : s1[2 * w - 3];
                        // hi: the upper 16 bits (cut, so that it cannot overflow); lo: what is
                        // left, exact but for its own rounding; none beside an infinity
                        const uint32_t h0 = __float_as_uint(v0) & 0xFFFF0000u, h1 = __float_as_uint(v1) & 0xFFFF0000u;
                        hi[w] = (h0 >> 16) | h1;
                        lo[w] = f32x2_to_bf16x2_bits(isinf(v0) ? 0.0f : v0 - __uint_as_float(h0),
                                                     isinf(v1) ? 0.0f : v1 - __uint_as_float(h1));
                    }
                    tile[row * kPitch + q] = hi;
                    tile[row * kPitch + chunks + q] = lo;
                } else if (q >= 2 * chunks) {
                    tile[row * kPitch + q] = u32x4{0u, 0u, 0u, 0u};
                }
            }
            __syncthreads();
            if (count <= 16)
                expand_rows<1, NM, TWICE, ODD>(p, r, m0, row0, n0, end, tile);
            else if (count <= 32 || kTile == 32)
                expand_rows<2, NM, TWICE, ODD>(p, r, m0, row0, n0, end, tile);
            else
                expand_rows<kTile / 16, NM, TWICE, ODD>(p, r, m0, row0, n0, end, tile);
        }
    }
}

int64_t blocks_of(int64_t M) { return (M + kRows - 1) / kRows; }

// Workgroups that share K, and the columns of a wave's part of it.
int splits_of(int64_t M, int64_t K, int64_t *slice) {
    const int64_t most = (K + 64 * kShrinkWaves - 1) / (64 * kShrinkWaves);
    int64_t splits = 512 / blocks_of(M);
    splits = splits < 1 ? 1 : splits > 16 ? 16 : splits;
    if (splits > most) splits = most;
    const int64_t per = (K + splits * kShrinkWaves - 1) / (splits * kShrinkWaves);
    *slice = (per + 63) / 64 * 64;
    return (int)splits;
}

template <int NR, bool ODD>
hipError_t launch_shrink(const LoraArgs &p, hipStream_t stream) {
    const dim3 grid((unsigned)(blocks_of(p.M) * p.slots), (unsigned)p.splits, (unsigned)((p.ranks + 16 * NR - 1) / (16 * NR)));
    hipLaunchKernelGGL((lora_shrink_kernel<NR, ODD>), grid, dim3(64 * kShrinkWaves), 0, stream, p);
    return hipGetLastError();
}

template <bool ODD>
hipError_t shrink(const LoraArgs &p, hipStream_t stream) {
    if (p.ranks <= 16) return launch_shrink<1, ODD>(p, stream);
    if (p.ranks <= 32) return launch_shrink<2, ODD>(p, stream);
    if (p.ranks <= 64) return launch_shrink<4, ODD>(p, stream);
    return launch_shrink<8, ODD>(p, stream);
}

template <int NM, bool TWICE, bool ODD>
hipError_t launch_expand(const LoraArgs &p, hipStream_t stream) {
    const int64_t groups = blocks_of(p.M) * p.slots * p.part_blocks[kMaxParts];
    if (!launch_fits(groups, 64 * kExpandWaves)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((lora_expand_kernel<NM, TWICE, ODD>), dim3((unsigned)groups), dim3(64 * kExpandWaves), 0, stream, p);
    return hipGetLastError();
}

template <int NM, bool ODD>
hipError_t expand_of(const LoraArgs &p, hipStream_t stream) {
    if constexpr (NM > 1)
        if (p.R / 8 == 2 * NM) return launch_expand<NM, true, ODD>(p, stream);
    return launch_expand<NM, false, ODD>(p, stream);
}

template <bool ODD>
hipError_t expand(const LoraArgs &p, hipStream_t stream) {
    const int products = (2 * (p.R / 8) + 3) / 4;
    if (products <= 1) return expand_of<1, ODD>(p, stream);
    if (products <= 2) return expand_of<2, ODD>(p, stream);
    if (products <= 4) return expand_of<4, ODD>(p, stream);
    if (products <= 8) return expand_of<8, ODD>(p, stream);
    return expand_of<16, ODD>(p, stream);
}

}  // namespace

int64_t lora_workspace_bytes(int64_t M, int64_t K, int32_t ranks) {
    int64_t slice;
    return splits_of(M, K, &slice) * M * ranks * 4;
}

hipError_t launch_lora_add(LoraArgs p, const int64_t *part_columns, int32_t parts, hipStream_t stream) {
    p.splits = splits_of(p.M, p.K, &p.slice);
    const int64_t blocks = blocks_of(p.M);
    p.slots = blocks <= 8 ? 64 : blocks <= 32 ? 16 : 4;
    p.columns = 128;
    while (p.columns < 1024 && blocks * ((p.N + p.columns - 1) / p.columns) >= 2048) p.columns *= 2;
    auto off = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) != 0; };
    bool odd = p.ldy % 8 != 0 || off(p.y);
    int64_t first = 0;
    int32_t block = 0;
    for (int i = 0; i < kMaxParts; ++i) {
        p.part_first[i] = first;
        p.part_blocks[i] = i < parts ? block : INT32_MAX;
        if (i >= parts) continue;
        odd |= part_columns[i] % 8 != 0;
        first += part_columns[i];
        block += (int32_t)((part_columns[i] + p.columns - 1) / p.columns);
    }
    p.part_first[kMaxParts] = first;
    p.part_blocks[kMaxParts] = block;
    if (!launch_fits(blocks * p.slots, 64 * kShrinkWaves)) return hipErrorInvalidValue;
    const bool odd_k = p.K % 8 != 0 || p.ldx % 8 != 0 || off(p.x);
    const hipError_t e = odd_k ? shrink<true>(p, stream) : shrink<false>(p, stream);
    if (e != hipSuccess) return e;
    return odd ? expand<true>(p, stream) : expand<false>(p, stream);
}

}  // namespace bi8
