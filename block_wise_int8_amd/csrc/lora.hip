// Low-rank adapters of many requests beside a shared projection (gfx950):
//
//   t[m, r]  = scales[e] sum_k x[m, k] a[e, r, k]             e = adapter[m]
//   y[m, n] += sum_j t[m, p R + j] b[e, n, j]                 p the part of n
//
//  * lora_shrink_kernel  t, split over K between waves (whose sums meet in LDS)
//                        and workgroups (whose sums meet in the second kernel);
//  * lora_expand_kernel  y, a workgroup for a block of its columns.
//
// Rows and adapters.  Both take 64 rows at a time, one a lane; the rows of an
// adapter are a ballot of the lanes that hold it, pushed together to tiles of 16.
// One or more workgroups, the slots, share the adapters of such a block.  No row is
// sorted and nothing is kept between calls; rows of one adapter that lie next to each
// other make full tiles.
//
// Matrix core: 16x16x32 bf16 with t's side transposed in both (ranks, then
// columns of y, are rows of the result), so that a lane ends up with neighbouring
// ranks or columns of one row.  t has no bf16 rounding: it is split into hi + lo,
// two bf16 values that hold 16 bits of it, which take the two halves of a longer
// sum over the ranks, each against the same b.
//
// Long batches are bound by HBM: x read once, y read and written once, the adapters in
// use once.  4096 rows, K = 4096, 28672 columns, rank 64 in 6 runs: 28 to 35 us and
// about 115 (y alone, read and written in the same order, 88).  Short ones are bound by
// their chains of loads: 64 rows of 64 adapters, 6144 columns, rank 16: 8 to 10 and 7
// (25 MB of a, 2.6 to 3.2 TB/s; 12.6 of b and 1.6 of y, 2.0); 1 row 4.6 and 4.8, the
// latency of two launches.
#include <algorithm>

#include "codes.hpp"
#include "internal.hpp"

namespace bi8 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 64;   // of a block of rows: one a lane
constexpr int kShrinkWaves = 8;
constexpr int kExpandWaves = 4;
constexpr int kMaxSplits = 8;   // workgroups that share K
constexpr int kColumns = 32;   // of a wave at a time

__device__ __forceinline__ f32x4 mfma(const u32x4 &a, const u32x4 &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// The thread's place, from here: what is derived from it is formed anew and not kept
// in registers from before a loop.
__device__ __forceinline__ int thread_here() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// The adapter of a block's row on each lane, -1 for none.
__device__ __forceinline__ int adapter_of(const LoraArgs &p, int64_t m0, int lane) {
    const int e = m0 + lane < p.M ? p.adapter[m0 + lane] : -1;
    return e >= 0 && e < p.L ? e : -1;
}

// The adapters of a block, each with the lanes that hold it as a list: entry l for
// l < count.  Uniform over the wave.  Of a few blocks each slot looks at candidates of
// its own: adapters slot, slot + slots, ..., or, where there are more than 64, rows,
// which stand for their adapter if no row before does.  Of many it walks over all in
// the order of their first rows and takes number slot, slot + slots, ..., so that the
// first slot always has work and the second has where an adapter ends (4096 rows of 6
// runs: 128 us against 131, of 200 runs, 4096 columns, 96 against 134; but 16 rows of
// 16 adapters 10.4 against 8.2).
struct Rows {
    int adapter, count, list;   // list: this lane's entry
};
struct Adapters {
    uint64_t left;   // walk: lanes whose adapter has not come yet
    int next;        // candidate; walk: number of the next one, modulo slots
};
__device__ __forceinline__ bool next_rows(const LoraArgs &p, int slots, int slot, int mine, int lane, Adapters &s, Rows &r) {
    uint64_t members;
    for (bool taken = false; !taken;) {
        if (p.walk) {
            if (s.left == 0) return false;
            r.adapter = __builtin_amdgcn_readlane(mine, __ffsll((unsigned long long)s.left) - 1);
            members = __ballot(mine == r.adapter);
            s.left &= ~members;
            taken = s.next == slot;
            s.next = s.next + 1 == slots ? 0 : s.next + 1;
        } else {
            if (s.next >= p.candidates) return false;
            r.adapter = p.by_adapter ? s.next : __builtin_amdgcn_readlane(mine, s.next);
            members = __ballot(mine == r.adapter);
            taken = r.adapter >= 0 && members != 0 &&
                    (p.by_adapter || __ffsll((unsigned long long)members) - 1 == s.next);
            s.next += slots;
        }
    }
    r.count = __popcll(members);
    const uint64_t lower = (1ull << lane) - 1;
    const bool in = (members >> lane) & 1;
    const int to = in ? __popcll(members & lower) : r.count + __popcll(~members & lower);
    r.list = __builtin_amdgcn_ds_permute(to << 2, lane);
    return true;
}

// The rows from entry row0 on, 16 at most.
__device__ __forceinline__ Rows part_of(const Rows &r, int row0, int lane) {
    return {r.adapter, min(r.count - row0, 16), __shfl(r.list, (lane + row0) & 63)};
}

// Lanes.  The matrix core wants row l % 16, chunk l / 16 of a tile of 16 rows of 4
// chunks on lane l, the memory pipe four neighbouring lanes on the four chunks of a
// row (each lane that goes to another row than the one before costs it a cycle: 138 us
// against 128 for the second kernel of 4096 rows, 28672 columns, rank 64).  So memory
// sees lane l at row l / 4, chunk l % 4, and registers change lanes in between.
__device__ __forceinline__ int to_core(int lane) { return (4 * (lane & 15) + (lane >> 4)) << 2; }
__device__ __forceinline__ int to_memory(int lane) { return (16 * (lane & 3) + (lane >> 2)) << 2; }

__device__ __forceinline__ u32x4 change_lanes(int from, const u32x4 &v) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v[i]);
    return o;
}

// Buffers begin at rows or adapters of the wave's, and offsets stay below 2^30 bytes
// (rows are at most 2^23 values apart); at kOobOffset loads give zeros and stores go
// nowhere, so rows and columns that are not there need no branch.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint16_t *base) { return make_rsrc(base, 0x7FFFFFFFu); }
__device__ __forceinline__ u32x4 load_at(__amdgpu_buffer_rsrc_t r, uint32_t offset, int64_t element) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)offset, (int)(2 * element), 0);
}

// Stores have no offset in a scalar register.  A store of four registers goes on reading
// them behind its issue; the compiler keeps writes of them two wait states away, but not
// behind a store with a scalar offset, where it takes them to be free at once.  They are
// not: the next instruction's 2^31 (the offset of a load that is not there) was stored in
// the place of the first register, two values of y as zeros, in a fifth of all calls of
// 333 rows and 5000 columns.
__device__ __forceinline__ void store_at(__amdgpu_buffer_rsrc_t r, uint32_t offset, const u32x4 &v) {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)offset, 0, 0);
}

// J tiles of 16 rows times the wave's NR tiles of 16 ranks from rank0 on, over the
// K columns [first, last) of its slice.  kAhead steps of 32 columns are on their way
// in a ring of registers while the oldest is multiplied.
template <int J, int NR, bool ODD>
__device__ __forceinline__ void shrink_product(const LoraArgs &p, const Rows &r, int64_t m0, int64_t first, int64_t last,
                                               int rank0, f32x4 (&acc)[J][NR]) {
    constexpr int kAhead = 3;
    const int lane = thread_here() & 63, at = lane >> 2, g = lane & 3, core = to_core(lane);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int f = 0; f < NR; ++f) acc[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (first >= last || rank0 >= p.ranks) return;
    const uint16_t *const x = p.x + m0 * p.ldx;
    const uint16_t *const a = p.a + ((int64_t)r.adapter * p.ranks + rank0) * p.K;
    const auto xbuf = buffer(x), abuf = buffer(a);
    uint32_t xoff[J], aoff[NR];   // bytes
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t row = (uint32_t)__shfl(r.list, (16 * j + at) & 63);
        xoff[j] = 16 * j + at < r.count ? row * (uint32_t)p.ldx * 2u + 16u * g : kOobOffset;
    }
#pragma unroll
    for (int f = 0; f < NR; ++f)
        aoff[f] = rank0 + 16 * f + at < p.ranks ? (uint32_t)(16 * f + at) * (uint32_t)p.K * 2u + 16u * g : kOobOffset;
    u32x4 xv[kAhead][J], av[kAhead][NR];
    auto load = [&](int64_t k, int d) __attribute__((always_inline)) {
        if constexpr (ODD) {
            const int64_t left = min(last - k, p.K - k) - 8 * g;   // of the row, from this lane's first column on
            const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < J; ++j)
                xv[d][j] = left > 0 && xoff[j] != kOobOffset ? load_bf16x8(x + k + xoff[j] / 2, left) : zero;
#pragma unroll
            for (int f = 0; f < NR; ++f)
                av[d][f] = left > 0 && aoff[f] != kOobOffset ? load_bf16x8(a + k + aoff[f] / 2, left) : zero;
        } else {   // K % 8 == 0: a chunk is there or not
            const bool in = k + 8 * g < last;
#pragma unroll
            for (int j = 0; j < J; ++j) xv[d][j] = load_at(xbuf, in ? xoff[j] : kOobOffset, k);
#pragma unroll
            for (int f = 0; f < NR; ++f) av[d][f] = load_at(abuf, in ? aoff[f] : kOobOffset, k);
        }
        __builtin_amdgcn_sched_barrier(0);   // in the order that they are waited for
    };
#pragma unroll
    for (int d = 0; d < kAhead; ++d) load(first + 32 * d, d);
    for (int64_t k = first; k < last; k += 32 * kAhead) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {   // (steps past the slice are of zeros)
            u32x4 xc[J];
#pragma unroll
            for (int j = 0; j < J; ++j) xc[j] = change_lanes(core, xv[d][j]);
#pragma unroll
            for (int f = 0; f < NR; ++f) {
                const u32x4 ac = change_lanes(core, av[d][f]);
#pragma unroll
                for (int j = 0; j < J; ++j) acc[j][f] = mfma(ac, xc[j], acc[j][f]);
            }
            load(k + 32 * (kAhead + d), d);
        }
    }
}

// The workgroup's waves are p.rank_waves groups of 16 NR ranks times slices of K,
// whose sums meet in LDS, a tile of rows at a time.
template <int J, int NR, bool ODD>
__device__ __forceinline__ void shrink_rows(const LoraArgs &p, const Rows &r, int64_t m0, int split, f32x4 *meet) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rank_wave = wave % p.rank_waves, slice = wave / p.rank_waves, slices = kShrinkWaves / p.rank_waves;
    f32x4 acc[J][NR];
    const int64_t first = (int64_t)(split * slices + slice) * p.slice;
    shrink_product<J, NR, ODD>(p, r, m0, first, min(first + p.slice, p.K), 16 * NR * rank_wave, acc);
    // meet[wave][row][4 NR quads of ranks], the quads of a row turned against bank conflicts
    constexpr int kQuads = 4 * NR, kTurn = (NR % 2 == 0 ? 8 : 4) - 1;   // (stays within the row)
    const int thread = thread_here(), lane = thread & 63, at = lane & 15, g = lane >> 4;
    const float scale = p.scales ? p.scales[r.adapter] : 1.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (16 * j >= r.count) break;
        __syncthreads();
#pragma unroll
        for (int f = 0; f < NR; ++f) meet[(wave * 16 + at) * kQuads + ((4 * f + g) ^ (at & kTurn))] = acc[j][f];
        __syncthreads();
        for (int base = 0; base < 16 * kQuads * p.rank_waves; base += 64 * kShrinkWaves) {
            const int i = base + thread, quad = i % kQuads, row = i / kQuads & 15, of = i / (16 * kQuads);
            const int from = __shfl(r.list, 16 * j + row);
            const int rank = 16 * NR * of + 4 * quad;
            if (of >= p.rank_waves || 16 * j + row >= r.count || rank >= p.ranks) continue;
            const f32x4 *m = meet + (of * 16 + row) * kQuads + (quad ^ (row & kTurn));
            f32x4 s = m[0];
            for (int w = 1; w < slices; ++w) s += m[w * p.rank_waves * 16 * kQuads];
            *reinterpret_cast<f32x4 *>(p.t + ((int64_t)split * p.M + m0 + from) * p.ranks + rank) = s * scale;
        }
    }
}

// Workgroup: split of K, fastest; then block of rows; then slot.  NARROW: rows are
// taken 16 at a time, in fewer registers, for more waves.
template <int NR, bool NARROW, bool ODD>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(LoraArgs p) {
    __shared__ f32x4 meet[kShrinkWaves * 16 * 4 * NR];
    const int lane = threadIdx.x & 63;
    const uint32_t id = blockIdx.x, rest = id / (uint32_t)p.splits;
    const int split = (int)(id - rest * p.splits);
    const int slot = (int)(rest / (uint32_t)p.blocks);
    const int64_t m0 = (int64_t)(rest - slot * (uint32_t)p.blocks) * kRows;
    const int mine = adapter_of(p, m0, lane);
    Adapters s = {__ballot(mine >= 0), p.walk ? 0 : slot};
    for (Rows r; next_rows(p, p.shrink_slots, slot, mine, lane, s, r);) {
        if constexpr (NARROW) {
            for (int row0 = 0; row0 < r.count; row0 += 16)
                shrink_rows<1, NR, ODD>(p, part_of(r, row0, lane), m0, split, meet);
        } else {
            if (r.count <= 16)
                shrink_rows<1, NR, ODD>(p, r, m0, split, meet);
            else if (r.count <= 32)
                shrink_rows<2, NR, ODD>(p, r, m0, split, meet);
            else
                shrink_rows<4, NR, ODD>(p, r, m0, split, meet);
        }
    }
}

// t of `count` rows from the list's entry row0 on, ranks of one part: the splits
// added, as hi and lo chunks of 8 (hi: chunks [0, R / 8); lo: the next; then zeros).
template <int NM>
__device__ __forceinline__ void fill_tile(const LoraArgs &p, const Rows &r, int64_t m0, int row0, int count, int part,
                                          u32x4 *tile) {
    constexpr int kChunks = 4 * NM, kPitch = kChunks + 1, kBatch = 4;   // splits in flight
    const int thread = thread_here(), quads = p.R / 4;
    const int64_t pitch = p.M * p.ranks / 4;   // of a split, in quads of ranks
    uint2 *const half = reinterpret_cast<uint2 *>(tile);
    for (int base = 0; base < count * quads; base += 64 * kExpandWaves) {
        const int idx = base + thread, row = idx / quads, quad = idx - row * quads;
        const int from = __shfl(r.list, (row0 + row) & 63);
        if (row >= count) continue;
        const f32x4 *t = reinterpret_cast<const f32x4 *>(p.t + (m0 + from) * p.ranks + part * p.R) + quad;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < p.splits; s += kBatch) {
            f32x4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] = t[min(s + i, p.splits - 1) * pitch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (s + i < p.splits) sum += v[i];
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            // hi: the upper 16 bits (cut, so that it cannot overflow); lo: what is left,
            // exact but for its own rounding; none beside an infinity
            hi[w] = __float_as_uint(sum[w]) & 0xFFFF0000u;
            const float left = isinf(sum[w]) ? 0.0f : sum[w] - __uint_as_float(hi[w]);
            lo[w] = __float_as_uint(left);
        }
        const int at = row * 2 * kPitch + quad;
        half[at] = make_uint2((hi[0] >> 16) | hi[1], (hi[2] >> 16) | hi[3]);
        half[at + quads] = make_uint2(f32x2_to_bf16x2_bits(__uint_as_float(lo[0]), __uint_as_float(lo[1])),
                                      f32x2_to_bf16x2_bits(__uint_as_float(lo[2]), __uint_as_float(lo[3])));
    }
    const int empty = kChunks - quads;   // chunks of zeros (hi and lo have quads chunks together)
    for (int i = thread; i < count * empty; i += 64 * kExpandWaves)
        tile[i / empty * kPitch + quads + i % empty] = u32x4{0u, 0u, 0u, 0u};
}

// J tiles of rows times the columns [n0, end) of one part: a wave has 32 at a time,
// NM matrix products each over the 4 NM chunks of `tile`, the next 32 on their way
// meanwhile.  TWICE: the chunks are hi and lo alone, and lo meets the registers of b
// that hi did.
template <int J, int NM, bool TWICE, bool ODD>
__device__ __forceinline__ void expand_rows(const LoraArgs &p, const Rows &r, int64_t m0, int row0, int count, int64_t n0,
                                            int64_t end, const u32x4 *tile) {
    constexpr int kPitch = 4 * NM + 1, kMoved = TWICE ? NM / 2 : NM, kStep = kColumns * kExpandWaves;
    const int thread = thread_here(), lane = thread & 63, at = lane >> 2, g = lane & 3;   // in memory
    const int core = to_core(lane), memory = to_memory(lane);
    const int wave = __builtin_amdgcn_readfirstlane(thread >> 6);
    const int chunks = p.R / 8;
    uint16_t *const y = p.y + m0 * p.ldy + n0;
    const uint16_t *const b = p.b + ((int64_t)r.adapter * p.N + n0) * p.R;
    const auto ybuf = buffer(y), bbuf = buffer(b);
    uint32_t yoff[J];   // bytes
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t row = (uint32_t)__shfl(r.list, (row0 + 16 * j + at) & 63);
        yoff[j] = 16 * j + at < count ? row * (uint32_t)p.ldy * 2u + 16u * g : kOobOffset;
    }
    const int columns = (int)(end - n0);
    // result row i of the two products: column 8 (i / 4) + i % 4 of the step, and 4 on
    const int column = 8 * (at >> 2) + (at & 3);
    struct Step {
        u32x4 y[J], b[kMoved][2];
    };
    auto load = [&](int n, Step &v) __attribute__((always_inline)) {
        const int left = columns - n;   // from the step's first column on
#pragma unroll
        for (int i = 0; i < kMoved; ++i) {
            const int q = 4 * i + g, from = TWICE || q < chunks ? q : q - chunks;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = column + 4 * h < left && (TWICE || from < chunks);
                v.b[i][h] = load_at(bbuf, in ? ((uint32_t)(column + 4 * h) * (uint32_t)p.R + 8u * from) * 2u : kOobOffset,
                                    (int64_t)n * p.R);
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if constexpr (ODD)
                v.y[j] = yoff[j] != kOobOffset && 8 * g < left ? load_bf16x8(y + n + yoff[j] / 2, left - 8 * g)
                                                               : u32x4{0u, 0u, 0u, 0u};
            else
                v.y[j] = load_at(ybuf, 8 * g < left ? yoff[j] : kOobOffset, n);
        }
        __builtin_amdgcn_sched_barrier(0);   // in the order that they are waited for
    };
    auto finish = [&](int n, Step &v) __attribute__((always_inline)) {
        f32x4 acc[J][2];
#pragma unroll
        for (int j = 0; j < J; ++j) acc[j][0] = acc[j][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        int from = (lane & 15) * kPitch + (lane >> 4);
        if (J * NM > 4) asm volatile("" : "+v"(from));   // read again each time: 4 J NM registers would hold it all
#pragma unroll
        for (int i = 0; i < kMoved; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) v.b[i][h] = change_lanes(core, v.b[i][h]);
#pragma unroll
        for (int i = 0; i < NM; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const u32x4 tv = tile[from + 16 * j * kPitch + 4 * i];
                acc[j][0] = mfma(v.b[i % kMoved][0], tv, acc[j][0]);
                acc[j][1] = mfma(v.b[i % kMoved][1], tv, acc[j][1]);
            }
        const int left = columns - n;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            u32x4 d[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) d[h] = change_lanes(memory, __builtin_bit_cast(u32x4, acc[j][h]));
            float f[8];
            unpack_bf16x8(v.y[j], f);
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = f32x2_to_bf16x2_bits(f[2 * i] + __uint_as_float(d[i >> 1][2 * i & 3]),
                                            f[2 * i + 1] + __uint_as_float(d[i >> 1][(2 * i & 3) + 1]));
            if constexpr (ODD) {
                if (yoff[j] != kOobOffset && 8 * g < left) store_bf16x8(y + n + yoff[j] / 2, o, left - 8 * g);
            } else {
                store_at(ybuf, 8 * g < left ? yoff[j] + 2u * n : kOobOffset, o);
            }
        }
    };
    Step one, two;
    int n = kColumns * wave;
    load(n, one);
    for (; n < columns; n += 2 * kStep) {   // (steps past the columns load zeros and store nothing)
        load(n + kStep, two);
        finish(n, one);
        load(n + 2 * kStep, one);
        finish(n + kStep, two);
    }
}

// Workgroup: block of columns, fastest; then block of rows; then slot.  NARROW as
// above.
template <int NM, bool TWICE, bool NARROW, bool ODD>
__global__ __launch_bounds__(64 * kExpandWaves, NM <= 4 ? (NARROW ? 4 : 3) : 2) void lora_expand_kernel(LoraArgs p) {
    constexpr int kTile = NARROW ? 16 : NM > 8 ? 32 : kRows;   // rows of t in LDS at a time
    __shared__ u32x4 tile[kTile * (4 * NM + 1)];
    const int lane = threadIdx.x & 63;
    const int column_blocks = p.part_blocks[kMaxParts];
    const uint32_t id = blockIdx.x, rest = id / (uint32_t)column_blocks;
    const int cb = (int)(id - rest * column_blocks);
    int part = 0;
#pragma unroll
    for (int i = 1; i < kMaxParts; ++i)
        if (cb >= p.part_blocks[i]) part = i;   // (parts that are not there begin past all blocks)
    const int64_t n0 = p.part_first[part] + (int64_t)(cb - p.part_blocks[part]) * p.columns;
    const int64_t end = min(n0 + p.columns, p.part_first[part + 1]);
    const int slot = (int)(rest / (uint32_t)p.blocks);
    const int64_t m0 = (int64_t)(rest - slot * (uint32_t)p.blocks) * kRows;
    const int mine = adapter_of(p, m0, lane);
    Adapters s = {__ballot(mine >= 0), p.walk ? 0 : slot};
    for (Rows r; next_rows(p, p.slots, slot, mine, lane, s, r);) {
        for (int row0 = 0; row0 < r.count; row0 += kTile) {
            const int count = min(r.count - row0, kTile);
            __syncthreads();   // the last tile is read
            fill_tile<NM>(p, r, m0, row0, count, part, tile);
            __syncthreads();
            if constexpr (NARROW) {
                expand_rows<1, NM, TWICE, ODD>(p, r, m0, row0, count, n0, end, tile);
            } else {
                if (count <= 16)
                    expand_rows<1, NM, TWICE, ODD>(p, r, m0, row0, count, n0, end, tile);
                else if (count <= 32 || kTile == 32)
                    expand_rows<2, NM, TWICE, ODD>(p, r, m0, row0, count, n0, end, tile);
                else
                    expand_rows<kTile / 16, NM, TWICE, ODD>(p, r, m0, row0, count, n0, end, tile);
            }
        }
    }
}

int64_t blocks_of(int64_t M) { return (M + kRows - 1) / kRows; }

// Tiles of 16 ranks a wave, and waves that share the ranks.
void rank_shape(int32_t ranks, int *tiles, int *waves) {
    const int all = (ranks + 15) / 16;
    *waves = all <= 4 ? 1 : all <= 8 ? 2 : 4;
    *tiles = (all + *waves - 1) / *waves;
}

// Workgroups that share K, and the columns of a wave's slice of it.
int splits_of(int64_t M, int64_t K, int32_t ranks, int64_t *slice) {
    int tiles, waves;
    rank_shape(ranks, &tiles, &waves);
    const int64_t slices = kShrinkWaves / waves, most = (K + 64 * slices - 1) / (64 * slices);
    int64_t splits = 256 / blocks_of(M);
    splits = splits < 1 ? 1 : splits > kMaxSplits ? kMaxSplits : splits;
    if (splits > most) splits = most;
    const int64_t per = (K + splits * slices - 1) / (splits * slices);
    *slice = (per + 31) / 32 * 32;
    return (int)splits;
}

int64_t shrink_groups(const LoraArgs &p) { return (int64_t)p.blocks * p.shrink_slots * p.splits; }
int64_t expand_groups(const LoraArgs &p) { return (int64_t)p.blocks * p.slots * p.part_blocks[kMaxParts]; }

template <int NR, bool ODD>
hipError_t launch_shrink(const LoraArgs &p, hipStream_t stream) {
    const int64_t groups = shrink_groups(p);
    if (p.narrow)
        hipLaunchKernelGGL((lora_shrink_kernel<NR, true, ODD>), dim3((unsigned)groups), dim3(64 * kShrinkWaves), 0, stream, p);
    else
        hipLaunchKernelGGL((lora_shrink_kernel<NR, false, ODD>), dim3((unsigned)groups), dim3(64 * kShrinkWaves), 0, stream, p);
    return hipGetLastError();
}

template <bool ODD>
hipError_t shrink(const LoraArgs &p, int tiles, hipStream_t stream) {
    switch (tiles) {
        case 1: return launch_shrink<1, ODD>(p, stream);
        case 2: return launch_shrink<2, ODD>(p, stream);
        case 3: return launch_shrink<3, ODD>(p, stream);
        default: return launch_shrink<4, ODD>(p, stream);
    }
}

template <int NM, bool TWICE, bool ODD>
hipError_t launch_expand(const LoraArgs &p, hipStream_t stream) {
    const int64_t groups = expand_groups(p);
    if (p.narrow)
        hipLaunchKernelGGL((lora_expand_kernel<NM, TWICE, true, ODD>), dim3((unsigned)groups), dim3(64 * kExpandWaves), 0,
                           stream, p);
    else
        hipLaunchKernelGGL((lora_expand_kernel<NM, TWICE, false, ODD>), dim3((unsigned)groups), dim3(64 * kExpandWaves), 0,
                           stream, p);
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

int64_t lora_workspace_need(int64_t M, int64_t K, int32_t ranks) {
    int64_t slice;
    return splits_of(M, K, ranks, &slice) * M * ranks * 4;
}

// The most that a batch of up to M rows needs: each number of splits above M's at the
// last batch that has it.
int64_t lora_workspace_bytes(int64_t M, int64_t K, int32_t ranks) {
    int64_t most = lora_workspace_need(M, K, ranks);
    for (int64_t splits = 2; splits <= kMaxSplits; ++splits) {
        const int64_t last = 256 / splits * kRows;
        if (last < M) most = std::max(most, lora_workspace_need(last, K, ranks));
    }
    return most;
}

hipError_t launch_lora_add(LoraArgs p, const int64_t *part_columns, int32_t parts, hipStream_t stream) {
    p.splits = splits_of(p.M, p.K, p.ranks, &p.slice);
    int tiles, rank_waves;
    rank_shape(p.ranks, &tiles, &rank_waves);
    p.rank_waves = rank_waves;
    const int64_t blocks = blocks_of(p.M);
    // 16 rows at a time where an adapter is likely to have no more (64 rows, 64
    // adapters of 48 ranks: 15.0 us against 16.9; but 17.1 against 11.4 where all 64
    // rows have the only one, 22.2 against 14.7 for 512 rows of 8).
    p.narrow = p.M <= 16 || p.M <= 2ll * p.L;
    p.by_adapter = p.L <= kRows;
    p.candidates = p.by_adapter ? p.L : kRows;
    // Workgroups for the adapters of a block: all at once while the grid is small; of
    // long batches few, since one without work costs its launch.
    p.walk = blocks > (p.L <= 16 ? 4 : 16);
    auto slots = [&](int s) { return s < p.candidates ? s : p.candidates; };
    p.slots = slots(blocks <= 2 ? kRows : blocks <= 16 ? 16 : p.by_adapter ? 1 : 4);
    p.shrink_slots = blocks <= 16 ? p.slots : slots(p.by_adapter ? 2 : 4);
    p.blocks = (int32_t)blocks;
    // Columns of a workgroup: more mean fewer sums over the splits (64 rows of their
    // own adapters, N = 6144: 13.4 us with 128, 8.5 256, 6.4 512, 7.1 1024), fewer
    // keep small grids wide (333 rows, N = 5000: 7.5, 6.6, 7.2, 9.3).
    const int64_t active = blocks * (p.slots < p.M ? p.slots : p.M);
    p.columns = 128;
    while (p.columns < 512 && active * ((p.N + 2 * p.columns - 1) / (2 * p.columns)) >= 512) p.columns *= 2;
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
    if (!launch_fits(shrink_groups(p), 64 * kShrinkWaves) || !launch_fits(expand_groups(p), 64 * kExpandWaves))
        return hipErrorInvalidValue;
    const bool odd_k = p.K % 8 != 0 || p.ldx % 8 != 0 || off(p.x);
    const hipError_t e = odd_k ? shrink<true>(p, tiles, stream) : shrink<false>(p, tiles, stream);
    if (e != hipSuccess) return e;
    return odd ? expand<true>(p, stream) : expand<false>(p, stream);
}

}  // namespace bi8
