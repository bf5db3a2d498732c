// lora.hip -- low-rank adapters of many requests at once:
//   shrink: v[t] = A_a x[t] (max_rank numbers a row, in the library's fixed
//     reduction order), a = the row's adapter;
//   expand: out[t] = base[t] + scale_a * (B_a v[t]).
// The shared projection beside them (base = W x), when the call computes it:
//   * up to four rows, and up to 3 tiles of 32 x 32 outputs a compute unit (16
//     with short k): base_few_kernel here, the F32 order;
//   * many rows in the split-16 arithmetic: dense_split16.hip;
//   * else eidm_matmul_id with one expert.  The same bits in each.
//
// An adapter is selected per row as an expert is (mlx-native 0.13.0,
// src/ops/dense_matmul_id_auto.rs: a stack of weights, one id per row).
//
// Two forms of each, with the same bits.  By rows (a decode batch, where
// rows have adapters of their own): a wavefront takes one row and streams its
// adapter.  By tiles (prompts, where many rows share an adapter): the rows are
// sorted by adapter (the library's id -> row map) and 16 rows of one adapter
// read it once.  A decode batch's shared projection and its shrink
// run side by side in one launch.
//
// Bounds.  By tiles the expand is a copy with a few products: the base rows
// in, the results out (16384 x 2048, 268 MB: 62 us, 4.3 TB/s, a copy's rate);
// the shrink reads the rows of x (16384 x 768: 16.5 us).  A few rows'
// projection is bound by what a compute unit takes in through its first-level
// cache, f32 rows and 16-bit weights: 32 x 1536 x 4096 moves 393 KB per unit in
// 12 us, the products alone would take 3.5 (with the shrink beside it 14.8 us,
// the expand 5.4).  One row of 4096 x 4096: 34 MB in 9.6 us (3.5 TB/s), two
// thirds of it the stream, the rest its start and end.
#include <algorithm>

#include "eidm.h"
#include "eidm_device.hpp"
#include "eidm_internal.hpp"
#include "few_map.hpp"
#include "few_rows.hpp"
#include "rows16.hpp"

namespace eidm {
namespace {

constexpr uint32_t kXcds = 8;

__device__ __forceinline__ uint32_t rank_of(const LoraArgs& a, uint32_t id) {
    return a.ranks ? min(a.ranks[id], a.max_rank) : a.max_rank;
}

__device__ __forceinline__ float scale_of(const LoraArgs& a, uint32_t id) { return a.scales ? a.scales[id] : 1.0f; }

// ids of the shared projection (one expert), written beside other work
__device__ __forceinline__ void write_zero_ids(const LoraArgs& a) {
    if (a.zero_ids)
        for (uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i < a.m; i += (uint64_t)gridDim.x * blockDim.x)
            a.zero_ids[i] = 0;
}

// Work of one block of 256 of the `blocks` that share row t: wavefront w takes
// the groups of four ranks block + blocks * (w, w + 4, ...); the row is staged
// in LDS.
template <int DT>
__device__ __forceinline__ void shrink_row(const LoraArgs& a, uint32_t t, uint32_t block, uint32_t blocks, float* xs) {
    const uint32_t q = threadIdx.x & 3;
    const uint32_t id = a.ids[t];
    if (id >= a.n_adapters) return;
    const uint32_t rank = rank_of(a, id);
    if (block * 4 >= rank) return;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t step = 16 * blocks;  // ranks between a wavefront's groups
    uint32_t i0 = 4 * (block + blocks * wave);
    auto weights_at = [&](uint32_t i, const uint8_t* (&to)[1]) {
        to[0] = a.a + (size_t)id * a.a_stride + (size_t)min(i + q, rank - 1) * a.k * DtypeSize<DT>::value;
    };
    const uint8_t* wrow[1];
    weights_at(i0, wrow);
    FewStream<DT, 1, DtypeSize<DT>::value == 4 ? 4 : 8, false> w;
    auto stage = few_stage<8>(xs, 1, a.k, [&](uint32_t) { return a.x + (size_t)t * a.k; });
    stage.issue();  // ahead of the weights: a thread's loads return in order
    w.start(wrow, (int)a.k);  // in every wavefront: behind a branch, the rows' wait would be for the weights too
    stage.finish();
    __syncthreads();
    while (i0 < rank) {  // wave-uniform
        auto emit = [&](uint32_t, const float (&v)[1]) {
            if (i0 + q < rank) a.v[(size_t)t * a.v_stride + i0 + q] = v[0];
        };
        auto row = [](uint32_t) { return 0; };
        const uint8_t* next[1] = {wrow[0]};
        if (i0 + step < rank) {
            weights_at(i0 + step, next);
            few_rows_tile<0, true>(w, wrow, next, xs, 0, 1, (int)a.k, row, emit);
            wrow[0] = next[0];
        } else {
            few_rows_tile<0, false>(w, wrow, next, xs, 0, 1, (int)a.k, row, emit);
        }
        i0 += step;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void shrink_row_kernel(LoraArgs a, uint32_t parts) {
    extern __shared__ __align__(16) float xs[];
    write_zero_ids(a);
    shrink_row<DT>(a, blockIdx.x / parts, blockIdx.x % parts, parts, xs);
}

// The shared projection (a.out = W x) and, in the last `shrinks` blocks of
// the same launch, the row form's shrink, which needs none of it.  CT = 0:
// RT row groups staged in LDS (0: one row, 1: up to four), each wavefront four
// columns; else blocks of 16*RT rows by 16*CT columns.
template <int DT, int RT, int CT>
__global__ __launch_bounds__(256) void base_few_kernel(LoraArgs a, const uint8_t* weights, uint32_t shrinks,
                                                       uint32_t parts) {
    extern __shared__ __align__(16) float xs[];
    const uint32_t block = blockIdx.x, bases = gridDim.x - shrinks, lane = threadIdx.x & 63;
    if (block >= bases) {
        shrink_row<DT>(a, (block - bases) / parts, (block - bases) % parts, parts, xs);
        return;
    }
    if constexpr (CT == 0) {
        const uint32_t q = lane & 3, col = block * 16 + (threadIdx.x >> 6) * 4 + q;
        const uint8_t* const wrow[1] = {weights + (size_t)min(col, a.n - 1) * a.k * DtypeSize<DT>::value};
        FewStream<DT, 1, DtypeSize<DT>::value == 4 ? 4 : 8, true> w;
        auto stage = few_stage<8>(xs, a.m, a.k, [&](uint32_t t) { return a.x + (size_t)t * a.k; });
        stage.issue();
        w.start(wrow, (int)a.k);
        stage.finish();
        __syncthreads();
        if (col - q >= a.n) return;  // wave-uniform
        few_rows_tile<RT, false>(w, wrow, wrow, xs, few_row_floats(a.k), a.m, (int)a.k, [](uint32_t i) { return i; },
                                 [&](uint32_t t, const float (&v)[1]) {
                                     if (col < a.n) a.out[(size_t)t * a.n + col] = v[0];
                                 });
    } else {
        // each XCD (blocks are dealt to them in turn) takes an equal share of
        // the tiles, the row tiles of a column tile one after the other, so
        // that its L2 serves the weights to all but the first
        const uint32_t rtiles = (a.m + 16 * RT - 1) / (16 * RT), i = lane & 15;
        const uint32_t tile = block % kXcds * (bases / kXcds) + block / kXcds;
        const uint32_t col0 = tile / rtiles * 16 * CT, row0 = tile % rtiles * 16 * RT;
        if (col0 >= a.n) return;  // past the last tile
        const uint8_t* wrow[CT];
        const float* xrow[RT];
#pragma unroll
        for (int c = 0; c < CT; ++c)
            wrow[c] = weights + (size_t)min(col0 + c * 16 + i, a.n - 1) * a.k * DtypeSize<DT>::value;
#pragma unroll
        for (int t = 0; t < RT; ++t) xrow[t] = a.x + (size_t)min(row0 + t * 16 + i, a.m - 1) * a.k;
        float total[RT][CT];
        rows16_product<DT, RT, CT, RT * CT <= 2 ? 4 : 2>(wrow, xrow, (int)a.k, xs, total);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const uint32_t r = row0 + t * 16 + 4 * (lane >> 4) + (threadIdx.x >> 6);
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (r < a.m && col0 + c * 16 + i < a.n) a.out[(size_t)r * a.n + col0 + c * 16 + i] = total[t][c];
        }
    }
}

// The sorted rows in tiles: 16 rows of one adapter each (fewer in an adapter's
// last).  Adapter a's tiles start at slot offsets[a] / 16 + a, which leaves
// room for every partial tile before it without counting them; a slot behind
// an adapter's last tile is empty.  Id n_adapters: the rows without an adapter.
struct Tile {
    uint32_t id, at, count;  // adapter, first sorted row, rows (0: empty slot)
};

__device__ __forceinline__ Tile tile_of(const LoraArgs& a, uint32_t slot) {
    const uint32_t lane = threadIdx.x & 63;
    uint32_t before = 0;  // ids whose first slot is at or before this one
    for (uint32_t i0 = 0; i0 <= a.n_adapters; i0 += 64) {
        const uint32_t i = min(i0 + lane, a.n_adapters);
        before += (uint32_t)__popcll(__ballot(i0 + lane <= a.n_adapters && a.offsets[i] / 16 + i <= slot));
    }
    const uint32_t id = (uint32_t)__builtin_amdgcn_readfirstlane((int)before) - 1;  // id 0 starts at slot 0
    const uint32_t begin = a.offsets[id], end = a.offsets[id + 1];
    const uint32_t at = begin + (slot - (begin / 16 + id)) * 16;
    return {id, at, at < end ? min(end - at, 16u) : 0u};
}

// A tile as the shrink leaves it for the expand: id << 5 | count, then the 16
// rows (the last one repeated) from word 4 on.
constexpr uint32_t kTileWords = 20;

// One block per (slot, 16*CT ranks).
template <int DT, int CT>
__global__ __launch_bounds__(256, 5 - CT - (DT == kDtypeF32)) void shrink_tile_kernel(LoraArgs a, uint32_t chunks) {
    __shared__ __align__(16) float xs[rows16_lds(CT)];
    const uint32_t lane = threadIdx.x & 63, i = lane & 15;
    write_zero_ids(a);
    const uint32_t slot = blockIdx.x / chunks, c0 = blockIdx.x % chunks * 16 * CT;
    const Tile t = tile_of(a, slot);
    const uint32_t row = t.count ? a.rows[t.at + min(i, t.count - 1)] : 0;
    if (c0 == 0 && threadIdx.x < 16) {
        uint32_t* entry = a.tiles + (size_t)slot * kTileWords;
        if (i == 0) entry[0] = t.id << 5 | t.count;
        entry[4 + i] = row;
    }
    if (!t.count || t.id == a.n_adapters) return;  // block-uniform
    const uint32_t rank = rank_of(a, t.id);
    if (c0 >= rank) return;
    const float* const xrow[1] = {a.x + (size_t)row * a.k};
    const uint8_t* wrow[CT];
#pragma unroll
    for (uint32_t c = 0; c < CT; ++c)
        wrow[c] = a.a + (size_t)t.id * a.a_stride + (size_t)min(c0 + 16 * c + i, rank - 1) * a.k * DtypeSize<DT>::value;
    float total[1][CT];
    rows16_product<DT, 1, CT, 4>(wrow, xrow, (int)a.k, xs, total);
    const uint32_t r = 4 * (lane >> 4) + (threadIdx.x >> 6);
    const uint32_t to = (uint32_t)__shfl((int)row, (int)r);
#pragma unroll
    for (uint32_t c = 0; c < CT; ++c)
        if (r < t.count && c0 + 16 * c + i < rank) a.v[(size_t)to * a.v_stride + c0 + 16 * c + i] = total[0][c];
}

// Ranks i0 .. i0+7 of one row of B, widened; those past max_rank are not read.
template <int DT>
__device__ __forceinline__ void load_b(const uint8_t* row, uint32_t i0, uint32_t max_rank, float (&b)[kGranule]) {
    constexpr int S = DtypeSize<DT>::value;
    if (i0 + kGranule <= max_rank) {
        fr_u32x4 p[S / 2];
#pragma unroll
        for (int h = 0; h < S / 2; ++h) p[h] = *reinterpret_cast<const fr_u32x4_a2*>(row + (size_t)i0 * S + 16 * h);
        few_widen<DT>(p, b);
    } else {
        load_weight_granule<DT>(row, (int)i0, (int)max_rank, true, false, b);
    }
}

// One thread per output: the row's adapter alone, 32 ranks' loads at once.
// Latency bound (id, then B, then the sums): the first loads do not wait for
// the row's rank, so up to 32 ranks they may take elements past it.
template <int DT>
__global__ __launch_bounds__(256) void expand_row_kernel(LoraArgs a) {
    constexpr uint32_t kBatch = 4;
    const uint32_t groups = (a.n + 255) / 256;
    for (uint64_t job = blockIdx.x; job < (uint64_t)a.m * groups; job += gridDim.x) {
        const uint64_t t = job / groups;
        const uint32_t j = (uint32_t)(job % groups) * 256 + threadIdx.x;
        if (j >= a.n) continue;
        const uint32_t id = a.ids[t];
        float y = a.base[t * a.n + j];
        if (id < a.n_adapters) {
            const uint8_t* row = a.b + (size_t)id * a.b_stride + (size_t)j * a.max_rank * DtypeSize<DT>::value;
            float b[kBatch][kGranule];
            auto load = [&](uint32_t i0) {
#pragma unroll
                for (uint32_t h = 0; h < kBatch; ++h)
                    if (i0 + h * kGranule < a.max_rank) load_b<DT>(row, i0 + h * kGranule, a.max_rank, b[h]);
            };
            load(0);
            const uint32_t rank = rank_of(a, id);
            const float* v = a.v + t * a.v_stride;
            float u = 0.0f;
            for (uint32_t i0 = 0; i0 < rank;) {
#pragma unroll
                for (uint32_t h = 0; h < kBatch; ++h) {
                    const float* vh = v + i0 + h * kGranule;
                    if (i0 + (h + 1) * kGranule <= rank) {
#pragma unroll
                        for (uint32_t i = 0; i < kGranule; ++i) u = fma_step(vh[i], b[h][i], u);
                    } else {  // the granule that the rank ends in
                        for (uint32_t i = 0; i0 + h * kGranule + i < rank; ++i) {
                            u = fma_step(vh[i], b[h][0], u);
#pragma unroll
                            for (uint32_t e = 0; e + 1 < kGranule; ++e) b[h][e] = b[h][e + 1];
                        }
                    }
                }
                i0 += kBatch * kGranule;
                if (i0 < rank) load(i0);
            }
            if (rank) y = fma_step(scale_of(a, id), u, y);
        } else if (id != EIDM_NO_ADAPTER) {
            y = quiet_nan();
        }
        a.out[t * a.n + j] = y;
    }
}

// One block per (slot, 256 columns), 64 columns per wavefront.
// v_mfma_f32_16x16x1_4b_f32, one rank per step: all four blocks take the 16
// rows of v, block s the columns 4i+s, so a lane's results are four
// consecutive columns of four rows.  The base rows dominate: their addresses
// wait for the tile's entry alone.
template <int DT>
__global__ __launch_bounds__(256) void expand_tile_kernel(LoraArgs a, uint32_t parts) {
    const uint32_t lane = threadIdx.x & 63, i = lane & 15, s = lane >> 4;
    const uint32_t* entry = a.tiles + (size_t)(blockIdx.x / parts) * kTileWords;
    const uint32_t j0 = (blockIdx.x % parts * 4 + (threadIdx.x >> 6)) * 64 + 4 * i;  // this lane's columns j0 .. j0+3
    const uint32_t id = entry[0] >> 5, count = entry[0] & 31;
    if (!count || j0 - 4 * i >= a.n) return;  // wave-uniform
    uint32_t row[4];  // this lane's rows 4s .. 4s+3
#pragma unroll
    for (uint32_t v = 0; v < 4; ++v) row[v] = entry[4 + 4 * s + v];
    const float* v_row = a.v + (size_t)entry[4 + i] * a.v_stride;
    f32x4 y[4];
#pragma unroll
    for (uint32_t v = 0; v < 4; ++v) {
        const float* p = a.base + (size_t)row[v] * a.n + j0;
        if (j0 + 4 <= a.n) y[v] = *reinterpret_cast<const fr_f32x4_a4*>(p);
        else
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) y[v][c] = j0 + c < a.n ? p[c] : 0.0f;
    }
    if (id < a.n_adapters) {  // wave-uniform
        const uint32_t rank = rank_of(a, id);
        const uint32_t col = min(j0 + s, a.n - 1);  // this lane's column of B
        const uint8_t* b_row = a.b + (size_t)id * a.b_stride + (size_t)col * a.max_rank * DtypeSize<DT>::value;
        f32x16 u{};
        for (uint32_t i0 = 0; i0 < rank; i0 += kGranule) {
            float b[kGranule];
            load_b<DT>(b_row, i0, a.max_rank, b);
            const f32x4 v0 = *reinterpret_cast<const f32x4*>(v_row + i0);
            const f32x4 v1 = *reinterpret_cast<const f32x4*>(v_row + i0 + 4);
#pragma unroll
            for (uint32_t e = 0; e < kGranule; ++e)
                if (i0 + e < rank)  // wave-uniform
                    u = __builtin_amdgcn_mfma_f32_16x16x1f32(e < 4 ? v0[e % 4] : v1[e % 4], b[e], u, 0, 0, 0);
        }
        if (rank) {
            const float scale = scale_of(a, id);
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r)
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) y[r][c] = fma_step(scale, u[4 * c + r], y[r][c]);
        }
    }
#pragma unroll
    for (uint32_t v = 0; v < 4; ++v) {
        if (4 * s + v >= count) continue;
        if (id == a.n_adapters && a.ids[row[v]] != EIDM_NO_ADAPTER)
            y[v] = f32x4{quiet_nan(), quiet_nan(), quiet_nan(), quiet_nan()};
        float* p = a.out + (size_t)row[v] * a.n + j0;
        if (j0 + 4 <= a.n) *reinterpret_cast<fr_f32x4_a4*>(p) = y[v];
        else
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c)
                if (j0 + c < a.n) p[c] = y[v][c];
    }
}

// Slots of the tiles of m sorted rows.
uint64_t lora_slots(uint32_t m, uint32_t n_adapters) { return (uint64_t)m / 16 + n_adapters + 1; }

uint32_t grid_of(uint64_t blocks, uint64_t most) { return (uint32_t)(blocks < most ? blocks : most); }

constexpr uint32_t kRowLds = 64 * 1024;  // LDS of staged rows

bool stages_rows(uint32_t rows, uint32_t k) { return (uint64_t)rows * few_row_floats(k) * 4 <= kRowLds; }

// the projection's form that stages all rows (base_few_kernel, CT = 0)
bool few_rows_staged(const LoraArgs& a) { return a.m <= 4 && stages_rows(a.m, a.k); }

template <int DT>
hipError_t shrink_dt(const LoraArgs& a, int device_cus, hipStream_t stream) {
    const uint32_t parts = (a.max_rank + 15) / 16;
    if (!a.rows) {
        const uint32_t lds = few_row_floats(a.k) * 4;
        hipLaunchKernelGGL(shrink_row_kernel<DT>, dim3(a.m * parts), dim3(256), lds, stream, a, parts);
        return launched(EIDM_KERNEL_LORA_SHRINK, a.m * parts, 256, lds);
    }
    // 32 ranks a block read the rows half as often; 16 while the blocks are
    // fewer than the compute units
    // (2048 rows, k 4096, rank 32, 290 blocks: 21.5 against 29 us; 800 rows of
    // it, 118 blocks, the whole call: 30.5 against 26.7)
    const uint64_t slots = lora_slots(a.m, a.n_adapters);
    if (parts > 1 && slots * parts > (uint64_t)device_cus) {
        const uint32_t chunks = (parts + 1) / 2, grid = (uint32_t)(slots * chunks);
        hipLaunchKernelGGL((shrink_tile_kernel<DT, 2>), dim3(grid), dim3(256), 0, stream, a, chunks);
        return launched(EIDM_KERNEL_LORA_SHRINK, grid, 256, 0);
    }
    const uint32_t grid = (uint32_t)(slots * parts);
    hipLaunchKernelGGL((shrink_tile_kernel<DT, 1>), dim3(grid), dim3(256), 0, stream, a, parts);
    return launched(EIDM_KERNEL_LORA_SHRINK, grid, 256, 0);
}

// Blocks per row of a shrink beside `bases` blocks of the projection.  A
// compute unit left to the shrink alone does not delay a tile, so the rows
// share those that the tiles leave; without enough of them a few rows take a
// block per four ranks, which adds least to each tile it runs beside, and
// more rows one per 16 (each block stages its row).
uint32_t shrink_parts(const LoraArgs& a, uint32_t bases, uint32_t cus) {
    const uint32_t groups = (a.max_rank + 3) / 4, left = bases < cus ? (cus - bases) / a.m : 0;
    if (left) return groups < left ? groups : left;
    return a.m <= 4 ? groups : (groups + 3) / 4;
}

template <int DT, int RT, int CT>
hipError_t base_few(const LoraArgs& a, const uint8_t* weights, bool with_shrink, uint32_t cus, hipStream_t stream) {
    constexpr uint32_t C = CT ? 16 * CT : 16, R = CT ? 16 * RT : 1;
    const uint32_t ctiles = (a.n + C - 1) / C, rtiles = (a.m + R - 1) / R;
    const uint32_t blocks = CT ? (ctiles * rtiles + kXcds - 1) / kXcds * kXcds : ctiles;
    const uint32_t parts = shrink_parts(a, ctiles * rtiles, cus), shrinks = with_shrink ? a.m * parts : 0;
    uint32_t lds = CT ? rows16_lds(RT * CT) * 4 : a.m * few_row_floats(a.k) * 4;
    if (with_shrink && lds < few_row_floats(a.k) * 4) lds = few_row_floats(a.k) * 4;
    hipLaunchKernelGGL((base_few_kernel<DT, RT, CT>), dim3(shrinks + blocks), dim3(256), lds, stream, a, weights,
                       shrinks, parts);
    return launched(EIDM_KERNEL_LORA_BASE, shrinks + blocks, 256, lds);
}

// Relative time of the busiest compute unit when the tiles of 16*rt x 16*ct
// are spread evenly, `each` the time of one.
uint64_t makespan(const LoraArgs& a, uint32_t rt, uint32_t ct, uint32_t each, uint32_t cus) {
    const uint64_t tiles = ((uint64_t)a.m + 16 * rt - 1) / (16 * rt) * ((a.n + 16 * ct - 1) / (16 * ct));
    return (tiles + cus - 1) / cus * each;
}

template <int DT>
hipError_t base_few_dt(const LoraArgs& a, const uint8_t* weights, bool with_shrink, int device_cus, hipStream_t stream) {
    const uint32_t cus = device_cus > 0 ? (uint32_t)device_cus : 256;
    if (few_rows_staged(a))
        return a.m == 1 ? base_few<DT, 0, 0>(a, weights, with_shrink, cus, stream)
                        : base_few<DT, 1, 0>(a, weights, with_shrink, cus, stream);
    // larger tiles read less per product, smaller ones spread more evenly; one
    // tile of each kind per compute unit takes 13, 17, 24 and 32 us at k = 4096
    const uint64_t one = makespan(a, 1, 1, 13, cus), two = makespan(a, 1, 2, 17, cus), four = makespan(a, 2, 2, 24, cus),
                   six = makespan(a, 2, 3, 32, cus);
    const uint64_t least = std::min({one, two, four, six});
    if (one == least) return base_few<DT, 1, 1>(a, weights, with_shrink, cus, stream);
    if (two == least) return base_few<DT, 1, 2>(a, weights, with_shrink, cus, stream);
    return four == least ? base_few<DT, 2, 2>(a, weights, with_shrink, cus, stream)
                         : base_few<DT, 2, 3>(a, weights, with_shrink, cus, stream);
}

template <int DT>
hipError_t expand_dt(const LoraArgs& a, int device_cus, hipStream_t stream) {
    if (!a.rows) {
        const uint32_t grid = grid_of((uint64_t)a.m * ((a.n + 255) / 256), (uint64_t)device_cus * 32);
        hipLaunchKernelGGL(expand_row_kernel<DT>, dim3(grid), dim3(256), 0, stream, a);
        return launched(EIDM_KERNEL_LORA_EXPAND, grid, 256, 0);
    }
    const uint32_t parts = (a.n + 255) / 256, grid = (uint32_t)(lora_slots(a.m, a.n_adapters) * parts);
    hipLaunchKernelGGL(expand_tile_kernel<DT>, dim3(grid), dim3(256), 0, stream, a, parts);
    return launched(EIDM_KERNEL_LORA_EXPAND, grid, 256, 0);
}

}  // namespace

// By rows, every row reads its own adapter; sorted, there are a map and a slot
// per adapter, whether it has rows or not, in both launches. A row weighs its
// adapter's bytes, B's short rows three times A's, and a part of its own. Over
// 2260 calls (65 - 8192 rows, rank 1 - 256, 1 - 2048 adapters, with a projection
// beside them and on given rows, scattered ids and runs) the chosen form takes
// 0.9 % more than the better one on average, 60 % at most. Given rows, bf16, us,
// by rows : sorted: 200 x 128 x 512, rank 64, 32 adapters 12 : 18, 256 adapters
// 12 : 22, 2048 adapters 13 : 77; 400 x 3000 x 200, rank 64, 256 adapters 55 : 28;
// 1600 x 4096 x 4096, rank 4, 32 adapters 58 : 31; rank 64, 2048 adapters 262 : 135.
bool lora_sorts_rows(uint32_t m, uint32_t n, uint32_t k, uint32_t n_adapters, uint32_t max_rank) {
    if (!stages_rows(1, k)) return true;  // the row form stages a row
    const double rows = m * ((max_rank + 8) * (3.0 * n + k) + 15e3);
    const double slots = (double)n_adapters * ((max_rank + 31) / 32 + (n + 255) / 256);  // blocks of empty slots
    return m > kLoraRowForm && rows > 70e6 + 24e3 * slots;
}

hipError_t launch_lora_shrink(const LoraArgs& a, int device_cus, hipStream_t stream) {
    switch (a.dtype) {
    case kDtypeF32: return shrink_dt<kDtypeF32>(a, device_cus, stream);
    case kDtypeF16: return shrink_dt<kDtypeF16>(a, device_cus, stream);
    case kDtypeBF16: return shrink_dt<kDtypeBF16>(a, device_cus, stream);
    default: return hipErrorInvalidValue;
    }
}

// Up to four rows staged in LDS: at any n (k 4096, bf16, us, this : the
// library's Direct or Grouped kernels: 1 x 32768 45 : 53, 2 x 32768 48 : 77,
// 4 x 65536 125 : 133; k 512, 4 x 65536 31 : 34). More rows: the Grouped kernels,
// which share activations through LDS, take over where 32x32 tiles fill the
// device more than three times and long products make up for their map and
// their other launches (some 9 us). Over 440 products (5 - 16384 rows, 128 - 4096
// tiles, k 64 - 4096, bf16 and f32) the chosen one takes 0.9 % more than the
// better one on average, 27 % at most: bf16, 512 x 2048, k 768 35 : 44, k 4096
// 112 : 110; 1024 x 4096, k 64 31 : 44; 2048 x 1024, k 4096 209 : 194; 512 x 1536,
// k 4096 72 : 100.
bool lora_base_few_supported(const LoraArgs& a, int device_cus) {
    if (few_rows_staged(a) && (a.n + 15) / 16 < (1u << 23)) return true;  // (a grid of below 2^32 threads)
    const uint64_t cus = device_cus > 0 ? (uint64_t)device_cus : 256;
    const uint64_t tiles = ((uint64_t)a.m + 31) / 32 * (((uint64_t)a.n + 31) / 32);
    return tiles <= cus * 3 || (tiles <= cus * 16 && tiles * ((uint64_t)a.k + 500) <= cus * 23400);
}

hipError_t launch_lora_base_few(const LoraArgs& a, int weight_dtype, const uint8_t* weights, int device_cus,
                                hipStream_t stream) {
    const bool together = weight_dtype == a.dtype && !a.rows;
    if (!together) {
        const hipError_t err = launch_lora_shrink(a, device_cus, stream);
        if (err != hipSuccess) return err;
    }
    switch (weight_dtype) {
    case kDtypeF32: return base_few_dt<kDtypeF32>(a, weights, together, device_cus, stream);
    case kDtypeF16: return base_few_dt<kDtypeF16>(a, weights, together, device_cus, stream);
    case kDtypeBF16: return base_few_dt<kDtypeBF16>(a, weights, together, device_cus, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_lora_expand(const LoraArgs& a, int device_cus, hipStream_t stream) {
    switch (a.dtype) {
    case kDtypeF32: return expand_dt<kDtypeF32>(a, device_cus, stream);
    case kDtypeF16: return expand_dt<kDtypeF16>(a, device_cus, stream);
    case kDtypeBF16: return expand_dt<kDtypeBF16>(a, device_cus, stream);
    default: return hipErrorInvalidValue;
    }
}

// ------------------------------------------------------------------ C ABI
namespace {

uint64_t align256(uint64_t v) { return (v + 255) & ~uint64_t(255); }

uint32_t size_of(int dtype) { return dtype == EIDM_DTYPE_F32 ? 4 : 2; }

struct LoraSizes {
    uint64_t weights, a, b;                   // extents needed, bytes
    // scratch: v | sort (histograms, counts, offsets, rows, tiles) | ids of the shared
    // projection | its own scratch
    uint64_t off_hist, off_counts, off_offsets, off_rows, off_tiles, off_ids, off_matmul, matmul, total;
    uint32_t v_stride;
};

eidm_shape shared_projection(const eidm_lora_shape* f) {
    eidm_shape s{};
    s.struct_size = sizeof(eidm_shape);
    s.weight_dtype = f->weight_dtype;
    s.m = f->m;
    s.n = f->n;
    s.k = f->k;
    s.top_k = 1;
    s.n_experts = 1;
    s.arith = f->arith;
    s.expert_stride_bytes = (uint64_t)f->n * f->k * size_of(f->weight_dtype);
    s.input_layout = EIDM_LAYOUT_SHARED_PER_TOKEN;
    s.id_multiplicity = EIDM_IDS_DISTINCT_PER_TOKEN;
    return s;
}

// One stack of adapter matrices [rows, cols]: eidm_matmul_id's checks of a
// stack of experts (dimensions, stride, overflow) for m rows.
int adapter_extent(const eidm_lora_shape* f, bool b, uint64_t* bytes) {
    eidm_shape s{};
    s.struct_size = sizeof(eidm_shape);
    s.weight_dtype = f->adapter_dtype;
    s.m = f->m;
    s.n = b ? f->n : f->max_rank;
    s.k = b ? f->max_rank : f->k;
    s.top_k = 1;
    s.n_experts = f->n_adapters;
    s.expert_stride_bytes = b ? f->b_stride_bytes : f->a_stride_bytes;
    eidm_requirements r{};
    r.struct_size = sizeof(r);
    const int rc = eidm_query(&s, EIDM_ROUTE_DIRECT, &r);
    *bytes = r.required_weight_bytes;
    return rc;
}

// shared: the call computes the shared projection itself
int lora_sizes(const eidm_lora_shape* f, bool shared, LoraSizes* z) {
    if (!f) return api_fail(EIDM_E_INVALID, "shape is NULL");
    if (f->struct_size != sizeof(eidm_lora_shape))
        return api_fail(EIDM_E_INVALID, "lora shape struct_size %u, expected %zu", f->struct_size,
                        sizeof(eidm_lora_shape));
    int rc = adapter_extent(f, false, &z->a);
    if (rc) return rc;
    rc = adapter_extent(f, true, &z->b);
    if (rc) return rc;
    if (f->max_rank > kMaxLoraRank)
        return api_fail(EIDM_E_UNSUPPORTED, "max_rank %u above the supported %u", f->max_rank, kMaxLoraRank);
    z->v_stride = (f->max_rank + 7) / 8 * 8;
    z->off_hist = align256((uint64_t)f->m * z->v_stride * 4);
    z->off_counts = z->off_offsets = z->off_rows = z->off_tiles = z->off_ids = z->off_hist;
    if (lora_sorts_rows(f->m, f->n, f->k, f->n_adapters, f->max_rank)) {
        // a launch has a block of 256 threads per slot and 256 columns or 32
        // ranks, and fewer than 2^32 threads
        const uint64_t columns = ((uint64_t)f->n + 255) / 256, ranks = (f->max_rank + 31) / 32;
        if (lora_slots(f->m, f->n_adapters) * std::max(columns, ranks) >= 1u << 24)
            return api_fail(EIDM_E_UNSUPPORTED, "the adapters' grid for %u rows of %u columns is too large", f->m, f->n);
        z->off_counts = z->off_hist + align256(map_hist_elements(f->m, f->n_adapters) * 4);
        z->off_offsets = z->off_counts + align256((uint64_t)(f->n_adapters + 1) * 4);
        z->off_rows = z->off_offsets + align256((uint64_t)(f->n_adapters + 2) * 4);
        z->off_tiles = z->off_rows + align256((uint64_t)f->m * 4);
        z->off_ids = z->off_tiles + align256(lora_slots(f->m, f->n_adapters) * kTileWords * 4);
    }
    z->off_matmul = z->off_ids + align256((uint64_t)f->m * 4);
    z->weights = z->matmul = 0;
    if (shared) {
        if (f->m == 1 && f->n >= 1u << 29)  // the Direct route's 128 threads per 16 columns
            return api_fail(EIDM_E_UNSUPPORTED, "the projection's grid for one row of %u columns is too large", f->n);
        const eidm_shape s = shared_projection(f);
        eidm_requirements q{};
        q.struct_size = sizeof(q);
        rc = eidm_query(&s, EIDM_ROUTE_GROUPED, &q);
        if (rc) return rc;
        z->weights = q.required_weight_bytes;
        z->matmul = q.scratch_bytes;
        if (f->arith == EIDM_ARITH_SPLIT16 && dense_split16_bytes(f->m, f->k) > z->matmul)
            z->matmul = dense_split16_bytes(f->m, f->k);
    }
    z->total = z->off_matmul + z->matmul;
    return EIDM_OK;
}

}  // namespace
}  // namespace eidm

extern "C" {

uint64_t eidm_lora_linear_scratch_bytes(const eidm_lora_shape* shape) {
    eidm::LoraSizes z{};
    if (eidm::lora_sizes(shape, true, &z) != EIDM_OK) return 0;
    eidm::api_ok();
    return z.total;
}

int eidm_lora_linear(const eidm_lora_shape* shape, const void* weights, uint64_t weight_bytes, const float* base,
                     const void* adapter_a, uint64_t a_bytes, const void* adapter_b, uint64_t b_bytes,
                     const uint32_t* ranks, const float* scales, const float* input, const uint32_t* adapter_ids,
                     float* output, void* scratch, uint64_t scratch_bytes, void* stream) {
    using eidm::api_fail;
    eidm::ReceiptScope dispatch_receipt;
    eidm::LoraSizes z{};
    int rc = eidm::lora_sizes(shape, weights != nullptr, &z);
    if (rc) return rc;
    if ((weights == nullptr) == (base == nullptr))
        return api_fail(EIDM_E_INVALID, "exactly one of weights and base must be given");
    if (!adapter_a || !adapter_b || !input || !adapter_ids || !output || !scratch)
        return api_fail(EIDM_E_INVALID, "a lora buffer is NULL");
    const struct {
        const char* what;
        uint64_t need, given;
    } extents[] = {{"weights", z.weights, weights ? weight_bytes : 0},
                   {"adapter A", z.a, a_bytes},
                   {"adapter B", z.b, b_bytes},
                   {"scratch", z.total, scratch_bytes}};
    for (const auto& x : extents)
        if (x.given < x.need)
            return api_fail(EIDM_E_SIZE, "%s: %llu bytes needed, %llu given", x.what, (unsigned long long)x.need,
                            (unsigned long long)x.given);
    auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    if (bits(scratch) % 256) return api_fail(EIDM_E_ALIGN, "the lora scratch must be 256-byte aligned");
    if ((bits(adapter_a) | bits(adapter_b)) % eidm::size_of(shape->adapter_dtype))
        return api_fail(EIDM_E_ALIGN, "adapters must be aligned to the scalar size");
    if ((bits(base) | bits(ranks) | bits(scales) | bits(input) | bits(adapter_ids) | bits(output)) % 4)
        return api_fail(EIDM_E_ALIGN, "lora buffers must be 4-byte aligned");
    if (weights) {  // the shared projection's own conditions, before anything is enqueued
        if (bits(weights) % eidm::size_of(shape->weight_dtype))
            return api_fail(EIDM_E_ALIGN, "weights must be aligned to the scalar size");
        if (shape->arith == EIDM_ARITH_SPLIT16 && ((bits(weights) | bits(input)) % 16 ||
                                                   (uint64_t)shape->n * shape->k * 2 % 16))
            return api_fail(EIDM_E_ALIGN, "the split-16 arithmetic needs weights and input 16-byte aligned");
    }

    hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(scratch);
    eidm::LoraArgs a{};
    a.dtype = shape->adapter_dtype;
    a.m = shape->m;
    a.n = shape->n;
    a.k = shape->k;
    a.n_adapters = shape->n_adapters;
    a.max_rank = shape->max_rank;
    a.v_stride = z.v_stride;
    a.a_stride = shape->a_stride_bytes;
    a.b_stride = shape->b_stride_bytes;
    a.a = static_cast<const uint8_t*>(adapter_a);
    a.b = static_cast<const uint8_t*>(adapter_b);
    a.ranks = ranks;
    a.ids = adapter_ids;
    a.scales = scales;
    a.x = input;
    a.base = weights ? output : base;
    a.v = reinterpret_cast<float*>(ws);
    a.out = output;
    const int cus = eidm::device_cus();
    hipError_t err;
    if (eidm::lora_sorts_rows(a.m, a.n, a.k, a.n_adapters, a.max_rank)) {
        auto at = [&](uint64_t off) { return reinterpret_cast<uint32_t*>(ws + off); };
        const eidm::MapBuffers buf{at(z.off_hist), at(z.off_counts), at(z.off_offsets), at(z.off_rows)};
        err = eidm::launch_map(adapter_ids, a.m, a.n_adapters, buf, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "map launch: %s", hipGetErrorString(err));
        a.offsets = buf.offsets;
        a.rows = buf.rows;
        a.tiles = at(z.off_tiles);
    }
    if (weights && shape->arith == EIDM_ARITH_F32 && eidm::lora_base_few_supported(a, cus)) {
        err = eidm::launch_lora_base_few(a, shape->weight_dtype, static_cast<const uint8_t*>(weights), cus, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "projection launch: %s", hipGetErrorString(err));
    } else if (weights && shape->arith == EIDM_ARITH_SPLIT16 && eidm::dense_split16_supported(a.m, a.n, a.k, cus)) {
        err = eidm::launch_lora_shrink(a, cus, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "adapter shrink launch: %s", hipGetErrorString(err));
        eidm::MatmulArgs p{};
        p.dtype = shape->weight_dtype;
        p.m = a.m;
        p.n = a.n;
        p.k = a.k;
        p.top_k = p.n_experts = 1;
        p.weights = weights;
        p.input = input;
        p.output = output;
        p.xsplit = reinterpret_cast<uint16_t*>(ws + z.off_matmul);
        err = eidm::launch_dense_split16(p, cus, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "projection launch: %s", hipGetErrorString(err));
    } else {
        if (weights) a.zero_ids = reinterpret_cast<uint32_t*>(ws + z.off_ids);
        err = eidm::launch_lora_shrink(a, cus, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "adapter shrink launch: %s", hipGetErrorString(err));
        if (weights) {
            const eidm_shape s = eidm::shared_projection(shape);
            rc = eidm_matmul_id(&s, EIDM_ROUTE_AUTO, weights, weight_bytes, input, a.zero_ids, output,
                                ws + z.off_matmul, z.matmul, stream, nullptr);
            if (rc) return rc;
        }
    }
    err = eidm::launch_lora_expand(a, cus, st);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "adapter expand launch: %s", hipGetErrorString(err));
    return eidm::api_ok();
}

}  // extern "C"
