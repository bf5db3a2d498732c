// lora.hip -- low-rank adapters of many requests at once:
//   shrink: v[t] = A_a x[t] (max_rank numbers a row, in the library's fixed
//     reduction order), a = the row's adapter;
//   expand: out[t] = base[t] + scale_a * (B_a v[t]).
// The shared projection beside them is eidm_matmul_id with one expert.
//
// An adapter is selected per row as an expert is (mlx-native 0.13.0,
// src/ops/dense_matmul_id_auto.rs: a stack of weights, one id per row).
//
// Two forms of each, with the same bits.  By rows (a decode batch, where
// rows have adapters of their own): a wavefront takes one row and streams its
// adapter.  By tiles (prompts, where neighbouring rows share an adapter):
// a wavefront takes 16 consecutive rows and runs once over each adapter that
// occurs among them, so no row needs sorting and all rows are read and
// written in their order.  A decode batch's shared projection and its shrink
// run side by side in one launch.
#include "eidm.h"
#include "eidm_device.hpp"
#include "eidm_internal.hpp"
#include "few_rows.hpp"
#include "rows16.hpp"

namespace eidm {
namespace {

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

// Work of one block of 256: ranks 16*part .. of row t, four per wavefront;
// the row is staged in LDS.
template <int DT>
__device__ __forceinline__ void shrink_row(const LoraArgs& a, uint32_t t, uint32_t part, float* xs) {
    const uint32_t q = threadIdx.x & 3;
    const uint32_t id = a.ids[t];
    if (id >= a.n_adapters) return;
    const uint32_t rank = rank_of(a, id);
    if (part * 16 >= rank) return;
    const uint32_t i0 = part * 16 + (threadIdx.x >> 6) * 4;
    const uint8_t* const wrow[1] = {a.a + (size_t)id * a.a_stride +
                                    (size_t)min(i0 + q, rank - 1) * a.k * DtypeSize<DT>::value};
    FewStream<DT, 1, DtypeSize<DT>::value == 4 ? 8 : 16, false> w;
    if (i0 < rank) w.start(wrow, (int)a.k);  // wave-uniform
    auto stage = few_stage<8>(xs, 1, a.k, [&](uint32_t) { return a.x + (size_t)t * a.k; });
    stage.issue();
    stage.finish();
    __syncthreads();
    if (i0 >= rank) return;
    few_rows_tile<0, false>(w, wrow, wrow, xs, 0, 1, (int)a.k, [](uint32_t) { return 0; },
                            [&](uint32_t, const float (&v)[1]) {
                                if (i0 + q < rank) a.v[(size_t)t * a.v_stride + i0 + q] = v[0];
                            });
}

template <int DT>
__global__ __launch_bounds__(256) void shrink_row_kernel(LoraArgs a, uint32_t parts) {
    extern __shared__ __align__(16) float xs[];
    write_zero_ids(a);
    shrink_row<DT>(a, blockIdx.x / parts, blockIdx.x % parts, xs);
}

// The shared projection of up to 64 rows (a.out = W x) and, in the first
// `shrinks` blocks of the same launch, the shrink of those rows, which needs
// none of it.  RG 0, 1 (one row, up to four): rows staged in LDS, each
// wavefront four columns; else RT = -RG row tiles of 16 rows against 16
// columns per block.
template <int DT, int RG>
__global__ __launch_bounds__(256) void base_few_kernel(LoraArgs a, const uint8_t* weights, uint32_t shrinks,
                                                       uint32_t parts) {
    extern __shared__ __align__(16) float xs[];
    if (blockIdx.x < shrinks) {
        shrink_row<DT>(a, blockIdx.x / parts, blockIdx.x % parts, xs);
        return;
    }
    const uint32_t block = blockIdx.x - shrinks, lane = threadIdx.x & 63;
    if constexpr (RG >= 0) {
        const uint32_t q = lane & 3, col = block * 16 + (threadIdx.x >> 6) * 4 + q;
        const bool live = col - q < a.n;  // wave-uniform
        const uint8_t* const wrow[1] = {weights + (size_t)min(col, a.n - 1) * a.k * DtypeSize<DT>::value};
        FewStream<DT, 1, DtypeSize<DT>::value == 4 ? 8 : 16, true> w;
        if (live) w.start(wrow, (int)a.k);
        auto stage = few_stage<8>(xs, a.m, a.k, [&](uint32_t t) { return a.x + (size_t)t * a.k; });
        stage.issue();
        stage.finish();
        __syncthreads();
        if (!live) return;
        few_rows_tile<RG, false>(w, wrow, wrow, xs, few_row_floats(a.k), a.m, (int)a.k, [](uint32_t i) { return i; },
                                 [&](uint32_t t, const float (&v)[1]) {
                                     if (col < a.n) a.out[(size_t)t * a.n + col] = v[0];
                                 });
    } else {
        constexpr int RT = -RG;
        const uint32_t i = lane & 15, col = block * 16 + i;
        const float* xrow[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) xrow[t] = a.x + (size_t)min(t * 16 + i, a.m - 1) * a.k;
        float total[RT];
        rows16_product<DT, RT, RT >= 4 ? 4 : 8, true>(weights + (size_t)min(col, a.n - 1) * a.k * DtypeSize<DT>::value,
                                                      xrow, (int)a.k, xs, total);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const uint32_t r = t * 16 + 4 * (lane >> 4) + (threadIdx.x >> 6);
            if (r < a.m && col < a.n) a.out[(size_t)r * a.n + col] = total[t];
        }
    }
}

// A tile of 16 consecutive rows: lane l holds row l%16's adapter (`none` for
// a row past the last).  Calls body(id, members) for every adapter id <
// n_adapters among them, members a bit per row of the tile.
template <typename Body>
__device__ __forceinline__ void for_each_adapter(uint32_t mine, uint32_t n_adapters, Body body) {
    uint32_t left = (uint32_t)__ballot(mine < n_adapters) & 0xffffu;
    while (left) {  // wave-uniform
        const uint32_t id = (uint32_t)__builtin_amdgcn_readlane((int)mine, __builtin_ctz(left));
        const uint32_t members = (uint32_t)__ballot(mine == id) & 0xffffu;
        left &= ~members;
        body(id, members);
    }
}

// One block per (16 rows, 16 ranks).
template <int DT>
__global__ __launch_bounds__(256) void shrink_tile_kernel(LoraArgs a) {
    __shared__ __align__(16) float xs[rows16_lds(1)];
    const uint32_t lane = threadIdx.x & 63, i = lane & 15;
    const uint32_t chunks = (a.max_rank + 15) / 16;
    const uint64_t tiles = ((uint64_t)a.m + 15) / 16;
    write_zero_ids(a);
    for (uint64_t job = blockIdx.x; job < tiles * chunks; job += gridDim.x) {
        const uint64_t t0 = job / chunks * 16;
        const uint32_t c0 = (uint32_t)(job % chunks) * 16;
        const uint64_t t = t0 + i < a.m ? t0 + i : a.m - 1;
        const uint32_t mine = t0 + i < a.m ? a.ids[t] : EIDM_NO_ADAPTER;
        for_each_adapter(mine, a.n_adapters, [&](uint32_t id, uint32_t members) {
            const uint32_t rank = rank_of(a, id);
            if (c0 >= rank) return;  // block-uniform
            const float* const xrow[1] = {a.x + t * a.k};
            float total[1];
            rows16_product<DT, 1, 8, false>(a.a + (size_t)id * a.a_stride +
                                                (size_t)min(c0 + i, rank - 1) * a.k * DtypeSize<DT>::value,
                                            xrow, (int)a.k, xs, total);
            const uint32_t r = 4 * (lane >> 4) + (threadIdx.x >> 6);
            if ((members >> r & 1) && c0 + i < rank) a.v[(t0 + r) * a.v_stride + c0 + i] = total[0];
        });
    }
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
            const uint32_t rank = rank_of(a, id);
            const uint8_t* row = a.b + (size_t)id * a.b_stride + (size_t)j * a.max_rank * DtypeSize<DT>::value;
            const float* v = a.v + t * a.v_stride;
            float u = 0.0f;
            for (uint32_t i0 = 0; i0 < rank; i0 += kBatch * kGranule) {
                float b[kBatch][kGranule];
#pragma unroll
                for (uint32_t h = 0; h < kBatch; ++h)
                    if (i0 + h * kGranule < rank) load_b<DT>(row, i0 + h * kGranule, a.max_rank, b[h]);
#pragma unroll
                for (uint32_t h = 0; h < kBatch; ++h)
#pragma unroll
                    for (uint32_t i = 0; i < kGranule; ++i)
                        if (i0 + h * kGranule + i < rank) u = fma_step(v[i0 + h * kGranule + i], b[h][i], u);
            }
            if (rank) y = fma_step(scale_of(a, id), u, y);
        } else if (id != EIDM_NO_ADAPTER) {
            y = quiet_nan();
        }
        a.out[t * a.n + j] = y;
    }
}

// One wavefront per (16 rows, 64 columns).  v_mfma_f32_16x16x1_4b_f32, one
// rank per step: all four blocks take the 16 rows of v, block s the columns
// 4i+s, so a lane's results are four consecutive columns of four rows.
template <int DT>
__global__ __launch_bounds__(256) void expand_tile_kernel(LoraArgs a) {
    const uint32_t lane = threadIdx.x & 63, i = lane & 15, s = lane >> 4;
    const uint32_t groups = (a.n + 63) / 64;
    const uint64_t tiles = ((uint64_t)a.m + 15) / 16;
    for (uint64_t job = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); job < tiles * groups; job += (uint64_t)gridDim.x * 4) {
        const uint64_t t0 = job / groups * 16;
        const uint32_t j0 = (uint32_t)(job % groups) * 64 + 4 * i;  // this lane's output columns j0 .. j0+3
        const uint64_t t = t0 + i < a.m ? t0 + i : a.m - 1;
        const uint32_t mine = t0 + i < a.m ? a.ids[t] : EIDM_NO_ADAPTER;
        f32x4 y[4];  // rows 4s .. 4s+3
#pragma unroll
        for (uint32_t v = 0; v < 4; ++v) {
            const uint64_t r = t0 + 4 * s + v;
            y[v] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (r < a.m) {
                const float* p = a.base + r * a.n + j0;
                if (j0 + 4 <= a.n) y[v] = *reinterpret_cast<const fr_f32x4_a4*>(p);
                else
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c)
                        if (j0 + c < a.n) y[v][c] = p[c];
            }
        }
        for_each_adapter(mine, a.n_adapters, [&](uint32_t id, uint32_t members) {
            const uint32_t rank = rank_of(a, id);
            if (!rank) return;
            const uint32_t col = min(j0 + s, a.n - 1);  // this lane's column of B
            const uint8_t* row = a.b + (size_t)id * a.b_stride + (size_t)col * a.max_rank * DtypeSize<DT>::value;
            const float* v = a.v + t * a.v_stride;
            f32x16 u{};
            for (uint32_t i0 = 0; i0 < rank; i0 += kGranule) {
                float b[kGranule];
                load_b<DT>(row, i0, a.max_rank, b);
                const f32x4 v0 = *reinterpret_cast<const f32x4*>(v + i0), v1 = *reinterpret_cast<const f32x4*>(v + i0 + 4);
#pragma unroll
                for (uint32_t e = 0; e < kGranule; ++e)
                    if (i0 + e < rank)  // wave-uniform
                        u = __builtin_amdgcn_mfma_f32_16x16x1f32(e < 4 ? v0[e % 4] : v1[e % 4], b[e], u, 0, 0, 0);
            }
            const float scale = scale_of(a, id);
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r)
                if (members >> (4 * s + r) & 1)
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c) y[r][c] = fma_step(scale, u[4 * c + r], y[r][c]);
        });
        const uint32_t bad = (uint32_t)__ballot(mine >= a.n_adapters && mine != EIDM_NO_ADAPTER) & 0xffffu;
#pragma unroll
        for (uint32_t v = 0; v < 4; ++v) {
            const uint64_t r = t0 + 4 * s + v;
            if (r >= a.m) continue;
            if (bad >> (4 * s + v) & 1) y[v] = f32x4{quiet_nan(), quiet_nan(), quiet_nan(), quiet_nan()};
            float* p = a.out + r * a.n + j0;
            if (j0 + 4 <= a.n) *reinterpret_cast<fr_f32x4_a4*>(p) = y[v];
            else
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c)
                    if (j0 + c < a.n) p[c] = y[v][c];
        }
    }
}

uint32_t grid_of(uint64_t blocks, uint64_t most) { return (uint32_t)(blocks < most ? blocks : most); }

// Rows of up to this many take the row forms.
constexpr uint32_t kRowForm = EIDM_DECODE_MAX_TOKENS;
constexpr uint32_t kRowLds = 64 * 1024;  // LDS of staged rows

bool stages_rows(uint32_t rows, uint32_t k) { return (uint64_t)rows * few_row_floats(k) * 4 <= kRowLds; }

template <int DT>
hipError_t shrink_dt(const LoraArgs& a, int device_cus, hipStream_t stream) {
    if (a.m <= kRowForm && stages_rows(1, a.k)) {
        const uint32_t parts = (a.max_rank + 15) / 16, lds = few_row_floats(a.k) * 4;
        hipLaunchKernelGGL(shrink_row_kernel<DT>, dim3(a.m * parts), dim3(256), lds, stream, a, parts);
        return launched(EIDM_KERNEL_LORA_SHRINK, a.m * parts, 256, lds);
    }
    const uint64_t jobs = ((uint64_t)a.m + 15) / 16 * ((a.max_rank + 15) / 16);
    const uint32_t grid = grid_of(jobs, (uint64_t)device_cus * 16);
    hipLaunchKernelGGL(shrink_tile_kernel<DT>, dim3(grid), dim3(256), 0, stream, a);
    return launched(EIDM_KERNEL_LORA_SHRINK, grid, 256, 0);
}

template <int DT, int RG>
hipError_t base_few(const LoraArgs& a, const uint8_t* weights, bool with_shrink, hipStream_t stream) {
    const uint32_t parts = (a.max_rank + 15) / 16, shrinks = with_shrink ? a.m * parts : 0;
    const uint32_t blocks = (a.n + 15) / 16;
    uint32_t lds = RG >= 0 ? a.m * few_row_floats(a.k) * 4 : rows16_lds(-RG) * 4;
    if (with_shrink && lds < few_row_floats(a.k) * 4) lds = few_row_floats(a.k) * 4;
    hipLaunchKernelGGL((base_few_kernel<DT, RG>), dim3(shrinks + blocks), dim3(256), lds, stream, a, weights, shrinks,
                       parts);
    return launched(EIDM_KERNEL_LORA_BASE, shrinks + blocks, 256, lds);
}

template <int DT>
hipError_t base_few_dt(const LoraArgs& a, const uint8_t* weights, bool with_shrink, hipStream_t stream) {
    if (a.m <= 4 && stages_rows(a.m, a.k))
        return a.m == 1 ? base_few<DT, 0>(a, weights, with_shrink, stream)
                        : base_few<DT, 1>(a, weights, with_shrink, stream);
    if (a.m <= 16) return base_few<DT, -1>(a, weights, with_shrink, stream);
    if (a.m <= 32) return base_few<DT, -2>(a, weights, with_shrink, stream);
    return base_few<DT, -4>(a, weights, with_shrink, stream);
}

template <int DT>
hipError_t expand_dt(const LoraArgs& a, int device_cus, hipStream_t stream) {
    if (a.m <= kRowForm) {
        const uint32_t grid = grid_of((uint64_t)a.m * ((a.n + 255) / 256), (uint64_t)device_cus * 32);
        hipLaunchKernelGGL(expand_row_kernel<DT>, dim3(grid), dim3(256), 0, stream, a);
        return launched(EIDM_KERNEL_LORA_EXPAND, grid, 256, 0);
    }
    const uint64_t jobs = ((uint64_t)a.m + 15) / 16 * ((a.n + 63) / 64);
    const uint32_t grid = grid_of((jobs + 3) / 4, (uint64_t)device_cus * 64);
    hipLaunchKernelGGL(expand_tile_kernel<DT>, dim3(grid), dim3(256), 0, stream, a);
    return launched(EIDM_KERNEL_LORA_EXPAND, grid, 256, 0);
}

}  // namespace

hipError_t launch_lora_shrink(const LoraArgs& a, int device_cus, hipStream_t stream) {
    switch (a.dtype) {
    case kDtypeF32: return shrink_dt<kDtypeF32>(a, device_cus, stream);
    case kDtypeF16: return shrink_dt<kDtypeF16>(a, device_cus, stream);
    case kDtypeBF16: return shrink_dt<kDtypeBF16>(a, device_cus, stream);
    default: return hipErrorInvalidValue;
    }
}

bool lora_base_few_supported(const LoraArgs& a) { return a.m <= kRowForm; }

hipError_t launch_lora_base_few(const LoraArgs& a, int weight_dtype, const uint8_t* weights, int device_cus,
                                hipStream_t stream) {
    const bool together = weight_dtype == a.dtype && stages_rows(1, a.k);
    if (!together) {
        const hipError_t err = launch_lora_shrink(a, device_cus, stream);
        if (err != hipSuccess) return err;
    }
    switch (weight_dtype) {
    case kDtypeF32: return base_few_dt<kDtypeF32>(a, weights, together, stream);
    case kDtypeF16: return base_few_dt<kDtypeF16>(a, weights, together, stream);
    case kDtypeBF16: return base_few_dt<kDtypeBF16>(a, weights, together, stream);
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
    uint64_t off_ids, off_matmul, matmul, total;  // scratch: v | ids of the shared projection | its own scratch
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
    z->off_ids = align256((uint64_t)f->m * z->v_stride * 4);
    z->off_matmul = z->off_ids + align256((uint64_t)f->m * 4);
    z->weights = z->matmul = 0;
    if (shared) {
        const eidm_shape s = shared_projection(f);
        eidm_requirements q{};
        q.struct_size = sizeof(q);
        rc = eidm_query(&s, EIDM_ROUTE_GROUPED, &q);
        if (rc) return rc;
        z->weights = q.required_weight_bytes;
        z->matmul = q.scratch_bytes;
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
    hipError_t err;
    if (weights && shape->arith == EIDM_ARITH_F32 && eidm::lora_base_few_supported(a)) {
        err = eidm::launch_lora_base_few(a, shape->weight_dtype, static_cast<const uint8_t*>(weights),
                                         eidm::device_cus(), st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "projection launch: %s", hipGetErrorString(err));
    } else {
        if (weights) a.zero_ids = reinterpret_cast<uint32_t*>(ws + z.off_ids);
        err = eidm::launch_lora_shrink(a, eidm::device_cus(), st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "adapter shrink launch: %s", hipGetErrorString(err));
        if (weights) {
            const eidm_shape s = eidm::shared_projection(shape);
            rc = eidm_matmul_id(&s, EIDM_ROUTE_AUTO, weights, weight_bytes, input, a.zero_ids, output,
                                ws + z.off_matmul, z.matmul, stream, nullptr);
            if (rc) return rc;
        }
    }
    err = eidm::launch_lora_expand(a, eidm::device_cus(), st);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "adapter expand launch: %s", hipGetErrorString(err));
    return eidm::api_ok();
}

}  // extern "C"
