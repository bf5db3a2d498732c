// lora.hip -- low-rank adapters of many requests at once:
//   shrink: v[t] = A_a x[t] (max_rank numbers a row, in the library's fixed
//     reduction order), a = the row's adapter;
//   expand: out[t] = base[t] + scale_a * (B_a v[t]).
// The shared projection beside them is eidm_matmul_id with one expert.
//
// An adapter is selected per row as an expert is (mlx-native 0.13.0,
// src/ops/dense_matmul_id_auto.rs: a stack of weights, one id per row).
#include "eidm.h"
#include "eidm_device.hpp"
#include "eidm_internal.hpp"
#include "few_rows.hpp"

namespace eidm {
namespace {

__device__ __forceinline__ uint32_t rank_of(const LoraArgs& a, uint32_t id) {
    return a.ranks ? min(a.ranks[id], a.max_rank) : a.max_rank;
}

// One wavefront per (row, four ranks).
template <int DT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs a) {
    const int lane = threadIdx.x & 63;
    const int b = lane >> 2, q = lane & 3;
    const uint32_t groups = (a.max_rank + 3) / 4;
    const uint64_t jobs = (uint64_t)a.m * groups;
    const uint64_t waves = (uint64_t)gridDim.x * 4;
    if (a.zero_ids)
        for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < a.m; i += (uint64_t)gridDim.x * 256)
            a.zero_ids[i] = 0;
    for (uint64_t job = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); job < jobs; job += waves) {
        const uint32_t t = (uint32_t)(job / groups);
        const uint32_t i0 = (uint32_t)(job % groups) * 4;
        const uint32_t id = a.ids[t];
        if (id >= a.n_adapters) continue;
        const uint32_t rank = rank_of(a, id);
        if (i0 >= rank) continue;
        const uint32_t i = min(i0 + q, rank - 1);
        const uint8_t* const wrow[1] = {a.a + (size_t)id * a.a_stride + (size_t)i * a.k * DtypeSize<DT>::value};
        const float* const xrow[1] = {a.x + (size_t)t * a.k};
        f32x4 acc[1][1];
        few_rows_product<DT, 1, 1, 8, true, false>(wrow, xrow, (int)a.k, acc);
        const float v = slice_tree(acc[0][0][0]);
        if (b == 0 && i0 + q < rank) a.v[(size_t)t * a.v_stride + i0 + q] = v;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs a) {
    constexpr int S = DtypeSize<DT>::value;
    const uint64_t total = (uint64_t)a.m * a.n;
    for (uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += (uint64_t)gridDim.x * 256) {
        const uint32_t t = (uint32_t)(at / a.n), j = (uint32_t)(at % a.n);
        const uint32_t id = a.ids[t];
        float y = a.base[at];
        if (id < a.n_adapters) {
            const uint32_t rank = rank_of(a, id);
            if (rank) {
                const uint8_t* row = a.b + (size_t)id * a.b_stride + (size_t)j * a.max_rank * S;
                const float* v = a.v + (size_t)t * a.v_stride;
                float u = 0.0f;
                for (uint32_t i = 0; i < rank; ++i) {
                    uint32_t bits;
                    if constexpr (S == 4) bits = *reinterpret_cast<const uint32_t*>(row + (size_t)i * 4);
                    else bits = *reinterpret_cast<const uint16_t*>(row + (size_t)i * 2);
                    u = fma_step(v[i], widen_bits<DT>(bits), u);
                }
                y = fma_step(a.scales ? a.scales[id] : 1.0f, u, y);
            }
        } else if (id != EIDM_NO_ADAPTER) {
            y = quiet_nan();
        }
        a.out[at] = y;
    }
}

uint32_t grid_of(uint64_t blocks, uint64_t most) { return (uint32_t)(blocks < most ? blocks : most); }

template <int DT>
hipError_t shrink_dt(const LoraArgs& a, int device_cus, hipStream_t stream) {
    const uint64_t jobs = (uint64_t)a.m * ((a.max_rank + 3) / 4);
    const uint32_t grid = grid_of((jobs + 3) / 4, (uint64_t)device_cus * 16);
    hipLaunchKernelGGL(lora_shrink_kernel<DT>, dim3(grid), dim3(256), 0, stream, a);
    return launched(EIDM_KERNEL_LORA_SHRINK, grid, 256, 0);
}

template <int DT>
hipError_t expand_dt(const LoraArgs& a, int device_cus, hipStream_t stream) {
    const uint32_t grid = grid_of(((uint64_t)a.m * a.n + 255) / 256, (uint64_t)device_cus * 32);
    hipLaunchKernelGGL(lora_expand_kernel<DT>, dim3(grid), dim3(256), 0, stream, a);
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
    a.zero_ids = weights ? reinterpret_cast<uint32_t*>(ws + z.off_ids) : nullptr;
    hipError_t err = eidm::launch_lora_shrink(a, eidm::device_cus(), st);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "adapter shrink launch: %s", hipGetErrorString(err));
    if (weights) {
        const eidm_shape s = eidm::shared_projection(shape);
        rc = eidm_matmul_id(&s, EIDM_ROUTE_AUTO, weights, weight_bytes, input, a.zero_ids, output, ws + z.off_matmul,
                            z.matmul, stream, nullptr);
        if (rc) return rc;
    }
    err = eidm::launch_lora_expand(a, eidm::device_cus(), st);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "adapter expand launch: %s", hipGetErrorString(err));
    return eidm::api_ok();
}

}  // extern "C"
