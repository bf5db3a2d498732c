// moe_decode.hip -- the expert FFN of a few tokens (m <= 64):
//   gate/up kernel: h[r] = silu(W_gate[e] x[t]) * (W_up[e] x[t]) for every
//     routed row r = t*top_k + s of expert e, both products and the
//     activation in one pass over the two weights;
//   down/combine kernel: out[t] = sum_s gate[t, s] W_down[e] h[r], a block
//     owning a few output columns of every token, so the sum over slots is
//     taken in LDS in slot order.
// Each touched expert's weights are read once per call, however many tokens
// chose it (up to 16 rows at a time).
//
// Every product is in the library's fixed reduction order, silu and the
// combine are the same f32 operations as the separate kernels', so the
// results are bit for bit those of eidm_moe_ffn.
//
// cortiq-engine 0.7.7, src/mimo_moe.rs, Dynamic::run (route, one FFN per
// pick, weighted sum); hf2q dense_ffn_arena.rs, MoeFfnArena (gate, up, h, y).
#include "eidm_device.hpp"
#include "eidm_internal.hpp"
#include "few_map.hpp"
#include "few_rows.hpp"

namespace eidm {
namespace {

constexpr int kWaves = 8;  // wavefronts per block

// Ring depth that keeps a slot ring within about 128 registers.
template <int DT, int C, int RG>
constexpr int few_depth() {
    constexpr int slot = C * DtypeSize<DT>::value * 2 + RG * 8;
    return 128 / slot > 8 ? 8 : (128 / slot < 2 ? 2 : 128 / slot);
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

// Up to 4*RG rows of one expert times 4*C weight rows: emit(row position in
// the list, c, total) for every live row, in the lanes that hold totals of
// column q = lane & 3.
template <int DT, int C, int RG, bool ONE, typename XRow, typename Emit>
__device__ __forceinline__ void few_rows_tile(const uint8_t* const (&wrow)[C], int k, uint32_t first, uint32_t end,
                                              XRow xrow_of, Emit emit) {
    const int lane = threadIdx.x & 63;
    const int b = lane >> 2, q = lane & 3;
    const float* xrow[RG];
#pragma unroll
    for (int g = 0; g < RG; ++g) xrow[g] = xrow_of(ONE ? first : min(first + 4 * g + q, end - 1));
    f32x4 acc[RG][C];
    few_rows_product<DT, C, RG, few_depth<DT, C, RG>(), ONE>(wrow, xrow, k, acc);
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        float v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = ONE ? slice_tree(acc[g][c][0]) : few_rows_total(acc[g][c]);
        const uint32_t at = ONE ? first : first + 4 * g + few_row(b);
        if (ONE ? b == 0 : ((b & 3) == 0 && at < end)) emit(at, v);
    }
}

// All rows [first, end) of an expert, 16 at a time.
template <int DT, int C, typename XRow, typename Emit>
__device__ __forceinline__ void few_rows_all(const uint8_t* const (&wrow)[C], int k, uint32_t first, uint32_t end,
                                             XRow xrow_of, Emit emit) {
    while (first < end) {  // wave-uniform
        const uint32_t left = end - first;
        if (left == 1) few_rows_tile<DT, C, 1, true>(wrow, k, first, end, xrow_of, emit);
        else if (left <= 4) few_rows_tile<DT, C, 1, false>(wrow, k, first, end, xrow_of, emit);
        else if (left <= 8) few_rows_tile<DT, C, 2, false>(wrow, k, first, end, xrow_of, emit);
        else few_rows_tile<DT, C, 4, false>(wrow, k, first, end, xrow_of, emit);
        first += 16;
    }
}

template <int DT>
__global__ __launch_bounds__(64 * kWaves) void gate_up_kernel(MoeDecodeArgs a) {
    constexpr int S = DtypeSize<DT>::value;
    extern __shared__ uint32_t lds[];
    const uint32_t rows = a.m * a.top_k;
    const FewMap map = few_map_at(lds, rows, a.n_experts);
    few_map_build(map, a.ids, rows, a.n_experts);

    const int q = threadIdx.x & 3;
    const int k = (int)a.hidden, n = (int)a.inter;
    const uint32_t groups = (a.inter + 3) / 4;
    const uint32_t jobs = *map.used * groups;
    const uint32_t waves = gridDim.x * kWaves;
    for (uint32_t job = blockIdx.x * kWaves + (threadIdx.x >> 6); job < jobs; job += waves) {
        const uint32_t u = (uint32_t)__builtin_amdgcn_readfirstlane((int)(job / groups));
        const uint32_t e = (uint32_t)__builtin_amdgcn_readfirstlane((int)map.id[u]);
        const uint32_t first = (uint32_t)__builtin_amdgcn_readfirstlane((int)map.off[u]);
        const uint32_t end = (uint32_t)__builtin_amdgcn_readfirstlane((int)map.off[u + 1]);
        const int col = (int)(job % groups) * 4 + q;
        const size_t at = (size_t)e * a.gate_up_stride + (size_t)min(col, n - 1) * k * S;
        const uint8_t* const wrow[2] = {a.w_gate + at, a.w_up + at};
        few_rows_all<DT, 2>(
            wrow, k, first, end, [&](uint32_t i) { return a.x + (size_t)(map.row[i] / a.top_k) * a.hidden; },
            [&](uint32_t i, const float (&v)[2]) {
                if (col < n) a.h[(size_t)map.row[i] * a.h_stride + col] = silu_mul(v[0], v[1]);
            });
    }
}

// C column groups per block; the wavefronts take the touched experts in turn.
template <int DT, int C>
__global__ __launch_bounds__(64 * kWaves) void down_combine_kernel(MoeDecodeArgs a, int cols) {
    constexpr int S = DtypeSize<DT>::value;
    extern __shared__ uint32_t lds[];
    const uint32_t rows = a.m * a.top_k;
    const FewMap map = few_map_at(lds, rows, a.n_experts);
    float* ys = reinterpret_cast<float*>(lds + few_map_words(rows, a.n_experts));  // [rows][4*C]
    few_map_build(map, a.ids, rows, a.n_experts);

    const int q = threadIdx.x & 3;
    const int k = (int)a.inter, n = (int)a.hidden;
    const int col0 = (int)blockIdx.x * cols;
    const uint32_t used = *map.used;
    for (uint32_t u0 = threadIdx.x >> 6; u0 < used; u0 += kWaves) {
        const uint32_t u = (uint32_t)__builtin_amdgcn_readfirstlane((int)u0);
        const uint32_t e = (uint32_t)__builtin_amdgcn_readfirstlane((int)map.id[u]);
        const uint32_t first = (uint32_t)__builtin_amdgcn_readfirstlane((int)map.off[u]);
        const uint32_t end = (uint32_t)__builtin_amdgcn_readfirstlane((int)map.off[u + 1]);
        const uint8_t* wrow[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 4 * c + q < cols ? min(col0 + 4 * c + q, n - 1) : col0;
            wrow[c] = a.w_down + (size_t)e * a.down_stride + (size_t)col * k * S;
        }
        const uint8_t* const(&wr)[C] = wrow;
        few_rows_all<DT, C>(
            wr, k, first, end, [&](uint32_t i) { return a.h + (size_t)map.row[i] * a.h_stride; },
            [&](uint32_t i, const float (&v)[C]) {
#pragma unroll
                for (int c = 0; c < C; ++c) ys[map.row[i] * (4 * C) + 4 * c + q] = v[c];
            });
    }
    __syncthreads();
    const int live = min(cols, n - col0);
    for (uint32_t i = threadIdx.x; i < a.m * 4 * C; i += blockDim.x) {
        const uint32_t t = i / (4 * C), c = i % (4 * C);
        if ((int)c < live) {
            float acc = 0.0f;
            for (uint32_t s = 0; s < a.top_k; ++s) {
                const uint32_t r = t * a.top_k + s;
                acc = __builtin_fmaf(a.gates[r], ys[r * (4 * C) + c], acc);
            }
            a.out[(size_t)t * a.hidden + col0 + c] = acc;
        }
    }
}

template <int DT>
hipError_t launch_dt(const MoeDecodeArgs& a, int device_cus, hipStream_t stream) {
    const uint32_t rows = a.m * a.top_k;
    const uint32_t map_bytes = few_map_words(rows, a.n_experts) * 4;
    const uint64_t jobs = (uint64_t)few_map_ids(rows, a.n_experts) * ((a.inter + 3) / 4);
    const uint32_t cus = device_cus > 0 ? (uint32_t)device_cus : 256;
    const uint64_t want = (jobs + kWaves - 1) / kWaves;
    const uint32_t grid = (uint32_t)(want < cus ? want : cus);
    hipLaunchKernelGGL(gate_up_kernel<DT>, dim3(grid), dim3(64 * kWaves), map_bytes, stream, a);
    hipError_t err = launched(EIDM_KERNEL_DECODE_GATE_UP, grid, 64 * kWaves, map_bytes);
    if (err != hipSuccess) return err;
    const int cols = a.hidden >= 8 * cus ? 8 : 4;
    const uint32_t blocks = (a.hidden + cols - 1) / cols;
    const uint32_t lds = map_bytes + rows * cols * 4;
    if (cols == 8)
        hipLaunchKernelGGL((down_combine_kernel<DT, 2>), dim3(blocks), dim3(64 * kWaves), lds, stream, a, cols);
    else
        hipLaunchKernelGGL((down_combine_kernel<DT, 1>), dim3(blocks), dim3(64 * kWaves), lds, stream, a, cols);
    return launched(EIDM_KERNEL_DECODE_DOWN, blocks, 64 * kWaves, lds);
}

}  // namespace

hipError_t launch_moe_decode(const MoeDecodeArgs& a, int device_cus, hipStream_t stream) {
    switch (a.dtype) {
    case kDtypeF32: return launch_dt<kDtypeF32>(a, device_cus, stream);
    case kDtypeF16: return launch_dt<kDtypeF16>(a, device_cus, stream);
    case kDtypeBF16: return launch_dt<kDtypeBF16>(a, device_cus, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace eidm

// ------------------------------------------------------------------ C ABI
namespace eidm {
namespace {

uint32_t h_stride(uint32_t inter) { return (inter + 7) / 8 * 8; }  // rows of h start 32-byte aligned

eidm_shape decode_projection(const eidm_ffn_shape* f, bool down) {
    eidm_shape s{};
    s.struct_size = sizeof(eidm_shape);
    s.weight_dtype = f->weight_dtype;
    s.m = f->m;
    s.n = down ? f->hidden : f->inter;
    s.k = down ? f->inter : f->hidden;
    s.top_k = f->top_k;
    s.n_experts = f->n_experts;
    s.expert_stride_bytes = down ? f->down_stride_bytes : f->gate_up_stride_bytes;
    s.input_layout = down ? EIDM_LAYOUT_SLOTTED : EIDM_LAYOUT_SHARED_PER_TOKEN;
    s.id_multiplicity = EIDM_IDS_DISTINCT_PER_TOKEN;
    return s;
}

// Checks the shape; the two projections' weight extents and the scratch size.
int decode_sizes(const eidm_ffn_shape* f, uint64_t* gate_up, uint64_t* down, uint64_t* scratch) {
    if (!f) return api_fail(EIDM_E_INVALID, "shape is NULL");
    if (f->struct_size != sizeof(eidm_ffn_shape))
        return api_fail(EIDM_E_INVALID, "ffn shape struct_size %u, expected %zu", f->struct_size,
                        sizeof(eidm_ffn_shape));
    eidm_requirements rg{}, rd{};
    rg.struct_size = rd.struct_size = sizeof(eidm_requirements);
    const eidm_shape gu = decode_projection(f, false), dn = decode_projection(f, true);
    int rc = eidm_query(&gu, EIDM_ROUTE_DIRECT, &rg);
    if (rc) return rc;
    rc = eidm_query(&dn, EIDM_ROUTE_DIRECT, &rd);
    if (rc) return rc;
    if (f->m > kMaxDecodeTokens)
        return api_fail(EIDM_E_UNSUPPORTED, "%u tokens: the decode FFN takes at most %u (eidm_moe_ffn takes any)", f->m,
                        kMaxDecodeTokens);
    if (f->top_k > kMaxDecodeTopK)
        return api_fail(EIDM_E_UNSUPPORTED, "top_k %u above the decode FFN's %u", f->top_k, kMaxDecodeTopK);
    *gate_up = rg.required_weight_bytes;
    *down = rd.required_weight_bytes;
    *scratch = (uint64_t)f->m * f->top_k * h_stride(f->inter) * 4;
    return EIDM_OK;
}

}  // namespace
}  // namespace eidm

extern "C" {

uint64_t eidm_moe_ffn_decode_scratch_bytes(const eidm_ffn_shape* shape) {
    uint64_t gate_up, down, scratch;
    if (eidm::decode_sizes(shape, &gate_up, &down, &scratch) != EIDM_OK) return 0;
    eidm::api_ok();
    return scratch;
}

int eidm_moe_ffn_decode(const eidm_ffn_shape* shape, const void* w_gate, const void* w_up, uint64_t gate_up_bytes,
                        const void* w_down, uint64_t down_bytes, const float* x, const float* logits,
                        const float* bias, int renormalize, uint32_t* ids, float* gates, float* out, void* scratch,
                        uint64_t scratch_bytes, void* stream) {
    using eidm::api_fail;
    eidm::ReceiptScope dispatch_receipt;
    uint64_t gate_up_need, down_need, scratch_need;
    int rc = eidm::decode_sizes(shape, &gate_up_need, &down_need, &scratch_need);
    if (rc) return rc;
    if (!w_gate || !w_up || !w_down || !x || !logits || !ids || !gates || !out || !scratch)
        return api_fail(EIDM_E_INVALID, "a decode FFN buffer is NULL");
    if (gate_up_bytes < gate_up_need)
        return api_fail(EIDM_E_SIZE, "gate/up weights: %llu bytes needed, %llu given",
                        (unsigned long long)gate_up_need, (unsigned long long)gate_up_bytes);
    if (down_bytes < down_need)
        return api_fail(EIDM_E_SIZE, "down weights: %llu bytes needed, %llu given", (unsigned long long)down_need,
                        (unsigned long long)down_bytes);
    if (scratch_bytes < scratch_need)
        return api_fail(EIDM_E_SIZE, "the decode FFN needs %llu bytes of scratch, got %llu",
                        (unsigned long long)scratch_need, (unsigned long long)scratch_bytes);
    auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    if (bits(scratch) % 256) return api_fail(EIDM_E_ALIGN, "the decode FFN scratch must be 256-byte aligned");
    const int size = shape->weight_dtype == EIDM_DTYPE_F32 ? 4 : 2;
    if ((bits(w_gate) | bits(w_up) | bits(w_down)) % size)
        return api_fail(EIDM_E_ALIGN, "weights must be aligned to the scalar size");
    if ((bits(x) | bits(logits) | bits(ids) | bits(gates) | bits(out) | bits(bias)) % 4)
        return api_fail(EIDM_E_ALIGN, "decode FFN buffers must be 4-byte aligned");

    hipStream_t st = static_cast<hipStream_t>(stream);
    eidm::MoeDecodeArgs a{};
    a.dtype = shape->weight_dtype;
    a.m = shape->m;
    a.hidden = shape->hidden;
    a.inter = shape->inter;
    a.top_k = shape->top_k;
    a.n_experts = shape->n_experts;
    a.h_stride = eidm::h_stride(shape->inter);
    a.gate_up_stride = shape->gate_up_stride_bytes;
    a.down_stride = shape->down_stride_bytes;
    a.w_gate = static_cast<const uint8_t*>(w_gate);
    a.w_up = static_cast<const uint8_t*>(w_up);
    a.w_down = static_cast<const uint8_t*>(w_down);
    a.x = x;
    a.ids = ids;
    a.gates = gates;
    a.h = static_cast<float*>(scratch);
    a.out = out;
    hipError_t err = eidm::launch_route(logits, bias, a.m, a.n_experts, a.top_k, renormalize, ids, gates, st);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "route launch: %s", hipGetErrorString(err));
    err = eidm::launch_moe_decode(a, eidm::device_cus(), st);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "decode FFN launch: %s", hipGetErrorString(err));
    return eidm::api_ok();
}

}  // extern "C"
