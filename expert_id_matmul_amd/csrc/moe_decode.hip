// moe_decode.hip -- the expert FFN of a few tokens (m <= 64):
//   gate/up kernel: h[r] = silu(W_gate[e] x[t]) * (W_up[e] x[t]) for every
//     routed row r = t*top_k + s of expert e, both products and the
//     activation in one pass over the two weights; with few tokens it also
//     routes them;
//   down kernel: with few rows, out[t] = sum_s gate[t, s] W_down[e] h[r], a
//     block owning a few output columns of every token, so the sum over slots
//     is taken in LDS in slot order; with more rows y[r] = W_down[e] h[r],
//     which the library's combine sums.
// Each touched expert's weights are read once per call, however many tokens
// chose it (up to 16 rows at a time).
//
// Every product is in the library's fixed reduction order, routing, silu and
// the combine are the same operations as the separate kernels', so the
// results are bit for bit those of eidm_moe_ffn.
//
// cortiq-engine 0.7.7, src/mimo_moe.rs, Dynamic::run (route, one FFN per
// pick, weighted sum); hf2q dense_ffn_arena.rs, MoeFfnArena (gate, up, h, y).
#include <atomic>

#include "eidm_device.hpp"
#include "eidm_internal.hpp"
#include "few_map.hpp"
#include "few_rows.hpp"
#include "route_wave.hpp"

namespace eidm {
namespace {

constexpr int kWaves = 8;  // wavefronts per block
// LDS for staged activation rows: 16 rows of 2048, one of the longest k
// (kMaxDecodeRow)
constexpr uint32_t kRowBytes = 16 * few_row_floats(2048) * 4;
static_assert(few_row_floats(kMaxDecodeRow) * 4 <= kRowBytes);
constexpr uint32_t kRouteExperts = 256;  // experts a block routes itself (4 per lane)

// most rows of k elements staged at once
__host__ __device__ constexpr uint32_t row_cap(uint32_t k) { return kRowBytes / (few_row_floats(k) * 4); }

// Rounds in flight: 16 16-byte loads per lane.  (C weight rows per lane; one
// load each for 16-bit weights, two for f32.)
template <int DT, int C>
constexpr int few_depth() { return 32 / (C * DtypeSize<DT>::value); }

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// Column-group jobs (expert u, group g) of all touched experts in order, cut
// into one contiguous range per block, so that a block meets one or two
// experts: it stages their rows in LDS and its wavefronts take the range's
// jobs in turn.  An expert whose rows do not fit takes several passes over
// its weights.  row_of(routed row): the activation row of k elements.
// weight_of(expert, group, wrow): this lane's weight rows.
// emit(routed row, group, totals).
template <int DT, int C, typename RowOf, typename WeightOf, typename Emit>
__device__ __forceinline__ void expert_major(const FewMap& map, float* xs, uint32_t groups, uint32_t k, RowOf row_of,
                                             WeightOf weight_of, Emit emit) {
    const uint32_t jobs = *map.used * groups;
    const uint32_t stride = few_row_floats(k);
    const uint32_t most = row_cap(k);
    const uint32_t per_expert = min(most, (uint32_t)kFewRows);
    uint32_t pos = (uint32_t)((uint64_t)jobs * blockIdx.x / gridDim.x);
    const uint32_t last = (uint32_t)((uint64_t)jobs * (blockIdx.x + 1) / gridDim.x);
    while (pos < last) {  // block-uniform
        uint32_t v = pos / groups;  // experts pos/groups .. v in this pass
        const uint32_t first = map.off[v];
        uint32_t end = map.off[v + 1];
        uint32_t passes = 1;
        if (end - first > per_expert) {
            passes = (end - first + per_expert - 1) / per_expert;
        } else {
            while ((v + 1) * groups < last && map.off[v + 2] - end <= per_expert && map.off[v + 2] - first <= most) {
                ++v;
                end = map.off[v + 1];
            }
        }
        const uint32_t stop = min(last, (v + 1) * groups);
        for (uint32_t p = 0; p < passes; ++p) {
            const uint32_t base = first + p * per_expert;
            const uint32_t limit = passes == 1 ? end : min(end, base + per_expert);
            __syncthreads();  // the rows of the pass before are done with
            few_rows_stage(xs, limit - base, k, [&](uint32_t i) { return row_of(map.row[base + i]); });
            __syncthreads();
            for (uint32_t job = pos + (threadIdx.x >> 6); job < stop; job += kWaves) {
                const uint32_t u = uniform(job / groups);
                const uint32_t g = uniform(job) - u * groups;
                const uint32_t from = max(uniform(map.off[u]), base), to = min(uniform(map.off[u + 1]), limit);
                const uint8_t* wrow[C];
                weight_of(uniform(map.id[u]), g, wrow);
                few_rows_any<DT, C, few_depth<DT, C>(), true>(
                    wrow, xs, stride, from - base, to - from, (int)k,
                    [&](uint32_t i, const float (&t)[C]) { emit(map.row[base + i], g, t); });
            }
        }
        pos = stop;
    }
}

// ROUTE: the block routes the call's tokens (at most one per wavefront)
// itself, every block the same, and the first block writes ids and gates.
template <int DT, bool ROUTE>
__global__ __launch_bounds__(64 * kWaves) void gate_up_kernel(MoeDecodeArgs a) {
    constexpr int S = DtypeSize<DT>::value;
    extern __shared__ __align__(16) uint32_t lds[];
    const uint32_t rows = a.m * a.top_k;
    const FewMap map = few_map_at(lds, rows, a.n_experts);
    float* xs = reinterpret_cast<float*>(lds + few_map_words(rows, a.n_experts));
    if constexpr (ROUTE) {
        __shared__ uint32_t picks[kWaves * kMaxDecodeTopK];
        const uint32_t t = threadIdx.x >> 6, lane = threadIdx.x & 63;
        if (t < a.m) {
            uint32_t id;
            float gate;
            route_token<kRouteExperts / 64>(a.logits + (size_t)t * a.n_experts, a.bias, a.n_experts, a.top_k,
                                            a.renormalize, id, gate);
            if (lane < a.top_k) {
                picks[t * a.top_k + lane] = id;
                if (blockIdx.x == 0) {
                    a.ids[t * a.top_k + lane] = id;
                    a.gates[t * a.top_k + lane] = gate;
                }
            }
        }
        __syncthreads();
        few_map_build(map, picks, rows, a.n_experts, a.m);
    } else {
        few_map_build(map, a.ids, rows, a.n_experts, a.m);
    }

    const uint32_t q = threadIdx.x & 3;
    expert_major<DT, 2>(
        map, xs, (a.inter + 3) / 4, a.hidden, [&](uint32_t r) { return a.x + (size_t)(r / a.top_k) * a.hidden; },
        [&](uint32_t e, uint32_t g, const uint8_t* (&wrow)[2]) {
            const size_t at = (size_t)e * a.gate_up_stride + (size_t)min(g * 4 + q, a.inter - 1) * a.hidden * S;
            wrow[0] = a.w_gate + at;
            wrow[1] = a.w_up + at;
        },
        [&](uint32_t r, uint32_t g, const float (&t)[2]) {
            if (g * 4 + q < a.inter) a.h[(size_t)r * a.inter + g * 4 + q] = silu_mul(t[0], t[1]);
        });
}

// y[r] = W_down[e] h[r], 4*C columns per job
template <int DT, int C>
__global__ __launch_bounds__(64 * kWaves) void down_kernel(MoeDecodeArgs a) {
    constexpr int S = DtypeSize<DT>::value;
    extern __shared__ __align__(16) uint32_t lds[];
    const uint32_t rows = a.m * a.top_k;
    const FewMap map = few_map_at(lds, rows, a.n_experts);
    float* xs = reinterpret_cast<float*>(lds + few_map_words(rows, a.n_experts));
    few_map_build(map, a.ids, rows, a.n_experts, a.m);
    const uint32_t q = threadIdx.x & 3;
    expert_major<DT, C>(
        map, xs, (a.hidden + 4 * C - 1) / (4 * C), a.inter, [&](uint32_t r) { return a.h + (size_t)r * a.inter; },
        [&](uint32_t e, uint32_t g, const uint8_t* (&wrow)[C]) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                wrow[c] = a.w_down + (size_t)e * a.down_stride +
                          (size_t)min((g * C + c) * 4 + q, a.hidden - 1) * a.inter * S;
        },
        [&](uint32_t r, uint32_t g, const float (&t)[C]) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint32_t col = (g * C + c) * 4 + q;
                if (col < a.hidden) a.y[(size_t)r * a.hidden + col] = t[c];
            }
        });
}

// Few rows: all of h staged; a block owns `cols` <= 4*C output columns of
// every token, its wavefronts take the touched experts in turn.
template <int DT, int C>
__global__ __launch_bounds__(64 * kWaves) void down_combine_kernel(MoeDecodeArgs a, uint32_t cols) {
    constexpr int S = DtypeSize<DT>::value;
    extern __shared__ __align__(16) uint32_t lds[];
    const uint32_t rows = a.m * a.top_k;
    const FewMap map = few_map_at(lds, rows, a.n_experts);
    float* ys = reinterpret_cast<float*>(lds + few_map_words(rows, a.n_experts));  // [rows][4*C]
    float* xs = ys + rows * 4 * C;
    few_map_build(map, a.ids, rows, a.n_experts, a.m);
    few_rows_stage(xs, rows, a.inter, [&](uint32_t i) { return a.h + (size_t)map.row[i] * a.inter; });
    __syncthreads();

    const uint32_t q = threadIdx.x & 3;
    const uint32_t col0 = blockIdx.x * cols;
    const uint32_t used = *map.used;
    for (uint32_t w = threadIdx.x >> 6; w < used; w += kWaves) {
        const uint32_t u = uniform(w);
        const uint32_t from = uniform(map.off[u]), to = uniform(map.off[u + 1]);
        const uint8_t* wrow[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint32_t col = 4 * c + q < cols ? min(col0 + 4 * c + q, a.hidden - 1) : col0;
            wrow[c] = a.w_down + (size_t)uniform(map.id[u]) * a.down_stride + (size_t)col * a.inter * S;
        }
        for (uint32_t at = from; at < to; at += kFewRows)
            few_rows_any<DT, C, few_depth<DT, C>(), true>(
                wrow, xs, few_row_floats(a.inter), at, min(to - at, (uint32_t)kFewRows), (int)a.inter,
                [&](uint32_t i, const float (&t)[C]) {
#pragma unroll
                    for (int c = 0; c < C; ++c) ys[map.row[i] * (4 * C) + 4 * c + q] = t[c];
                });
    }
    __syncthreads();
    const uint32_t live = min(cols, a.hidden - col0);
    for (uint32_t i = threadIdx.x; i < a.m * 4 * C; i += blockDim.x) {
        const uint32_t t = i / (4 * C), c = i % (4 * C);
        if (c < live) {
            float acc = 0.0f;
            for (uint32_t s = 0; s < a.top_k; ++s) {
                const uint32_t r = t * a.top_k + s;
                acc = __builtin_fmaf(a.gates[r], ys[r * (4 * C) + c], acc);
            }
            a.out[(size_t)t * a.hidden + col0 + c] = acc;
        }
    }
}

// Allows a kernel the whole LDS of a compute unit, once per device.
hipError_t allow_lds(const void* kernel, std::atomic<uint64_t>& done) {
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    err = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024 - 1024);
    if (err == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

template <typename Kernel, typename... Args>
hipError_t launch_one(int receipt, Kernel kernel, std::atomic<uint64_t>& done, uint32_t grid, uint32_t lds,
                      hipStream_t stream, Args... args) {
    if (lds > 64 * 1024) {
        const hipError_t err = allow_lds(reinterpret_cast<const void*>(kernel), done);
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * kWaves), lds, stream, args...);
    return launched(receipt, grid, 64 * kWaves, lds);
}

// Every row of h fits in LDS beside the map and the output rows
bool combine_in_down(const MoeDecodeArgs& a) { return a.m * a.top_k <= row_cap(a.inter); }

template <int DT>
hipError_t launch_dt(const MoeDecodeArgs& a, int device_cus, hipStream_t stream) {
    static std::atomic<uint64_t> done[6];
    const uint32_t rows = a.m * a.top_k;
    const uint32_t touched = few_map_ids(rows, a.n_experts);  // at most
    const uint32_t map_bytes = few_map_words(rows, a.n_experts) * 4;
    const uint32_t cus = device_cus > 0 ? (uint32_t)device_cus : 256;
    auto blocks_of = [&](uint32_t groups) {
        const uint64_t jobs = (uint64_t)touched * groups;
        return (uint32_t)(jobs < cus ? jobs : cus);
    };
    auto staged = [&](uint32_t k) { return (rows < row_cap(k) ? rows : row_cap(k)) * few_row_floats(k) * 4; };
    const bool route = a.m <= (uint32_t)kWaves && a.n_experts <= kRouteExperts;
    hipError_t err = hipSuccess;
    if (!route) {
        err = launch_route(a.logits, a.bias, a.m, a.n_experts, a.top_k, a.renormalize, a.ids, a.gates, stream);
        if (err != hipSuccess) return err;
    }
    const uint32_t up_blocks = blocks_of((a.inter + 3) / 4), up_lds = map_bytes + staged(a.hidden);
    err = route ? launch_one(EIDM_KERNEL_DECODE_GATE_UP, gate_up_kernel<DT, true>, done[0], up_blocks, up_lds, stream, a)
                : launch_one(EIDM_KERNEL_DECODE_GATE_UP, gate_up_kernel<DT, false>, done[1], up_blocks, up_lds, stream, a);
    if (err != hipSuccess) return err;
    if (combine_in_down(a)) {
        const uint32_t cols = a.hidden >= 8 * cus ? 8 : 4;
        const uint32_t blocks = (a.hidden + cols - 1) / cols;
        const uint32_t lds = map_bytes + rows * cols * 4 + staged(a.inter);
        return cols == 8 ? launch_one(EIDM_KERNEL_DECODE_DOWN, down_combine_kernel<DT, 2>, done[2], blocks, lds, stream, a, cols)
                         : launch_one(EIDM_KERNEL_DECODE_DOWN, down_combine_kernel<DT, 1>, done[3], blocks, lds, stream, a, cols);
    }
    err = launch_one(EIDM_KERNEL_DECODE_DOWN, down_kernel<DT, 4>, done[4], blocks_of((a.hidden + 15) / 16),
                     map_bytes + staged(a.inter), stream, a);
    if (err != hipSuccess) return err;
    return launch_combine(a.m, a.top_k, a.hidden, a.y, a.gates, a.out, stream);
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

// scratch: h [m*top_k][inter] | y [m*top_k][hidden]
uint64_t h_bytes(const eidm_ffn_shape* f) {
    return ((uint64_t)f->m * f->top_k * f->inter * 4 + 255) & ~uint64_t(255);
}

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
    if (f->hidden > kMaxDecodeRow || f->inter > kMaxDecodeRow)
        return api_fail(EIDM_E_UNSUPPORTED, "hidden %u, inter %u: the decode FFN takes rows of at most %u", f->hidden,
                        f->inter, kMaxDecodeRow);
    *gate_up = rg.required_weight_bytes;
    *down = rd.required_weight_bytes;
    *scratch = h_bytes(f) + (uint64_t)f->m * f->top_k * f->hidden * 4;
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
    a.gate_up_stride = shape->gate_up_stride_bytes;
    a.down_stride = shape->down_stride_bytes;
    a.w_gate = static_cast<const uint8_t*>(w_gate);
    a.w_up = static_cast<const uint8_t*>(w_up);
    a.w_down = static_cast<const uint8_t*>(w_down);
    a.x = x;
    a.logits = logits;
    a.bias = bias;
    a.renormalize = renormalize;
    a.ids = ids;
    a.gates = gates;
    a.h = static_cast<float*>(scratch);
    a.y = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + eidm::h_bytes(shape));
    a.out = out;
    const hipError_t err = eidm::launch_moe_decode(a, eidm::device_cus(), st);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "decode FFN launch: %s", hipGetErrorString(err));
    return eidm::api_ok();
}

}  // extern "C"
