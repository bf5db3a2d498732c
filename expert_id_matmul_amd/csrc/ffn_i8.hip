// ffn_i8.hip -- the mixture-of-experts expert FFN with 8-bit weights and rows
// (ffn.hip: the f32 one and its sources):
//
//   ids, gates = route(logits, bias)
//   xq = x in 8 bits, a scale for each token
//   g, u = the 8-bit products of xq with W_gate and W_up
//   h = silu(g) * u, rounded once to f32 from 64 bits
//   hq = h in 8 bits, a scale for each routed row
//   y = the 8-bit products of hq with W_down, out = combine(y, gates)
//
// Every rounding is defined and every sum of products exact, so the two forms
// have the same bits:
//   Direct   two or three launches: routing and x's quantising side by side (of
//            a few tokens, in the next launch); gate and up products of one
//            routed row at a time; the down products, quantising h as they read
//            it, and the combine.
//   Grouped  each expert's rows share its reads: routing and quantising, map,
//            gate and up tiles, h's quantising, down tiles, combine.
#include <hip/hip_runtime.h>

#include "api_checks.hpp"
#include "eidm.h"
#include "i8_args.hpp"
#include "quant8.hpp"
#include "route_wave.hpp"

namespace eidm {
namespace {

// Blocks below `quantising` (0 with x in 8 bits already): a token's x to 8 bits;
// the blocks after them: four tokens' routing.  Either kind takes tokens in turn.
template <int NV>
__global__ __launch_bounds__(256) void i8_ffn_start_kernel(const float* __restrict__ logits,
                                                           const float* __restrict__ bias, uint32_t m,
                                                           uint32_t n_experts, uint32_t top_k, int renormalize,
                                                           uint32_t* __restrict__ ids, float* __restrict__ gates,
                                                           const float* __restrict__ x, uint32_t hidden,
                                                           int8_t* __restrict__ q, float* __restrict__ scales,
                                                           uint32_t quantising) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (blockIdx.x >= quantising) {
        const uint32_t each = (gridDim.x - quantising) * 4;
        for (uint32_t t = (blockIdx.x - quantising) * 4 + wave; t < m; t += each) {
            uint32_t id;
            float gate;
            route_token<NV>(logits + (size_t)t * n_experts, bias, n_experts, top_k, renormalize, id, gate);
            if (lane < top_k) {
                ids[(size_t)t * top_k + lane] = id;
                gates[(size_t)t * top_k + lane] = gate;
            }
        }
        return;
    }
    __shared__ uint32_t part[4];
    constexpr uint32_t kHeld = 4;  // units of 8 a thread holds; longer rows are read twice
    for (uint32_t t = blockIdx.x; t < m; t += quantising) {
        const uint8_t* row = reinterpret_cast<const uint8_t*>(x + (size_t)t * hidden);
        float v[kHeld][8];
        uint32_t most = 0;
#pragma unroll
        for (uint32_t u = 0; u < kHeld; ++u) {
            load_row<kDtypeF32, 8>(row, min((u * 256 + threadIdx.x) * 8, hidden), hidden, v[u]);
#pragma unroll
            for (int j = 0; j < 8; ++j) most = max(most, magnitude(v[u][j]));
        }
        for (uint32_t i = (kHeld * 256 + threadIdx.x) * 8; i < hidden; i += 2048) {
            float w[8];
            load_row<kDtypeF32, 8>(row, i, hidden, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) most = max(most, magnitude(w[j]));
        }
        most = wave_max_u32(most);
        if (lane == 0) part[wave] = most;
        __syncthreads();
        const RowScale s = row_scale(max(max(part[0], part[1]), max(part[2], part[3])));
        if (threadIdx.x == 0) scales[t] = s.scale;
        int8_t* to = q + (size_t)t * hidden;
#pragma unroll
        for (uint32_t u = 0; u < kHeld; ++u) store_q(to, min((u * 256 + threadIdx.x) * 8, hidden), hidden, v[u], s);
        for (uint32_t i = (kHeld * 256 + threadIdx.x) * 8; i < hidden; i += 2048) {
            float w[8];
            load_row<kDtypeF32, 8>(row, i, hidden, w);
            store_q(to, i, hidden, w, s);
        }
        if (quantising < m) __syncthreads();  // the next token's maxima
    }
}

struct FfnI8Plan {
    uint64_t routed = 0, gate_up_bytes = 0, down_bytes = 0;
    // scratch: xq | x scales | h | hq | h scales | y | the down projection's map
    uint64_t xq = 0, xs = 0, h = 0, hq = 0, hs = 0, y = 0, map = 0, total = 0;
    eidm_i8_shape up{}, down{};
};

int check_ffn(const eidm_ffn_i8_shape* s, FfnI8Plan* p) {
    if (!s) return api_fail(EIDM_E_INVALID, "shape is NULL");
    if (s->struct_size != sizeof(eidm_ffn_i8_shape))
        return api_fail(EIDM_E_INVALID, "ffn shape struct_size %u, expected %zu", s->struct_size, sizeof(eidm_ffn_i8_shape));
    p->up = {sizeof(eidm_i8_shape), EIDM_LAYOUT_SHARED_PER_TOKEN, s->m, s->inter, s->hidden, s->top_k, s->n_experts, 0,
             s->gate_up_stride_bytes};
    p->down = {sizeof(eidm_i8_shape), EIDM_LAYOUT_SLOTTED, s->m, s->hidden, s->inter, s->top_k, s->n_experts, 0,
               s->down_stride_bytes};
    const uint64_t map_bytes = eidm_matmul_id_i8_scratch_bytes(&p->up);
    if (!map_bytes) return check_i8_shape(&p->up);
    if (!eidm_matmul_id_i8_scratch_bytes(&p->down)) return check_i8_shape(&p->down);
    if (s->top_k > kMaxRouterTopK || s->top_k > s->n_experts)
        return api_fail(s->top_k > s->n_experts ? EIDM_E_INVALID : EIDM_E_UNSUPPORTED,
                        "router limits: top_k <= min(n_experts, %u)", kMaxRouterTopK);
    p->routed = (uint64_t)s->m * s->top_k;
    const uint64_t body = (uint64_t)s->inter * s->hidden;
    p->gate_up_bytes = (s->n_experts - 1) * s->gate_up_stride_bytes + body;
    p->down_bytes = (s->n_experts - 1) * s->down_stride_bytes + body;
    // the products below stay under 2^31 * 131071 * 4 bytes each
    uint64_t at = 0;
    auto take = [&](uint64_t* where, uint64_t bytes) {
        *where = at;
        at = round256(at + bytes);
    };
    take(&p->xq, (uint64_t)s->m * s->hidden);
    take(&p->xs, (uint64_t)s->m * 4);
    take(&p->h, p->routed * s->inter * 4);
    take(&p->hq, p->routed * s->inter);
    take(&p->hs, p->routed * 4);
    take(&p->y, p->routed * s->hidden * 4);
    take(&p->map, map_bytes);
    p->total = at;
    return EIDM_OK;
}

bool ffn_i8_direct(const eidm_ffn_i8_shape* s) {
    return s->top_k <= kI8DownTopK &&
           i8_rows_by_themselves(s->m, s->top_k, s->n_experts, 3ull * s->hidden * s->inter,
                                 2 * i8_row_bytes(s->inter, s->hidden) + i8_row_bytes(s->hidden, s->inter));
}

bool direct_grid_fits(const eidm_ffn_i8_shape* s) {
    return (uint64_t)s->m * ((s->hidden + 7) / 8) * 64 * s->top_k < 1ull << 32;
}

// Routing, and x (if it is given) to 8 bits.
int launch_start(const eidm_ffn_i8_shape* s, const float* logits, const float* bias, int renormalize, uint32_t* ids,
                 float* gates, const float* x, int8_t* q, float* scales, hipStream_t st) {
    // a token or four to a block while the launch has fewer than 2^32 threads
    constexpr uint32_t kMost = 1u << 22;
    const uint32_t quantising = x ? (s->m < kMost ? s->m : kMost) : 0, fours = (s->m + 3) / 4;
    const uint32_t grid = quantising + (fours < kMost ? fours : kMost), nv = (s->n_experts + 63) / 64;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, st, logits, bias, s->m, s->n_experts, s->top_k, renormalize,
                           ids, gates, x, s->hidden, q, scales, quantising);
    };
    if (nv <= 1) go(i8_ffn_start_kernel<1>);
    else if (nv <= 2) go(i8_ffn_start_kernel<2>);
    else if (nv <= 4) go(i8_ffn_start_kernel<4>);
    else if (nv <= 8) go(i8_ffn_start_kernel<8>);
    else if (nv <= 16) go(i8_ffn_start_kernel<16>);
    else go(i8_ffn_start_kernel<32>);
    const hipError_t err = launched(EIDM_KERNEL_I8_FFN_START, grid, 256, 0);
    return err == hipSuccess ? EIDM_OK : api_fail(EIDM_E_DEVICE, "routing launch: %s", hipGetErrorString(err));
}

}  // namespace
}  // namespace eidm

extern "C" {

using namespace eidm;

uint64_t eidm_moe_ffn_i8_scratch_bytes(const eidm_ffn_i8_shape* shape) {
    FfnI8Plan p;
    if (check_ffn(shape, &p) != EIDM_OK) return 0;
    api_ok();
    return p.total;
}

int eidm_moe_ffn_i8(const eidm_ffn_i8_shape* shape, int route, const int8_t* w_gate, const float* gate_scales,
                    const int8_t* w_up, const float* up_scales, uint64_t gate_up_bytes, const int8_t* w_down,
                    const float* down_scales, uint64_t down_bytes, const float* x, const int8_t* xq,
                    const float* x_scales, const float* logits, const float* bias, int renormalize, uint32_t* ids,
                    float* gates, float* out, void* scratch, uint64_t scratch_bytes, void* stream, int* route_taken) {
    ReceiptScope receipt;
    FfnI8Plan p;
    const int rc = check_ffn(shape, &p);
    if (rc) return rc;
    const eidm_ffn_i8_shape* s = shape;
    if (!w_gate || !gate_scales || !w_up || !up_scales || !w_down || !down_scales || !logits || !ids || !gates || !out ||
        !scratch)
        return api_fail(EIDM_E_INVALID, "an FFN buffer is NULL");
    if (x ? (xq || x_scales) : (!xq || !x_scales))
        return api_fail(EIDM_E_INVALID, "exactly one of x and (xq with x_scales) is given");
    if (gate_up_bytes < p.gate_up_bytes || down_bytes < p.down_bytes)
        return api_fail(EIDM_E_SIZE, "weights: %llu and %llu bytes needed, %llu and %llu given",
                        (unsigned long long)p.gate_up_bytes, (unsigned long long)p.down_bytes,
                        (unsigned long long)gate_up_bytes, (unsigned long long)down_bytes);
    if (scratch_bytes < p.total)
        return api_fail(EIDM_E_SIZE, "the FFN needs %llu bytes of scratch, got %llu", (unsigned long long)p.total,
                        (unsigned long long)scratch_bytes);
    if (!is_aligned(scratch, 256)) return api_fail(EIDM_E_ALIGN, "the FFN scratch must be 256-byte aligned");
    if (!is_aligned(gate_scales, 4) || !is_aligned(up_scales, 4) || !is_aligned(down_scales, 4) || !is_aligned(x, 4) ||
        !is_aligned(x_scales, 4) || !is_aligned(logits, 4) || !is_aligned(bias, 4) || !is_aligned(ids, 4) ||
        !is_aligned(gates, 4) || !is_aligned(out, 4))
        return api_fail(EIDM_E_ALIGN, "FFN buffers must be 4-byte aligned");
    if (route != EIDM_ROUTE_AUTO && route != EIDM_ROUTE_DIRECT && route != EIDM_ROUTE_GROUPED)
        return api_fail(EIDM_E_INVALID, "unknown route %d", route);
    if (route == EIDM_ROUTE_DIRECT && (s->top_k > kI8DownTopK || !direct_grid_fits(s)))
        return api_fail(EIDM_E_UNSUPPORTED, "the Direct form takes top_k <= %u and fewer than 2^32 threads", kI8DownTopK);
    const bool direct = route == EIDM_ROUTE_DIRECT || (route == EIDM_ROUTE_AUTO && ffn_i8_direct(s) && direct_grid_fits(s));

    hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(scratch);
    int8_t* q = reinterpret_cast<int8_t*>(ws + p.xq);
    float* qs = reinterpret_cast<float*>(ws + p.xs);
    float* h = reinterpret_cast<float*>(ws + p.h);
    I8Args a{};
    a.m = s->m;
    a.n = s->inter;
    a.k = s->hidden;
    a.top_k = s->top_k;
    a.n_experts = s->n_experts;
    a.stride = s->gate_up_stride_bytes;
    a.w = w_gate;
    a.w2 = w_up;
    a.ws = gate_scales;
    a.ws2 = up_scales;
    a.x = x ? q : xq;
    a.xs = x ? qs : x_scales;
    a.ids = ids;
    a.out = h;
    const bool one = direct && i8_one_supported(a, device_cus());
    hipError_t err;
    if (one) {
        err = launch_i8_gate_up_one({a, x, logits, bias, renormalize, ids, gates}, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "gate and up launch: %s", hipGetErrorString(err));
    } else {
        const int rc = launch_start(s, logits, bias, renormalize, ids, gates, x, q, qs, st);
        if (rc) return rc;
    }
    if (direct) {
        err = one ? hipSuccess : launch_i8_rows(a, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "gate and up launch: %s", hipGetErrorString(err));
        const I8DownArgs d{s->m, s->hidden, s->inter, s->top_k, s->n_experts, s->down_stride_bytes, w_down, down_scales,
                           h, ids, gates, out};
        err = launch_i8_down_combine(d, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "down launch: %s", hipGetErrorString(err));
    } else {
        const MapBuffers map = i8_map_at(&p.up, ws + p.map);
        err = launch_map(ids, (uint32_t)p.routed, s->n_experts, map, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "map launch: %s", hipGetErrorString(err));
        a.offsets = map.offsets;
        a.rows = map.rows;
        err = launch_i8_tiles(a, device_cus(), st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "gate and up launch: %s", hipGetErrorString(err));
        int8_t* hq = reinterpret_cast<int8_t*>(ws + p.hq);
        float* hs = reinterpret_cast<float*>(ws + p.hs);
        float* y = reinterpret_cast<float*>(ws + p.y);
        err = launch_quantize_rows(kDtypeF32, h, (uint32_t)p.routed, s->inter, hq, hs, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "quantise launch: %s", hipGetErrorString(err));
        a.n = s->hidden;
        a.k = s->inter;
        a.stride = s->down_stride_bytes;
        a.slotted = true;
        a.w = w_down;
        a.w2 = nullptr;
        a.ws = down_scales;
        a.ws2 = nullptr;
        a.x = hq;
        a.xs = hs;
        a.out = y;
        err = launch_i8_tiles(a, device_cus(), st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "down launch: %s", hipGetErrorString(err));
        err = launch_combine(s->m, s->top_k, s->hidden, y, gates, out, st);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "combine launch: %s", hipGetErrorString(err));
    }
    const int taken = direct ? EIDM_ROUTE_DIRECT : EIDM_ROUTE_GROUPED;
    receipt_route(taken);
    if (route_taken) *route_taken = taken;
    return api_ok();
}

}  // extern "C"
