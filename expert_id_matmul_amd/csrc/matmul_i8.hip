// matmul_i8.hip -- products of 8-bit integers with a scale for each routed row
// and each channel, by expert ids or with one weight for all rows:
//
//   y[r, j] = (f32(sum_c W_e[j, c] * x_row(r)[c]) * sx[row(r)]) * sw[e, j]
//
// The sums are 32-bit integers (k is bounded so that none overflows) and
// therefore exact: every form below gives the same bits, in any order.
//
// Rows (a wavefront takes a routed row and a few of its columns): bound by
// HBM.  16 bytes a lane make 1 KB of one weight row a load, and 16 loads are
// in flight; the row's own bytes stay in registers for all columns.  One token
// of 8 of 256 experts of 1536 x 4096 (50 MB): 10.4 us, 4.8 TB/s.
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "api_checks.hpp"
#include "eidm.h"
#include "few_map.hpp"
#include "i8_args.hpp"
#include "quant8.hpp"
#include "route_wave.hpp"

namespace eidm {
namespace {

__device__ __forceinline__ int dot4(uint32_t a, uint32_t b, int acc) {
    return __builtin_amdgcn_sdot4((int)a, (int)b, acc, false);
}

__device__ __forceinline__ int dot16(u32x4 a, u32x4 b, int acc) {
    return dot4(a.w, b.w, dot4(a.z, b.z, dot4(a.y, b.y, dot4(a.x, b.x, acc))));
}

// Sum over the wavefront, the same in every lane.
__device__ __forceinline__ int wave_total(int v) {
    return __builtin_amdgcn_readlane((int)wave_prefix((uint32_t)v), 63);
}

// C weight rows times one row of x over the wavefront: acc[c] per lane.
// ONCE: the weights past the caches.
template <int C, bool ONCE, typename LoadX>
__device__ __forceinline__ void row_products(const int8_t* const (&w)[C], uint32_t k, LoadX load_x, int (&acc)[C]) {
    constexpr int U = 16 / C;  // units of 1 KB a weight row and turn: 16 loads in flight
    const uint32_t lane = threadIdx.x & 63;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0;
    if (k < 16) {
        const u32x4 xv = load_x(0);
        if (lane == 0)
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = dot16(load_unit_bytes(w[c], 0, k), xv, 0);
        return;
    }
    for (uint32_t k0 = 0; k0 < k; k0 += 1024 * U) {
        u32x4 wv[C][U], xv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t kk = k0 + u * 1024 + lane * 16;
            if (k0 + u * 1024 < k) {  // the same for all lanes
#pragma unroll
                for (int c = 0; c < C; ++c) wv[c][u] = load_unit<ONCE>(w[c], kk, k);
                xv[u] = load_x(kk);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + u * 1024 < k)
#pragma unroll
                for (int c = 0; c < C; ++c) acc[c] = dot16(wv[c][u], xv[u], acc[c]);
    }
}

// DUAL: C / 2 columns of gate and of up, out = silu(gate) * up
template <int C, bool DUAL, bool ONCE>
__global__ __launch_bounds__(256) void i8_rows_kernel(I8Args a, uint32_t groups, uint64_t jobs) {
    constexpr int N = DUAL ? C / 2 : C;  // columns of a job
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    for (uint64_t job = (uint64_t)blockIdx.x * 4 + wave; job < jobs; job += (uint64_t)gridDim.x * 4) {
        const uint32_t r = (uint32_t)(job / groups), col = (uint32_t)(job % groups) * N;
        const uint32_t e = a.ids ? (uint32_t)__builtin_amdgcn_readfirstlane((int)a.ids[r]) : 0;
        float* y = a.out + (size_t)r * a.n;
        if (e >= a.n_experts) {
            if (lane < N && col + lane < a.n) y[col + lane] = quiet_nan();
            continue;
        }
        const uint32_t in = a.slotted ? r : r / a.top_k;
        const int8_t* x = a.x + (size_t)in * a.k;
        const int8_t* w[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint32_t j = min(col + c % N, a.n - 1);
            w[c] = (c < N ? a.w : a.w2) + e * a.stride + (size_t)j * a.k;
        }
        const float sx = a.xs[in];
        const uint32_t j = min(col + lane % N, a.n - 1);
        const float sw = a.ws[(size_t)e * a.n + j];
        const float sw2 = DUAL ? a.ws2[(size_t)e * a.n + j] : 0.0f;
        int acc[C];
        const uint32_t k = a.k;
        row_products<C, ONCE>(w, k, [&](uint32_t kk) {
            return k < 16 ? load_unit_bytes(x, 0, k) : unit_keep(load_unit(x, kk, k), kk, k);
        }, acc);
        int mine = 0, mine2 = 0;  // lane c < N: column c's sums
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int t = wave_total(acc[c]);
            if ((int)lane % N == c % N) (c < N ? mine : mine2) = t;
        }
        float v = scaled_sum(mine, sx, sw);
        if constexpr (DUAL) v = silu_mul(v, scaled_sum(mine2, sx, sw2));
        if (lane < N && col + lane < a.n) y[col + lane] = v;
    }
}

// Gate and up products of a few tokens with the routing and x's quantising in
// the same launch: a block takes four column groups of one routed row, routes
// its token and quantises its x by itself (from the L2), which takes some 2 us
// before the weights start, and saves a launch and its start (7.6 us for 25 MB
// of 8 experts of 768 x 2048).  The block of a token's first row and columns
// writes its ids and gates.
template <int NV, bool ONCE>
__global__ __launch_bounds__(256) void i8_gate_up_one_kernel(I8OneArgs o, uint32_t blocks_a_row) {
    constexpr int C = 4, N = 2;
    __shared__ float score[64 * NV];
    __shared__ uint32_t code[64 * NV];
    __shared__ uint32_t part[4];
    extern __shared__ u32x4 x_lds[];  // a's k bytes
    int8_t* xq = reinterpret_cast<int8_t*>(x_lds);
    const I8Args& a = o.a;
    const uint32_t tid = threadIdx.x, lane = tid & 63, k = a.k;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
    const uint32_t r = blockIdx.x / blocks_a_row, t = r / a.top_k, slot = r % a.top_k;
    const uint32_t col = (blockIdx.x % blocks_a_row * 4 + wave) * N;
    RouteInputs<NV> in;
    route_inputs_issue<NV>(o.logits + (size_t)t * a.n_experts, o.bias, a.n_experts, in);
    constexpr uint32_t kHeld = kI8OneRow / 2048;  // units of 8 a thread holds
    float v[kHeld][8];
    uint32_t top = 0;
    if (o.x) {
        const uint8_t* row = reinterpret_cast<const uint8_t*>(o.x + (size_t)t * k);
#pragma unroll
        for (uint32_t u = 0; u < kHeld; ++u)
            if (u * 2048 < k) load_row<kDtypeF32, 8>(row, min((u * 256 + tid) * 8, k), k, v[u]);
    } else {
        for (uint32_t i = tid; i < k; i += 256) xq[i] = a.x[(size_t)t * k + i];
    }
    route_inputs_score<NV>(in, a.n_experts, score, code);
    if (o.x) {
#pragma unroll
        for (uint32_t u = 0; u < kHeld; ++u)
            if (u * 2048 < k)
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, magnitude(v[u][j]));
        top = wave_max_u32(top);
        if (lane == 0) part[wave] = top;
    }
    __syncthreads();
    float sx;
    if (o.x) {
        const RowScale s = row_scale(max(max(part[0], part[1]), max(part[2], part[3])));
        sx = s.scale;
#pragma unroll
        for (uint32_t u = 0; u < kHeld; ++u)
            if (u * 2048 < k) store_q(xq, min((u * 256 + tid) * 8, k), k, v[u], s);
    } else {
        sx = a.xs[t];
    }
    // every wavefront picks for itself, as far as this row's slot; one of the token, all of them
    const bool writes = slot == 0 && blockIdx.x % blocks_a_row == 0 && wave == 0;
    RouteScores<NV> sc;
    route_scores_lds<NV>(score, code, sc);
    uint32_t id;
    float mine_score;
    const float sum = route_select<NV>(sc, writes ? a.top_k : slot + 1, id, mine_score);
    if (writes && lane < a.top_k) {
        o.ids[(size_t)t * a.top_k + lane] = id;
        o.gates[(size_t)t * a.top_k + lane] = o.renormalize ? __fdiv_rn(mine_score, sum) : mine_score;
    }
    const uint32_t e = (uint32_t)__builtin_amdgcn_readlane((int)id, (int)slot);
    __syncthreads();
    if (col >= a.n) return;  // a wavefront past the columns
    const int8_t* w[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
        w[c] = (c < N ? a.w : a.w2) + e * a.stride + (size_t)min(col + c % N, a.n - 1) * k;
    const uint32_t j = min(col + lane % N, a.n - 1);
    const float sw = a.ws[(size_t)e * a.n + j], sw2 = a.ws2[(size_t)e * a.n + j];
    int acc[C];
    row_products<C, ONCE>(w, k, [&](uint32_t kk) {
        return k < 16 ? load_unit_bytes(xq, 0, k) : unit_keep(load_unit(xq, kk, k), kk, k);
    }, acc);
    int mine = 0, mine2 = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int total = wave_total(acc[c]);
        if ((int)lane % N == c % N) (c < N ? mine : mine2) = total;
    }
    if (lane < N && col + lane < a.n)
        a.out[(size_t)r * a.n + col + lane] = silu_mul(scaled_sum(mine, sx, sw), scaled_sum(mine2, sx, sw2));
}

// One block: a token and C columns of its output, a wavefront per slot.  The
// weights of the first U KB of a row are requested before anything else; h,
// which the launch before left in the L2, is quantised meanwhile, by every
// block again (its largest magnitude handed on by atomics took 30 us for one
// token: thousands of maxima on a cache line).  6.0 us for the 12.6 MB of the
// same 8 experts: two thirds are the launch, the ids and h from the L2.
template <int C, int U, int SLOTS, bool ONCE>
__global__ __launch_bounds__(64 * SLOTS) void i8_down_combine_kernel(I8DownArgs a, uint32_t groups) {
    __shared__ float y[SLOTS][C];
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t s = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t t = blockIdx.x / groups, col = blockIdx.x % groups * C;
    const uint32_t r = t * a.top_k + s, k = a.k;
    const uint32_t e = (uint32_t)__builtin_amdgcn_readfirstlane((int)a.ids[r]);
    const uint32_t j = min(col + lane % C, a.n - 1);
    const int8_t* w[C];
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = a.w + e * a.stride + (size_t)min(col + c, a.n - 1) * k;
    const uint8_t* h = reinterpret_cast<const uint8_t*>(a.h + (size_t)r * k);
    int acc[C] = {};
    u32x4 wv[C][U];
    auto load_w = [&](uint32_t k0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + u * 1024 < k)  // the same for all lanes
#pragma unroll
                for (int c = 0; c < C; ++c) wv[c][u] = load_unit<ONCE>(w[c], k0 + u * 1024 + lane * 16, k);
    };
    // 16 values of h as load_unit() lays them out
    auto load_h = [&](uint32_t kk, float (&v)[16]) {
        const uint32_t from = k < 16 ? 0u : min(kk, k - 16);
        load_row<kDtypeF32, 8>(h, from, k, *reinterpret_cast<float(*)[8]>(v));
        load_row<kDtypeF32, 8>(h, from + 8, k, *reinterpret_cast<float(*)[8]>(v + 8));
    };
    if (k >= 16) load_w(0);
    const float sw = a.ws[(size_t)e * a.n + j];
    float v[U][16];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (u * 1024 < k) {
            load_h(u * 1024 + lane * 16, v[u]);
#pragma unroll
            for (int i = 0; i < 16; ++i) top = max(top, magnitude(v[u][i]));
        }
    for (uint32_t kk = U * 1024 + lane * 16; kk < k; kk += 1024) {
        float more[16];
        load_h(kk, more);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, magnitude(more[i]));
    }
    const RowScale scale = row_scale(wave_max_u32(top));
    auto pack = [&](uint32_t kk, const float (&x)[16]) {
        int q[16];
        quantized(x, scale, q);
        const u32x4 p = {pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]), pack4(q[8], q[9], q[10], q[11]),
                         pack4(q[12], q[13], q[14], q[15])};
        return k < 16 ? p : unit_keep(p, kk, k);
    };
    if (k < 16) {
        const u32x4 p = pack(0, v[0]);
        if (lane == 0)
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = dot16(load_unit_bytes(w[c], 0, k), p, 0);
    } else {
        for (uint32_t k0 = 0;;) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + u * 1024 < k) {
                    const u32x4 p = pack(k0 + u * 1024 + lane * 16, v[u]);
#pragma unroll
                    for (int c = 0; c < C; ++c) acc[c] = dot16(wv[c][u], p, acc[c]);
                }
            k0 += U * 1024;
            if (k0 >= k) break;
            load_w(k0);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + u * 1024 < k) load_h(k0 + u * 1024 + lane * 16, v[u]);
        }
    }
    int mine = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int total = wave_total(acc[c]);
        if ((int)lane % C == c) mine = total;
    }
    if (lane < C) y[s][lane] = scaled_sum(mine, scale.scale, sw);
    __syncthreads();
    if (threadIdx.x < C && col + threadIdx.x < a.n) {
        float v = 0.0f;
        for (uint32_t i = 0; i < a.top_k; ++i) v = __builtin_fmaf(a.gates[(size_t)t * a.top_k + i], y[i][threadIdx.x], v);
        a.out[(size_t)t * a.n + col + threadIdx.x] = v;
    }
}

}  // namespace

hipError_t launch_i8_rows(const I8Args& a, hipStream_t stream) {
    constexpr int C = 4;
    const bool dual = a.w2 != nullptr;
    const uint32_t each = dual ? C / 2 : C, groups = (a.n + each - 1) / each;
    const uint64_t jobs = (uint64_t)a.m * a.top_k * groups, blocks = (jobs + 3) / 4;
    const uint32_t grid = blocks < (1u << 20) ? (uint32_t)blocks : 1u << 20;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, a, groups, jobs);
        return launched(dual ? EIDM_KERNEL_I8_GATE_UP_ROWS : EIDM_KERNEL_I8_ROWS, grid, 256, 0);
    };
    if (a.ids && i8_read_once(a.m, a.top_k, a.n_experts, (dual ? 2ull : 1ull) * a.n * a.k))
        return dual ? go(i8_rows_kernel<C, true, true>) : go(i8_rows_kernel<C, false, true>);
    return dual ? go(i8_rows_kernel<C, true, false>) : go(i8_rows_kernel<C, false, false>);
}

// us of a call, through the caches : past them. FFN of one token: 2048 x 768, 8 of 128 (25 MB of gate and up
// weights) 13.4 : 13.9, 4096 x 1536, 8 of 256 (101 MB) 36.5 : 33.9; 4 tokens of the first (101 MB) 36.4 : 35.4;
// products of 4 tokens of 1536 x 4096, 8 of 256 (201 MB) 40.6 : 38.4; 8 rows of one weight of 4096 x 4096 14.5 : 18.5.
bool i8_read_once(uint32_t m, uint32_t top_k, uint32_t n_experts, uint64_t expert_bytes) {
    const uint64_t routed = (uint64_t)m * top_k;
    return routed <= n_experts && routed * expert_bytes >= 64000000;
}

bool i8_one_supported(const I8Args& a, int device_cus) {
    // as many blocks as route and quantise again for less than a launch takes. us, this : routing in a launch of its
    // own, 2048 x 768, 8 of 128: one token 13.8 : 17.5, 2 20.5 : 21.7, 4 36.3 : 37.3, 8 65.4 : 63.0; 256 x 96, 4 of 16: one 14.1 : 17.4.
    // Many experts are more routing a block: 512 x 128, 8 of 2048, one 19.5 : 22.9; 256 x 128, 8 tokens (1024 blocks) 8 of
    // 256 14.0 : 14.0, of 512 16.5 : 15.7, of 1024 21.2 : 18.3, of 2048 31.3 : 25.6
    const uint64_t blocks = (uint64_t)a.m * a.top_k * ((a.n + 7) / 8);
    return a.k <= kI8OneRow && blocks <= (uint64_t)device_cus * 16;
}

hipError_t launch_i8_gate_up_one(const I8OneArgs& o, hipStream_t stream) {
    const I8Args& a = o.a;
    const uint32_t blocks = (a.n + 7) / 8, grid = a.m * a.top_k * blocks, lds = (a.k + 15) / 16 * 16, nv = (a.n_experts + 63) / 64;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), lds, stream, o, blocks);
        return launched(EIDM_KERNEL_I8_GATE_UP_ONE, grid, 256, lds);
    };
    auto by_width = [&](auto flag) {
        constexpr bool ONCE = decltype(flag)::value;
        if (nv <= 1) return go(i8_gate_up_one_kernel<1, ONCE>);
        if (nv <= 2) return go(i8_gate_up_one_kernel<2, ONCE>);
        if (nv <= 4) return go(i8_gate_up_one_kernel<4, ONCE>);
        if (nv <= 8) return go(i8_gate_up_one_kernel<8, ONCE>);
        if (nv <= 16) return go(i8_gate_up_one_kernel<16, ONCE>);
        return go(i8_gate_up_one_kernel<32, ONCE>);
    };
    return i8_read_once(a.m, a.top_k, a.n_experts, 2ull * a.n * a.k) ? by_width(std::true_type{}) : by_width(std::false_type{});
}

hipError_t launch_i8_down_combine(const I8DownArgs& a, hipStream_t stream) {
    // up to 8 slots: 16 columns' loads in flight (4 : 8 : 16 columns 40.0 : 42.0 : 37.4 us for the FFN of one token of 8
    // of 256 experts of 4096 x 1536, 256 blocks of 16; not measured where fewer columns leave compute units without a
    // block); twice the wavefronts have half the registers each
    const bool few = a.top_k <= 8;
    const uint32_t cols = few ? 16 : 8, groups = (a.n + cols - 1) / cols, block = 64 * a.top_k;
    const uint64_t grid = (uint64_t)groups * a.m;
    if (grid * block >= 1ull << 32) return hipErrorInvalidValue;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(block), 0, stream, a, groups);
        return launched(EIDM_KERNEL_I8_DOWN_ROWS, (uint32_t)grid, block, 0);
    };
    // (the FFN's gate and up weights, twice as many, went before)
    if (i8_read_once(a.m, a.top_k, a.n_experts, 2ull * a.n * a.k))
        return few ? go(i8_down_combine_kernel<16, 1, 8, true>) : go(i8_down_combine_kernel<8, 1, 16, true>);
    return few ? go(i8_down_combine_kernel<16, 1, 8, false>) : go(i8_down_combine_kernel<8, 1, 16, false>);
}

}  // namespace eidm

namespace {

using namespace eidm;

struct I8Plan {
    uint64_t routed = 0, in_rows = 0, weight_bytes = 0;
    uint64_t off_counts = 0, off_offsets = 0, off_rows = 0, scratch = 0;
};

int check_i8(const eidm_i8_shape* s, I8Plan* p) {
    if (!s) return api_fail(EIDM_E_INVALID, "shape is NULL");
    if (s->struct_size != sizeof(eidm_i8_shape))
        return api_fail(EIDM_E_INVALID, "shape.struct_size is %u, expected %zu", s->struct_size, sizeof(eidm_i8_shape));
    if (s->input_layout != EIDM_LAYOUT_SHARED_PER_TOKEN && s->input_layout != EIDM_LAYOUT_SLOTTED)
        return api_fail(EIDM_E_INVALID, "unknown input layout %d", s->input_layout);
    if (!s->m || !s->n || !s->k || !s->top_k || !s->n_experts)
        return api_fail(EIDM_E_INVALID, "zero dimension (m=%u n=%u k=%u top_k=%u n_experts=%u)", s->m, s->n, s->k,
                        s->top_k, s->n_experts);
    if (s->n_experts > kMaxExperts)
        return api_fail(EIDM_E_UNSUPPORTED, "n_experts %u above the supported %u", s->n_experts, kMaxExperts);
    if (s->k > EIDM_I8_MAX_K)
        return api_fail(EIDM_E_UNSUPPORTED, "k %u above %u, where a 32-bit sum of products could overflow", s->k,
                        EIDM_I8_MAX_K);
    uint64_t body, need, routed, groups, elements;
    if (s->n > kIndex31 || !mul_fits(s->n, s->k, &body))
        return api_fail(EIDM_E_UNSUPPORTED, "n at or above 2^31");
    if (s->expert_stride_bytes < body)
        return api_fail(EIDM_E_INVALID, "expert stride %llu is shorter than one expert (%llu bytes)",
                        (unsigned long long)s->expert_stride_bytes, (unsigned long long)body);
    if (!mul_fits(s->n_experts - 1, s->expert_stride_bytes, &need) || !add_fits(need, body, &need))
        return api_fail(EIDM_E_INVALID, "required weight bytes overflow");
    if (!mul_fits(s->m, s->top_k, &routed) || routed > kIndex31)
        return api_fail(EIDM_E_UNSUPPORTED, "m*top_k at or above 2^31");
    if (!mul_fits(routed, s->n, &elements) || elements >= 1ull << 61)
        return api_fail(EIDM_E_INVALID, "output size overflows");
    // jobs of the tile form are counted in 31 bits: every expert may have a partial tile
    if (!mul_fits(routed / 16 + s->n_experts + 1, ((uint64_t)s->n + 63) / 64, &groups) || groups > kIndex31)
        return api_fail(EIDM_E_UNSUPPORTED, "%llu tiles are too many", (unsigned long long)groups);
    p->routed = routed;
    p->in_rows = s->input_layout == EIDM_LAYOUT_SLOTTED ? routed : s->m;
    p->weight_bytes = need;
    p->off_counts = round256(map_hist_elements(routed, s->n_experts) * 4);
    p->off_offsets = p->off_counts + round256((uint64_t)(s->n_experts + 1) * 4);
    p->off_rows = p->off_offsets + round256((uint64_t)(s->n_experts + 2) * 4);
    p->scratch = p->off_rows + round256(routed * 4);
    return EIDM_OK;
}

int i8_route(int route, const eidm_i8_shape* s, const I8Plan& p, bool dense, uint64_t scratch_bytes, int* chosen) {
    if (route != EIDM_ROUTE_AUTO && route != EIDM_ROUTE_DIRECT && route != EIDM_ROUTE_GROUPED)
        return api_fail(EIDM_E_INVALID, "unknown route %d", route);
    *chosen = route;
    if (route != EIDM_ROUTE_AUTO) return EIDM_OK;
    const bool alone =
        dense ? i8_dense_rows_by_themselves(s->m, s->n, s->k, s->k % 16 == 0)
              : scratch_bytes < p.scratch ||
                    i8_rows_by_themselves(s->m, s->top_k, s->n_experts, (uint64_t)s->n * s->k, i8_row_bytes(s->n, s->k));
    *chosen = alone ? EIDM_ROUTE_DIRECT : EIDM_ROUTE_GROUPED;
    return EIDM_OK;
}

MapBuffers i8_map(const I8Plan& p, void* scratch) {
    uint8_t* at = static_cast<uint8_t*>(scratch);
    return {reinterpret_cast<uint32_t*>(at), reinterpret_cast<uint32_t*>(at + p.off_counts),
            reinterpret_cast<uint32_t*>(at + p.off_offsets), reinterpret_cast<uint32_t*>(at + p.off_rows)};
}

}  // namespace

namespace eidm {

// us in a graph, rows by themselves : tiles. FFN of 2048 x 768, 8 of 128: 4
// tokens 33.5 : 43.2, 8 59.0 : 62.7, 16 106 : 87; 1024 x 512, 4 of 32: 16 tokens
// 26.4 : 31.3, 32 42.8 : 31.3; 4096 x 1536, 8 of 256: 4 tokens 115 : 130, 8 212 :
// 214, 16 404 : 320.  Products of 1536 x 4096, 8 of 256: 8 tokens 71.6 : 84.4,
// 32 257 : 221; 768 x 2048, 8 of 128: 8 tokens 17.9 : 23.5, 32 50.5 : 34.0;
// 4096 x 1024, 2 of 16: 8 tokens 13.8 : 18.2, 16 21.2 : 19.8.
// Short k (a job of four loads takes 0.4 ns of the device at 64 bytes a load, 0.48 at 512): 64
// tokens of 8 of 256, n 3400: k 64 176 : 31, 256 195 : 45, 512 208 : 73; 16 tokens, n 2048, k 64 28.8 : 16.3; 32 tokens
// of 8 of 64, n 1000, k 255 37.8 : 13.6.
uint64_t i8_row_bytes(uint32_t n, uint32_t k) { return (uint64_t)n * (k < 512 ? 512 : k); }

bool i8_rows_by_themselves(uint32_t m, uint32_t top_k, uint32_t n_experts, uint64_t expert_bytes, uint64_t row_bytes) {
    const double routed = (double)m * top_k, experts = (double)n_experts;
    const double share = top_k < n_experts ? top_k / experts : 1.0;
    const double touched = experts * (1.0 - std::pow(1.0 - share, (double)m));
    return routed * (double)row_bytes - touched * (double)expert_bytes <= 64e6;
}

// us in a graph with the quantising, rows by themselves : tiles. 4096 x 4096: 8 rows 13.3 :
// 14.7, 16 20.2 : 14.8; 4096 x 512: 4 rows 6.0 : 6.6, 8 7.9 : 6.7; 1024 x 1024: 16
// rows 6.2 : 7.8; rows that are not whole units, 500 x 3000: 16 rows 7.4 : 20.0.
// A row costs n loads of up to 1 KB of k, a tile its steps along k.
bool i8_dense_rows_by_themselves(uint32_t m, uint32_t n, uint32_t k, bool whole_units) {
    const double loads = (double)(m - 1) * n * (k < 1024 ? 1024.0 : (double)k);
    return loads <= (double)k * (whole_units ? 36e3 : 75e3);
}

int check_i8_shape(const eidm_i8_shape* shape) {
    I8Plan p;
    return check_i8(shape, &p);
}

MapBuffers i8_map_at(const eidm_i8_shape* shape, void* scratch) {
    I8Plan p;
    check_i8(shape, &p);
    return i8_map(p, scratch);
}

}  // namespace eidm

extern "C" {

uint64_t eidm_matmul_id_i8_scratch_bytes(const eidm_i8_shape* shape) {
    I8Plan p;
    if (check_i8(shape, &p) != EIDM_OK) return 0;
    api_ok();
    return p.scratch;
}

int eidm_matmul_id_i8(const eidm_i8_shape* shape, int route, const int8_t* weights, uint64_t weight_bytes,
                      const float* weight_scales, const int8_t* input, const float* input_scales, const uint32_t* ids,
                      float* output, void* scratch, uint64_t scratch_bytes, void* stream, int* route_taken) {
    ReceiptScope receipt;
    I8Plan p;
    int rc = check_i8(shape, &p), chosen = 0;
    if (rc) return rc;
    if (!weights || !weight_scales || !input || !input_scales || !output)
        return api_fail(EIDM_E_INVALID, "a buffer is NULL");
    if (weight_bytes < p.weight_bytes)
        return api_fail(EIDM_E_SIZE, "weight extent %llu below the required %llu bytes", (unsigned long long)weight_bytes,
                        (unsigned long long)p.weight_bytes);
    if (!ids && (shape->n_experts != 1 || shape->top_k != 1))
        return api_fail(EIDM_E_INVALID, "without ids there is one expert and one slot");
    if (!is_aligned(weight_scales, 4) || !is_aligned(input_scales, 4) || !is_aligned(ids, 4) || !is_aligned(output, 4))
        return api_fail(EIDM_E_ALIGN, "scales, ids and output must be 4-byte aligned");
    if ((rc = i8_route(route, shape, p, !ids, scratch ? scratch_bytes : 0, &chosen))) return rc;
    I8Args a{};
    a.m = shape->m;
    a.n = shape->n;
    a.k = shape->k;
    a.top_k = shape->top_k;
    a.n_experts = shape->n_experts;
    a.stride = shape->expert_stride_bytes;
    a.slotted = shape->input_layout == EIDM_LAYOUT_SLOTTED;
    a.w = weights;
    a.ws = weight_scales;
    a.x = input;
    a.xs = input_scales;
    a.ids = ids;
    a.out = output;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t err;
    if (chosen == EIDM_ROUTE_DIRECT) {
        err = launch_i8_rows(a, st);
    } else {
        if (ids) {
            if (!scratch || scratch_bytes < p.scratch)
                return api_fail(EIDM_E_SIZE, "Grouped route needs %llu bytes of scratch, got %llu",
                                (unsigned long long)p.scratch, (unsigned long long)(scratch ? scratch_bytes : 0));
            if (!is_aligned(scratch, 256)) return api_fail(EIDM_E_ALIGN, "scratch must be 256-byte aligned");
            const MapBuffers map = i8_map(p, scratch);
            err = launch_map(ids, (uint32_t)p.routed, shape->n_experts, map, st);
            if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "map launch: %s", hipGetErrorString(err));
            a.offsets = map.offsets;
            a.rows = map.rows;
        }
        err = launch_i8_tiles(a, device_cus(), st);
    }
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "8-bit product launch: %s", hipGetErrorString(err));
    receipt_route(chosen);
    if (route_taken) *route_taken = chosen;
    return api_ok();
}

}  // extern "C"
