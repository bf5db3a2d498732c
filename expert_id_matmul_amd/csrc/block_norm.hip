// block_norm.hip -- the norms before and after a block with its gate and
// residual scale, forward and backward.
//
//   z      = sum_s slot_gates[t, s] * y[t, s]            the block's output
//   n      = z * rstd(z) * w_post (or z),  rstd(v) = 1 / sqrt(mean(v^2) + eps)
//   out    = residual_scale * x + gate * n
//   normed = out * rstd(out) * w_pre, also in 8 bits (quant8.hpp)
//
// and for the gradients D of out, u = d_normed * w_pre (all means over a row):
//   D      = d_out + rstd(out) * (u - out * rstd(out)^2 * mean(u * out))
//   d_x    = residual_scale * D,  v = gate * D,  p = v * w_post
//   d_z    = rstd(z) * (p - z * rstd(z)^2 * mean(p * z)) (or v)
//   d_slot_gates[t, s] = sum_j d_z * y[t, s],  d_gate = D * n summed over what shares it,
//   d_w_post = sum_t v * z * rstd(z),  d_w_pre = sum_t d_normed * out * rstd(out)
//
// Bound by memory: every input is read once and every output written once; a
// row stays in registers between its reductions.  (Rows longer than a block
// holds are read again, and the slots of a row of any length for d_slot_gates,
// from the L2: 8 slots of 2048 x 2048 65 us of gradients, 42 at a copy's rate.)
// A row's values and sums are 64-bit, each output is rounded once: an 8-bit
// value next to a border would otherwise move by a whole step with the order of
// a sum, and on CDNA4 a 64-bit fma issues at the rate of an f32 one, so the
// loads still bound: 8 slots of 2048 x 2048 (155 MB) 30.9 us, 5.0 TB/s;
// gradients of 4096 x 2048 (185 MB) 39.8 and 5.2 for the column sums.
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "api_checks.hpp"
#include "eidm.h"
#include "eidm_internal.hpp"
#include "quant8.hpp"
#include "route_wave.hpp"

namespace eidm {
namespace {

// Values a thread takes at a time: 16 bytes of an f32 row, so that a wavefront's
// load is whole lines (with 8 the same kernels need over 200 registers).
constexpr int kUnit = 4;

struct NormArgs {
    uint32_t m, hidden, top_k;
    int stream_dtype, weight_dtype, gate_layout;
    double eps, residual_scale, per_value;  // per_value: 1 / hidden
    const void* x;  // forward: the stream; backward: what the pre-norm read
    const float *y, *slot_gates, *gate;
    const void *w_post, *w_pre;
    // forward
    void* out;
    float* normed;
    int8_t* q;
    float* q_scales;
    // backward
    const float *d_out, *d_normed;
    float *d_x, *d_z, *d_slot_gates, *d_gate;
    float* partial;  // [blocks][3][hidden]: column sums of d_w_pre, d_w_post, d_gate
    float* rest;     // [blocks][hidden] of the rows read twice: a row's d_z less what is stored of it
    uint32_t sums;   // which of the three are wanted (bits)
};

constexpr uint32_t kSumPre = 1, kSumPost = 2, kSumGate = 4;

// ---------------------------------------------------------------- rows of any type
// A unit of a row as it stands in memory: requested first, widened when it is
// used, so that no load waits for another.  WHOLE: k is a multiple of kUnit and
// the unit lies in the row; else what lies past k is 0.
struct Raw {
    uint32_t w[kUnit];
};

template <bool WHOLE>
__device__ __forceinline__ Raw raw_of(int dtype, const void* base, size_t row, uint32_t i, uint32_t k) {
    Raw r;
    if (dtype == kDtypeF32) {
        const float* p = static_cast<const float*>(base) + row * k;
        if (WHOLE || i + kUnit <= k) __builtin_memcpy(r.w, p + i, 4 * kUnit);
        else
#pragma unroll
            for (uint32_t j = 0; j < kUnit; ++j) r.w[j] = i + j < k ? __float_as_uint(p[i + j]) : 0;
        return r;
    }
    const uint16_t* p = static_cast<const uint16_t*>(base) + row * k;
    r.w[2] = r.w[3] = 0;
    if (WHOLE || i + kUnit <= k) {
        __builtin_memcpy(r.w, p + i, 2 * kUnit);
    } else {
        uint32_t h[kUnit];
#pragma unroll
        for (uint32_t j = 0; j < kUnit; ++j) h[j] = i + j < k ? p[i + j] : 0;
        r.w[0] = h[0] | h[1] << 16;
        r.w[1] = h[2] | h[3] << 16;
    }
    return r;
}

// A unit of f32 numbers that nothing reads again: past the caches (8 slots of
// 2048 x 2048: 48.0 -> 44.5 us with its quantising).
template <bool WHOLE>
__device__ __forceinline__ Raw raw_once(const float* row, uint32_t i, uint32_t k) {
    typedef uint32_t Quad __attribute__((ext_vector_type(4), aligned(4)));
    Raw r;
    if (WHOLE || i + kUnit <= k) {
        const Quad v = __builtin_nontemporal_load(reinterpret_cast<const Quad*>(row + i));
#pragma unroll
        for (int j = 0; j < kUnit; ++j) r.w[j] = v[j];
    } else {
#pragma unroll
        for (uint32_t j = 0; j < kUnit; ++j) r.w[j] = i + j < k ? __float_as_uint(row[i + j]) : 0;
    }
    return r;
}

__device__ __forceinline__ void widen(int dtype, const Raw& r, float (&v)[kUnit]) {
    if (dtype == kDtypeF32) {
#pragma unroll
        for (int j = 0; j < kUnit; ++j) v[j] = __uint_as_float(r.w[j]);
    } else if (dtype == kDtypeF16) {
        widen_pair<kDtypeF16>(r.w[0], v[0], v[1]);
        widen_pair<kDtypeF16>(r.w[1], v[2], v[3]);
    } else {
        widen_pair<kDtypeBF16>(r.w[0], v[0], v[1]);
        widen_pair<kDtypeBF16>(r.w[1], v[2], v[3]);
    }
}

// Where a thread of a held row takes its unit i from, WHOLE or not: a unit that
// ends past the row is loaded as the row's last kUnit values, without a branch
// about the load (3908 x 2047: 35 -> 24 us, gradients 79 -> 51), and moved into its
// place when it is used.
template <bool WHOLE>
struct Place {
    uint32_t unit, from, drop;  // drop: values of the load that belong to the unit before, kUnit or more: all
    bool past;
    __device__ Place() = default;
    __device__ __forceinline__ Place(uint32_t i, uint32_t h) {
        past = i >= h;
        unit = WHOLE && past ? 0 : i;
        from = WHOLE ? unit : min(i, h - kUnit);
        drop = unit - from;
    }
    // does this thread's unit count, and is it stored?  (without WHOLE it is zeros, and stores look for themselves)
    __device__ __forceinline__ bool live() const { return !WHOLE || !past; }
    template <typename T>
    __device__ __forceinline__ void down(T (&v)[kUnit]) const {
        if (WHOLE || !drop) return;
#pragma unroll
        for (int j = 0; j < kUnit; ++j) v[j] = drop & 1 ? (j + 1 < kUnit ? v[j + 1] : T(0)) : v[j];
#pragma unroll
        for (int j = 0; j < kUnit; ++j) v[j] = drop & 2 ? (j + 2 < kUnit ? v[j + 2] : T(0)) : v[j];
#pragma unroll
        for (int j = 0; j < kUnit; ++j) v[j] = drop >= kUnit ? T(0) : v[j];
    }
    template <typename T>
    __device__ __forceinline__ void up(T (&v)[kUnit]) const {
        if (WHOLE || !drop) return;
#pragma unroll
        for (int j = kUnit - 1; j >= 0; --j) v[j] = drop & 1 ? (j >= 1 ? v[j - 1] : T(0)) : v[j];
#pragma unroll
        for (int j = kUnit - 1; j >= 0; --j) v[j] = drop & 2 ? (j >= 2 ? v[j - 2] : T(0)) : v[j];
#pragma unroll
        for (int j = 0; j < kUnit; ++j) v[j] = drop >= kUnit ? T(0) : v[j];
    }
    __device__ __forceinline__ void widen_to(int dtype, const Raw& r, float (&v)[kUnit]) const {
        widen(dtype, r, v);
        down(v);
    }
};

__device__ __forceinline__ uint32_t bf16_bits(float f) {
    const uint32_t u = __float_as_uint(f);
    if (f != f) return u >> 16 | 0x40u;
    return (u + 0x7fffu + (u >> 16 & 1u)) >> 16;
}

// v rounded to the type, and its bits
__device__ __forceinline__ uint32_t rounded(int dtype, float& v) {
    if (dtype == kDtypeF32) return __float_as_uint(v);
    if (dtype == kDtypeF16) {
        const _Float16 h = (_Float16)v;
        v = (float)h;
        return __builtin_bit_cast(uint16_t, h);
    }
    const uint32_t b = bf16_bits(v);
    v = __uint_as_float(b << 16);
    return b;
}

template <bool WHOLE>
__device__ __forceinline__ void store_f32(float* row, uint32_t i, uint32_t k, const float (&v)[kUnit]) {
    if (WHOLE || i + kUnit <= k) {
        __builtin_memcpy(row + i, v, 4 * kUnit);
        return;
    }
#pragma unroll
    for (uint32_t j = 0; j < kUnit; ++j)
        if (i + j < k) row[i + j] = v[j];
}

// The same past the caches: a training batch's gradients, of which they would keep
// little (4096 x 4096: 76.4 -> 67.9 us, 4096 x 2048 46.1 -> 44.5).
template <bool WHOLE>
__device__ __forceinline__ void store_once(float* row, uint32_t i, uint32_t k, const float (&v)[kUnit]) {
    typedef float Quad __attribute__((ext_vector_type(4), aligned(4)));
    if (WHOLE || i + kUnit <= k) __builtin_nontemporal_store(Quad{v[0], v[1], v[2], v[3]}, reinterpret_cast<Quad*>(row + i));
    else store_f32<false>(row, i, k, v);
}

// v, rounded to the type already, of which b are the bits
template <bool WHOLE>
__device__ __forceinline__ void store_of(int dtype, void* base, size_t row, uint32_t i, uint32_t k,
                                         const float (&v)[kUnit], const uint32_t (&b)[kUnit]) {
    if (dtype == kDtypeF32) {
        store_f32<WHOLE>(static_cast<float*>(base) + row * k, i, k, v);
        return;
    }
    uint16_t* to = static_cast<uint16_t*>(base) + row * k;
    if (WHOLE || i + kUnit <= k) {
        const uint32_t p[2] = {b[0] | b[1] << 16, b[2] | b[3] << 16};
        __builtin_memcpy(to + i, p, 2 * kUnit);
        return;
    }
#pragma unroll
    for (uint32_t j = 0; j < kUnit; ++j)
        if (i + j < k) to[i + j] = (uint16_t)b[j];
}

// ---------------------------------------------------------------- sums over a row's threads
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
    const int2 p = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, int2{__builtin_amdgcn_mov_dpp(p.x, CTRL, 0xf, 0xf, false),
                                           __builtin_amdgcn_mov_dpp(p.y, CTRL, 0xf, 0xf, false)});
}

__device__ __forceinline__ double lane64(double v, int lane) {
    const int2 p = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, int2{__builtin_amdgcn_readlane(p.x, lane), __builtin_amdgcn_readlane(p.y, lane)});
}

// Sum over the wavefront, the same bits in every lane: quads, half rows and
// rows by DPP, then the four rows' sums.
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp64<0xb1>(v);
    v += dpp64<0x4e>(v);
    v += dpp64<0x141>(v);
    v += dpp64<0x140>(v);
    return (lane64(v, 0) + lane64(v, 16)) + (lane64(v, 32) + lane64(v, 48));
}

// Threads of a block that share a row: GROUP of BLOCK.  Each reduction takes the
// other of two LDS buffers, so that one barrier is enough: a thread writes a
// buffer again only after a barrier that follows every read of it.
template <int GROUP, int BLOCK>
struct RowGroup {
    static constexpr int kGroup = GROUP, kWaves = GROUP / 64, kRows = BLOCK / GROUP, kMost = 4;
    struct Shared {
        double sum[2][kRows][kWaves][kMost];
        uint32_t top[2][kRows][kWaves];
    };
    Shared& s;
    uint32_t turn = 0;
    __device__ explicit RowGroup(Shared& shared) : s(shared) {}

    template <int N>
    __device__ void sum(double (&v)[N]) {
        static_assert(N <= kMost, "as many as the buffer holds");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
        if constexpr (kWaves > 1) {
            const uint32_t g = threadIdx.x / GROUP, w = threadIdx.x % GROUP >> 6;
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int i = 0; i < N; ++i) s.sum[turn][g][w][i] = v[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                double t = s.sum[turn][g][0][i];
#pragma unroll
                for (int j = 1; j < kWaves; ++j) t += s.sum[turn][g][j][i];
                v[i] = t;
            }
            turn ^= 1;
        }
    }
    __device__ uint32_t top(uint32_t v) {
        v = wave_max_u32(v);
        if constexpr (kWaves > 1) {
            const uint32_t g = threadIdx.x / GROUP, w = threadIdx.x % GROUP >> 6;
            if ((threadIdx.x & 63) == 0) s.top[turn][g][w] = v;
            __syncthreads();
            v = s.top[turn][g][0];
#pragma unroll
            for (int j = 1; j < kWaves; ++j) v = max(v, s.top[turn][g][j]);
            turn ^= 1;
        }
        return v;
    }
};

// Q slots of a unit of the block's output z, their loads at once.  ONCE: nothing
// reads them again.
template <int Q, bool WHOLE, bool ONCE>
__device__ __forceinline__ void add_slots(const float* y, const float* g, uint32_t i, uint32_t h, double (&z)[kUnit]) {
    Raw v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if constexpr (ONCE) v[q] = raw_once<WHOLE>(y + (size_t)q * h, i, h);
        else v[q] = raw_of<WHOLE>(kDtypeF32, y, q, i, h);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < kUnit; ++j) z[j] = __builtin_fma((double)g[q], (double)__uint_as_float(v[q].w[j]), z[j]);
}

// A unit of z, MOST slots' loads at once.
template <bool WHOLE, bool ONCE = false, int MOST = 8>
__device__ __forceinline__ void slots_of(const NormArgs& a, size_t t, uint32_t i, double (&z)[kUnit]) {
    const float* y = a.y + t * a.top_k * a.hidden;
    if (!a.slot_gates) {
        float v[kUnit];
        load_row<kDtypeF32, kUnit, WHOLE>(reinterpret_cast<const uint8_t*>(y), i, a.hidden, v);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) z[j] = (double)v[j];
        return;
    }
#pragma unroll
    for (int j = 0; j < kUnit; ++j) z[j] = 0.0;
    const float* g = a.slot_gates + t * a.top_k;
    uint32_t s = 0;
    if constexpr (MOST >= 8)
        for (; s + 8 <= a.top_k; s += 8) add_slots<8, WHOLE, ONCE>(y + (size_t)s * a.hidden, g + s, i, a.hidden, z);
    for (; s + 4 <= a.top_k; s += 4) add_slots<4, WHOLE, ONCE>(y + (size_t)s * a.hidden, g + s, i, a.hidden, z);
    for (; s < a.top_k; ++s) add_slots<1, WHOLE, ONCE>(y + (size_t)s * a.hidden, g + s, i, a.hidden, z);
}

// A unit's weights of the norm after the block; ones without it.
template <bool WHOLE>
__device__ __forceinline__ Raw post_of(const NormArgs& a, uint32_t i) {
    if (a.w_post) return raw_of<WHOLE>(a.weight_dtype, a.w_post, 0, i, a.hidden);
    return {{0, 0, 0, 0}};
}
__device__ __forceinline__ void widen_post(const NormArgs& a, const Raw& r, float (&v)[kUnit]) {
    widen(a.weight_dtype, r, v);
    if (!a.w_post)
#pragma unroll
        for (int j = 0; j < kUnit; ++j) v[j] = 1.0f;
}

__device__ __forceinline__ double rstd(double squares, const NormArgs& a) {
    return rsqrt(__builtin_fma(squares, a.per_value, a.eps));
}

// The row of a thread: the same for a wavefront.
template <int GROUP>
__device__ __forceinline__ uint32_t group_of() {
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / GROUP));
}

// Rows that a block holds: GROUP threads a row, U units a thread.  Blocks stay
// and take rows in turn, with the channels' weights in 64-bit registers: a
// conversion between 32 and 64 bits takes the time of four fmas.
// WHOLE: hidden is a multiple of kUnit; threads past the row then work on its
// first unit, count nothing and store nothing.  Four wavefronts a SIMD, which
// with two units a thread takes fewer slots' loads at once and w_pre in 32 bits
// (4096 x 4096: 49.0 -> 40.2 us, 976 x 8192 26.7 -> 23.8).
template <int GROUP, int U, bool WHOLE>
__global__ __launch_bounds__(GROUP < 256 ? 256 : GROUP, 4) void block_norm_kernel(NormArgs a) {
    constexpr int BLOCK = GROUP < 256 ? 256 : GROUP;
    using Rows = RowGroup<GROUP, BLOCK>;
    __shared__ typename Rows::Shared shared;
    Rows rows(shared);
    const uint32_t at = threadIdx.x % GROUP, h = a.hidden;
    Place<WHOLE> place[U];
    double post[U][kUnit];  // w_post times a channel's gate
    std::conditional_t<(U > 1), float, double> pre[U][kUnit];  // w_pre
#pragma unroll
    for (int u = 0; u < U; ++u) {
        place[u] = Place<WHOLE>((u * GROUP + at) * kUnit, h);
        float w[kUnit], g[kUnit], n[kUnit];
        Raw none{}, raw = a.w_post ? raw_of<true>(a.weight_dtype, a.w_post, 0, place[u].from, h) : none;
        Raw gate = a.gate_layout == EIDM_GATE_CHANNEL ? raw_of<true>(kDtypeF32, a.gate, 0, place[u].from, h) : none;
        Raw next = a.w_pre ? raw_of<true>(a.weight_dtype, a.w_pre, 0, place[u].from, h) : none;
        place[u].widen_to(a.weight_dtype, raw, w);
        place[u].widen_to(kDtypeF32, gate, g);
        place[u].widen_to(a.weight_dtype, next, n);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) {
            post[u][j] = (a.w_post ? (double)w[j] : 1.0) * (a.gate_layout == EIDM_GATE_CHANNEL ? (double)g[j] : 1.0);
            pre[u][j] = n[j];
        }
    }
    // the next row is requested while this one is worked on (of many slots the stream alone)
    const uint64_t stride = (uint64_t)gridDim.x * Rows::kRows;
    Raw x_next[U], y_next[U];
    auto request = [&](uint64_t t) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x_next[u] = raw_of<true>(a.stream_dtype, a.x, t, place[u].from, h);
            if (a.y && !a.slot_gates) y_next[u] = raw_once<true>(a.y + t * h, place[u].from, h);
        }
    };
    uint64_t t = (uint64_t)blockIdx.x * Rows::kRows + group_of<GROUP>();
    if (t < a.m) request(t);
    for (; t < a.m; t += stride) {  // (a block of one row at a time: the same for all threads; else a wavefront's)
        Raw x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = x_next[u];
            y[u] = y_next[u];
        }
        float o[U][kUnit];
        double total[1] = {0.0};
        if (a.y) {
            double z[U][kUnit];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (a.slot_gates) slots_of<true, true, (U > 1) ? 4 : 8>(a, t, place[u].from, z[u]);
                else
#pragma unroll
                    for (int j = 0; j < kUnit; ++j) z[u][j] = (double)__uint_as_float(y[u].w[j]);
                place[u].down(z[u]);
            }
            if (t + stride < a.m) request(t + stride);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                double s = 0.0;
#pragma unroll
                for (int j = 0; j < kUnit; ++j) s = __builtin_fma(z[u][j], z[u][j], s);
                total[0] += place[u].live() ? s : 0.0;
            }
            double scale = a.gate_layout == EIDM_GATE_TOKEN ? (double)a.gate[t] : 1.0;
            if (a.w_post) {
                rows.sum(total);
                scale *= rstd(total[0], a);
            }
            total[0] = 0.0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                place[u].widen_to(a.stream_dtype, x[u], o[u]);
                uint32_t bits[kUnit];
#pragma unroll
                for (int j = 0; j < kUnit; ++j) {
                    o[u][j] = (float)__builtin_fma(a.residual_scale, (double)o[u][j], z[u][j] * scale * post[u][j]);
                    bits[j] = rounded(a.stream_dtype, o[u][j]);
                }
                if (place[u].live()) store_of<WHOLE>(a.stream_dtype, a.out, t, place[u].unit, h, o[u], bits);
            }
            if (!a.w_pre) continue;
        } else {
            if (t + stride < a.m) request(t + stride);
#pragma unroll
            for (int u = 0; u < U; ++u) place[u].widen_to(a.stream_dtype, x[u], o[u]);
        }
        double r[U][kUnit];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                r[u][j] = (double)o[u][j];
                s = __builtin_fma(r[u][j], r[u][j], s);
            }
            total[0] += place[u].live() ? s : 0.0;
        }
        rows.sum(total);
        const double inv = rstd(total[0], a);
        uint32_t top = 0;
        float n[U][kUnit];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                n[u][j] = (float)(r[u][j] * inv * (double)pre[u][j]);
                top = max(top, place[u].live() ? magnitude(n[u][j]) : 0u);
            }
            if (a.normed && (place[u].live())) store_f32<WHOLE>(a.normed + t * h, place[u].unit, h, n[u]);
        }
        if (!a.q) continue;
        const RowScale s = row_scale(rows.top(top));
        if (at == 0) a.q_scales[t] = s.scale;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (place[u].live()) store_q<kUnit, WHOLE>(a.q + t * h, place[u].unit, h, n[u], s);
    }
}

// Longer rows: any number of units a thread, read again in each pass (the
// stream from `out`, where a thread finds what it wrote).
constexpr int kLongBlock = 1024;

__global__ __launch_bounds__(kLongBlock) void block_norm_long_kernel(NormArgs a) {
    constexpr bool WHOLE = false;
    using Rows = RowGroup<kLongBlock, kLongBlock>;
    __shared__ typename Rows::Shared shared;
    Rows rows(shared);
    const uint32_t h = a.hidden, step = kLongBlock * kUnit, first = threadIdx.x * kUnit;
    const void* held = a.y ? a.out : a.x;
    for (uint64_t t = blockIdx.x; t < a.m; t += gridDim.x) {
        double z[kUnit], total[1] = {0.0}, scale = a.gate_layout == EIDM_GATE_TOKEN ? (double)a.gate[t] : 1.0;
        float o[kUnit], w[kUnit], g[kUnit];
        if (a.w_post) {
            for (uint32_t i = first; i < h; i += step) {
                slots_of<WHOLE, false, 4>(a, t, i, z);
#pragma unroll
                for (int j = 0; j < kUnit; ++j) total[0] = __builtin_fma(z[j], z[j], total[0]);
            }
            rows.sum(total);
            scale *= rstd(total[0], a);
        }
        total[0] = 0.0;
        for (uint32_t i = first; i < h; i += step) {
            widen(a.stream_dtype, raw_of<WHOLE>(a.stream_dtype, a.x, t, i, h), o);
            if (a.y) {
                slots_of<WHOLE, false, 4>(a, t, i, z);
                widen_post(a, post_of<WHOLE>(a, i), w);
                const bool channel = a.gate_layout == EIDM_GATE_CHANNEL;
                if (channel) widen(kDtypeF32, raw_of<WHOLE>(kDtypeF32, a.gate, 0, i, h), g);
                uint32_t bits[kUnit];
#pragma unroll
                for (int j = 0; j < kUnit; ++j) {
                    const double p = (double)w[j] * (channel ? (double)g[j] : 1.0);
                    o[j] = (float)__builtin_fma(a.residual_scale, (double)o[j], z[j] * scale * p);
                    bits[j] = rounded(a.stream_dtype, o[j]);
                }
                store_of<WHOLE>(a.stream_dtype, a.out, t, i, h, o, bits);
            }
#pragma unroll
            for (int j = 0; j < kUnit; ++j) total[0] = __builtin_fma((double)o[j], (double)o[j], total[0]);
        }
        if (!a.w_pre) continue;
        rows.sum(total);
        const double inv = rstd(total[0], a);
        float n[kUnit];
        auto norm = [&](uint32_t i) {
            widen(a.stream_dtype, raw_of<WHOLE>(a.stream_dtype, held, t, i, h), o);
            widen(a.weight_dtype, raw_of<WHOLE>(a.weight_dtype, a.w_pre, 0, i, h), w);
#pragma unroll
            for (int j = 0; j < kUnit; ++j) n[j] = (float)((double)o[j] * inv * (double)w[j]);
        };
        uint32_t top = 0;
        for (uint32_t i = first; i < h; i += step) {
            norm(i);
#pragma unroll
            for (int j = 0; j < kUnit; ++j) top = max(top, magnitude(n[j]));
            if (a.normed) store_f32<WHOLE>(a.normed + t * h, i, h, n);
        }
        if (!a.q) continue;
        const RowScale s = row_scale(rows.top(top));
        if (threadIdx.x == 0) a.q_scales[t] = s.scale;
        for (uint32_t i = first; i < h; i += step) {
            norm(i);
            store_q<kUnit, WHOLE>(a.q + t * h, i, h, n, s);
        }
    }
}

// ---------------------------------------------------------------- backward
// d_slot_gates of a row, four slots a reduction; y's row comes from the L2 once
// more.  part(s, dot): adds a thread's share of slots s .. s+3 to dot.
template <typename Rows>
__device__ __forceinline__ void slot_sums(const NormArgs& a, Rows& rows, size_t t, bool live, uint32_t s0, double (&dot)[4]) {
    rows.sum(dot);
#pragma unroll
    for (uint32_t s = 0; s < 4; ++s)
        if (live && threadIdx.x % Rows::kGroup == 0 && s0 + s < a.top_k) a.d_slot_gates[t * a.top_k + s0 + s] = (float)dot[s];
}

template <typename Rows, typename PartOf>
__device__ __forceinline__ void slot_gradients(const NormArgs& a, Rows& rows, size_t t, bool live, uint32_t first, PartOf part) {
    for (uint32_t s0 = first; s0 < a.top_k; s0 += 4) {
        double dot[4] = {0.0, 0.0, 0.0, 0.0};
        part(s0, dot);
        slot_sums(a, rows, t, live, s0, dot);
    }
}

template <bool WHOLE>
__device__ __forceinline__ void slot_products(const NormArgs& a, size_t t, uint32_t i, uint32_t s0, const double (&dz)[kUnit],
                                              double (&dot)[4]) {
    float v[4][kUnit];
#pragma unroll
    for (uint32_t s = 0; s < 4; ++s)
        load_row<kDtypeF32, kUnit, WHOLE>(
            reinterpret_cast<const uint8_t*>(a.y + (t * a.top_k + min(s0 + s, a.top_k - 1)) * a.hidden), i, a.hidden, v[s]);
#pragma unroll
    for (uint32_t s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < kUnit; ++j) dot[s] = __builtin_fma(dz[j], (double)v[s][j], dot[s]);
}

// Rows that a block holds, as in the forward kernel; a thread's columns' sums
// over its block's rows stay in 64-bit registers.  BLOCK / GROUP rows at a time:
// every thread takes part in the reductions' barriers, rows past the last count
// nothing and store nothing.
template <int GROUP, int BLOCK, int U, bool WHOLE>
__global__ __launch_bounds__(BLOCK) void block_norm_backward_kernel(NormArgs a) {
    using Rows = RowGroup<GROUP, BLOCK>;
    __shared__ typename Rows::Shared shared;
    Rows rows(shared);
    const uint32_t at = threadIdx.x % GROUP, h = a.hidden;
    Place<WHOLE> place[U];
    double pre[U][kUnit], through[U][kUnit];  // w_pre; w_post times a channel's gate
    // sums over rows: d_normed * r * rstd(r), and gate of the token * D * z * rstd(z), of which d_w_post is the
    // channel's gate times as much, and a channel's d_gate w_post times as much
    double s_pre[U][kUnit] = {}, s_post[U][kUnit] = {};
    const bool by_channel = a.gate_layout == EIDM_GATE_CHANNEL;
    auto weights = [&](int u, double (&w)[kUnit], double (&g)[kUnit]) {
        float v[kUnit];
        const Raw none{};
        place[u].widen_to(a.weight_dtype, a.w_post ? raw_of<true>(a.weight_dtype, a.w_post, 0, place[u].from, h) : none, v);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) w[j] = a.w_post ? (double)v[j] : 1.0;
        place[u].widen_to(kDtypeF32, by_channel ? raw_of<true>(kDtypeF32, a.gate, 0, place[u].from, h) : none, v);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) g[j] = by_channel ? (double)v[j] : 1.0;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
        place[u] = Place<WHOLE>((u * GROUP + at) * kUnit, h);
        float n[kUnit];
        double w[kUnit], g[kUnit];
        const Raw none{};
        place[u].widen_to(a.weight_dtype, a.w_pre ? raw_of<true>(a.weight_dtype, a.w_pre, 0, place[u].from, h) : none, n);
        weights(u, w, g);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) {
            pre[u][j] = (double)n[j];
            through[u][j] = w[j] * g[j];
        }
    }
    // the next row is requested while this one is worked on (of many slots all but y)
    Raw dn_next[U], r_next[U], d_next[U], y_next[U];
    auto request = [&](uint64_t t) {
        const Raw none{};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            dn_next[u] = a.w_pre ? raw_once<true>(a.d_normed + t * h, place[u].from, h) : none;
            r_next[u] = a.w_pre ? raw_of<true>(a.stream_dtype, a.x, t, place[u].from, h) : none;
            d_next[u] = a.d_out ? raw_once<true>(a.d_out + t * h, place[u].from, h) : none;
            y_next[u] = a.y && !a.slot_gates ? raw_once<true>(a.y + t * h, place[u].from, h) : none;
        }
    };
    const uint64_t stride = (uint64_t)gridDim.x * Rows::kRows;
    auto row_of = [&](uint64_t t0) { return min(t0 + group_of<GROUP>(), (uint64_t)a.m - 1); };
    request(row_of((uint64_t)blockIdx.x * Rows::kRows));
    for (uint64_t t0 = (uint64_t)blockIdx.x * Rows::kRows; t0 < a.m; t0 += stride) {
        const uint64_t t = row_of(t0);
        const bool live = t0 + group_of<GROUP>() < a.m;
        Raw dn_raw[U], r_raw[U], d_raw[U];
        double z[U][kUnit], r[U][kUnit], q[U][kUnit];  // q: d_normed
        double sums[3] = {0.0, 0.0, 0.0};                   // r^2, d_normed * w_pre * r, z^2
#pragma unroll
        for (int u = 0; u < U; ++u) {
            dn_raw[u] = dn_next[u];
            r_raw[u] = r_next[u];
            d_raw[u] = d_next[u];
            if (a.slot_gates) slots_of<true>(a, t, place[u].from, z[u]);
            else
#pragma unroll
                for (int j = 0; j < kUnit; ++j) z[u][j] = (double)__uint_as_float(y_next[u].w[j]);
            place[u].down(z[u]);
        }
        if (t0 + stride < a.m) request(row_of(t0 + stride));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[kUnit], n[kUnit];
            place[u].widen_to(a.stream_dtype, r_raw[u], v);
            place[u].widen_to(kDtypeF32, dn_raw[u], n);
            double s0 = 0.0, s1 = 0.0, s2 = 0.0;
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                r[u][j] = (double)v[j];
                q[u][j] = (double)n[j];
                s0 = __builtin_fma(r[u][j], r[u][j], s0);
                s1 = __builtin_fma(q[u][j] * pre[u][j], r[u][j], s1);
                s2 = __builtin_fma(z[u][j], z[u][j], s2);
            }
            if (place[u].live()) {
                sums[0] += s0;
                sums[1] += s1;
                sums[2] += s2;
            }
        }
        rows.sum(sums);
        const double inv_r = rstd(sums[0], a), back = inv_r * inv_r * inv_r * (sums[1] * a.per_value);
        // the gradient of the stream after the block
        double d[U][kUnit];
        const double scale = a.y ? a.residual_scale : 1.0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool counts = live && place[u].live();
            float v[kUnit];
            place[u].widen_to(kDtypeF32, d_raw[u], v);
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                d[u][j] = (double)v[j];
                if (a.w_pre) {
                    d[u][j] = __builtin_fma(q[u][j] * pre[u][j], inv_r, __builtin_fma(-r[u][j], back, d[u][j]));
                    if (counts) s_pre[u][j] = __builtin_fma(q[u][j] * r[u][j], inv_r, s_pre[u][j]);
                }
                v[j] = (float)(scale * d[u][j]);
            }
            if (counts) store_once<WHOLE>(a.d_x + t * h, place[u].unit, h, v);
        }
        if (!a.y) continue;
        const double token = a.gate_layout == EIDM_GATE_TOKEN ? (double)a.gate[t] : 1.0;
        const double inv_z = a.w_post ? rstd(sums[2], a) : 1.0, gated = token * inv_z;
        double cross[1] = {0.0};  // channel's gate * D * w_post * z
#pragma unroll
        for (int u = 0; u < U; ++u) {
            double c = 0.0;
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                if (live && place[u].live()) s_post[u][j] = __builtin_fma(d[u][j] * z[u][j], gated, s_post[u][j]);
                d[u][j] *= through[u][j];
                c = __builtin_fma(d[u][j], z[u][j], c);
            }
            cross[0] += place[u].live() ? c : 0.0;
        }
        rows.sum(cross);
        if (live && at == 0 && a.gate_layout == EIDM_GATE_TOKEN && a.d_gate) a.d_gate[t] = (float)(cross[0] * inv_z);
        const double back_z = a.w_post ? gated * inv_z * inv_z * (cross[0] * a.per_value) : 0.0;
        double dz[U][kUnit];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[kUnit];
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                dz[u][j] = __builtin_fma(d[u][j], gated, -(z[u][j] * back_z));
                v[j] = (float)dz[u][j];
                if (!place[u].live()) dz[u][j] = 0.0;
            }
            if (live && place[u].live()) store_once<WHOLE>(a.d_z + t * h, place[u].unit, h, v);
            place[u].up(dz[u]);
        }
        if (a.d_slot_gates)
            slot_gradients(a, rows, t, live, 0, [&](uint32_t s0, double(&dot)[4]) {
#pragma unroll
                for (int u = 0; u < U; ++u) slot_products<true>(a, t, place[u].from, s0, dz[u], dot);
            });
    }
    // the row groups of a block share columns: added in the groups' order
    float* mine = a.partial + (size_t)blockIdx.x * 3 * h;
    __shared__ float columns[GROUP < BLOCK ? BLOCK * kUnit : 1];
    auto put = [&](int u, uint32_t which, const double (&sum)[kUnit], const double (&times)[kUnit]) {
        float v[kUnit];
#pragma unroll
        for (int j = 0; j < kUnit; ++j) v[j] = (float)(sum[j] * times[j]);
        if constexpr (Rows::kRows > 1) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kUnit; ++j) columns[threadIdx.x * kUnit + j] = v[j];
            __syncthreads();
            const uint32_t from = u * GROUP * kUnit;
            for (uint32_t c = threadIdx.x; c < GROUP * kUnit && from + c < h; c += BLOCK) {
                float total = 0.0f;
                for (uint32_t g = 0; g < Rows::kRows; ++g) total += columns[g * GROUP * kUnit + c];
                mine[which * h + from + c] = total;
            }
        } else if (place[u].live()) {
            store_f32<WHOLE>(mine + which * h, place[u].unit, h, v);
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
        double w[kUnit], g[kUnit];
        const double ones[kUnit] = {1.0, 1.0, 1.0, 1.0};
        if (a.sums & (kSumPost | kSumGate)) weights(u, w, g);
        if (a.sums & kSumPre) put(u, 0, s_pre[u], ones);
        if (a.sums & kSumPost) put(u, 1, s_post[u], g);
        if (a.sums & kSumGate) put(u, 2, s_post[u], w);
    }
}

// Longer rows, read twice: the sums first, with those of D * w_post * z taken
// apart into sums that need no D (2000 x 8192 with a pass of its own for them
// 235 -> 200 us); the columns' sums are kept in LDS (IN_LDS: 200 -> 166 us) or in
// the block's partial rows, each column by one thread.  SLOTS: d_slot_gates, the
// first four of them in the second pass (without them 166 -> 152 us).
template <bool IN_LDS, bool SLOTS>
__global__ __launch_bounds__(kLongBlock) void block_norm_backward_long_kernel(NormArgs a) {
    constexpr bool WHOLE = false;
    using Rows = RowGroup<kLongBlock, kLongBlock>;
    __shared__ typename Rows::Shared shared;
    Rows rows(shared);
    const uint32_t h = a.hidden, step = kLongBlock * kUnit, first = threadIdx.x * kUnit;
    extern __shared__ float4 lds_sums[];  // [3][units of a row]
    const uint32_t units = (h + kUnit - 1) / kUnit;
    float *mine = a.partial + (size_t)blockIdx.x * 3 * h, *rest = a.rest + (size_t)blockIdx.x * h;
    const float zeros[kUnit] = {};
    for (uint32_t i = first; i < h; i += step)
        for (uint32_t which = 0; which < 3; ++which) {
            if (IN_LDS) lds_sums[which * units + i / kUnit] = float4{0.0f, 0.0f, 0.0f, 0.0f};
            else store_f32<WHOLE>(mine + which * h, i, h, zeros);
        }
    for (uint64_t t = blockIdx.x; t < a.m; t += gridDim.x) {
        float r[kUnit] = {}, dn[kUnit] = {}, wn[kUnit] = {}, wp[kUnit], g[kUnit], v[kUnit];
        double z[kUnit] = {};
        const double token = a.gate_layout == EIDM_GATE_TOKEN ? (double)a.gate[t] : 1.0;
        auto read = [&](uint32_t i) {
            const Raw none{};
            widen(kDtypeF32, a.d_out ? raw_of<WHOLE>(kDtypeF32, a.d_out, t, i, h) : none, v);
            if (a.w_pre) {
                widen(a.stream_dtype, raw_of<WHOLE>(a.stream_dtype, a.x, t, i, h), r);
                widen(kDtypeF32, raw_of<WHOLE>(kDtypeF32, a.d_normed, t, i, h), dn);
                widen(a.weight_dtype, raw_of<WHOLE>(a.weight_dtype, a.w_pre, 0, i, h), wn);
            }
            if (!a.y) return;
            slots_of<WHOLE, false, 4>(a, t, i, z);
            widen_post(a, post_of<WHOLE>(a, i), wp);
#pragma unroll
            for (int j = 0; j < kUnit; ++j) g[j] = 1.0f;
            if (a.gate_layout == EIDM_GATE_CHANNEL) widen(kDtypeF32, raw_of<WHOLE>(kDtypeF32, a.gate, 0, i, h), g);
        };
        // r^2, d_normed * w_pre * r, z^2; and with p = channel's gate * w_post * z: d_out * p, d_normed * w_pre * p, r * p
        double sums[3] = {0.0, 0.0, 0.0}, parts[3] = {0.0, 0.0, 0.0};
        for (uint32_t i = first; i < h; i += step) {
            read(i);
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                const double u = (double)dn[j] * (double)wn[j];
                sums[0] = __builtin_fma((double)r[j], (double)r[j], sums[0]);
                sums[1] = __builtin_fma(u, (double)r[j], sums[1]);
                if (!a.y) continue;
                const double p = (double)g[j] * (double)wp[j] * z[j];
                sums[2] = __builtin_fma(z[j], z[j], sums[2]);
                parts[0] = __builtin_fma((double)v[j], p, parts[0]);
                parts[1] = __builtin_fma(u, p, parts[1]);
                parts[2] = __builtin_fma((double)r[j], p, parts[2]);
            }
        }
        rows.sum(sums);
        const double inv_r = a.w_pre ? rstd(sums[0], a) : 0.0, back = inv_r * inv_r * (sums[1] * a.per_value);
        const double inv_z = a.w_post ? rstd(sums[2], a) : 1.0;
        double cross = 0.0;  // D * p
        if (a.y) {
            rows.sum(parts);
            cross = __builtin_fma(inv_r, parts[1] - back * parts[2], parts[0]);
            if (threadIdx.x == 0 && a.gate_layout == EIDM_GATE_TOKEN && a.d_gate) a.d_gate[t] = (float)(cross * inv_z);
        }
        const double back_z = a.w_post ? token * inv_z * inv_z * (cross * a.per_value) : 0.0;
        const double scale = a.y ? a.residual_scale : 1.0;
        auto add = [&](uint32_t wanted, uint32_t which, uint32_t i, const double (&by)[kUnit]) {
            if (!(a.sums & wanted)) return;
            if constexpr (IN_LDS) {
                float4& s = lds_sums[which * units + i / kUnit];
                s = float4{s.x + (float)by[0], s.y + (float)by[1], s.z + (float)by[2], s.w + (float)by[3]};
                return;
            }
            float* to = mine + which * h;
            float now[kUnit];
            widen(kDtypeF32, raw_of<WHOLE>(kDtypeF32, to, 0, i, h), now);
#pragma unroll
            for (int j = 0; j < kUnit; ++j) now[j] += (float)by[j];
            store_f32<WHOLE>(to, i, h, now);
        };
        double dots[4] = {0.0, 0.0, 0.0, 0.0};  // of the first four slots
        for (uint32_t i = first; i < h; i += step) {
            read(i);
            double d[kUnit], by[kUnit];
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                d[j] = __builtin_fma(inv_r, (double)dn[j] * (double)wn[j] - (double)r[j] * back, (double)v[j]);
                by[j] = (double)dn[j] * (double)r[j] * inv_r;
                v[j] = (float)(scale * d[j]);
            }
            store_f32<WHOLE>(a.d_x + t * h, i, h, v);
            add(kSumPre, 0, i, by);
            if (!a.y) continue;
            double by_gate[kUnit], dz[kUnit];
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                const double e = token * (double)g[j] * d[j];
                dz[j] = inv_z * (e * (double)wp[j] - z[j] * back_z);
                v[j] = (float)dz[j];
                by[j] = e * z[j] * inv_z;
                by_gate[j] = d[j] * (double)wp[j] * z[j] * inv_z;
            }
            store_f32<WHOLE>(a.d_z + t * h, i, h, v);
            if constexpr (SLOTS) {
                slot_products<WHOLE>(a, t, i, 0, dz, dots);
                if (a.top_k > 4) {
#pragma unroll
                    for (int j = 0; j < kUnit; ++j) v[j] = (float)(dz[j] - (double)v[j]);
                    store_f32<WHOLE>(rest, i, h, v);
                }
            }
            add(kSumPost, 1, i, by);
            add(kSumGate, 2, i, by_gate);
        }
        if constexpr (SLOTS) {
            slot_sums(a, rows, t, true, 0, dots);
            // further ones from d_z as it was stored and what that left of it, zeros past the row: of a d_z rounded to f32
            // alone, the products with a slot that the norm scales out again cancel but for eps, and leave its rounding
            slot_gradients(a, rows, t, true, 4, [&](uint32_t s0, double(&dot)[4]) {
                for (uint32_t i = first; i < h; i += step) {
                    float less[kUnit];
                    widen(kDtypeF32, raw_of<WHOLE>(kDtypeF32, a.d_z, t, i, h), v);
                    widen(kDtypeF32, raw_of<WHOLE>(kDtypeF32, rest, 0, i, h), less);
                    double dz[kUnit];
#pragma unroll
                    for (int j = 0; j < kUnit; ++j) dz[j] = (double)v[j] + (double)less[j];
                    slot_products<WHOLE>(a, t, i, s0, dz, dot);
                }
            });
        }
    }
    if constexpr (IN_LDS)
        for (uint32_t i = first; i < h; i += step)
            for (uint32_t which = 0; which < 3; ++which) {
                const float4 v = lds_sums[which * units + i / kUnit];
                const float sum[kUnit] = {v.x, v.y, v.z, v.w};
                store_f32<WHOLE>(mine + which * h, i, h, sum);
            }
}

// The blocks' column sums, added in their order (64 bits).
__global__ __launch_bounds__(256) void column_sums_kernel(const float* __restrict__ partial, uint32_t blocks, uint32_t h,
                                                          float* __restrict__ d_w_pre, float* __restrict__ d_w_post,
                                                          float* __restrict__ d_gate) {
    __shared__ double part[4][64];
    float* to[3] = {d_w_pre, d_w_post, d_gate};
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    float* out = to[blockIdx.y];
    if (!out) return;  // block-uniform
    double v = 0.0;
    if (c < h)
#pragma unroll 8
        for (uint32_t b = wave; b < blocks; b += 4) v += (double)partial[((size_t)b * 3 + blockIdx.y) * h + c];
    part[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < h) out[c] = (float)((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]));
}

int check_norm(const eidm_norm_shape* s) {
    if (!s) return api_fail(EIDM_E_INVALID, "shape is NULL");
    if (s->struct_size != sizeof(eidm_norm_shape))
        return api_fail(EIDM_E_INVALID, "shape.struct_size is %u, expected %zu", s->struct_size, sizeof(eidm_norm_shape));
    if (!scalar_bytes(s->stream_dtype) || !scalar_bytes(s->weight_dtype))
        return api_fail(EIDM_E_INVALID, "unknown dtype (stream %d, weights %d)", s->stream_dtype, s->weight_dtype);
    if (s->gate_layout < EIDM_GATE_NONE || s->gate_layout > EIDM_GATE_CHANNEL)
        return api_fail(EIDM_E_INVALID, "unknown gate layout %d", s->gate_layout);
    if (!s->m || !s->hidden || !s->top_k)
        return api_fail(EIDM_E_INVALID, "zero dimension (m=%u hidden=%u top_k=%u)", s->m, s->hidden, s->top_k);
    if (!(s->eps > 0.0f) || !std::isfinite(s->eps) || !std::isfinite(s->residual_scale))
        return api_fail(EIDM_E_INVALID, "eps must be positive and finite, the residual scale finite");
    uint64_t routed;
    if (!mul_fits(s->m, s->top_k, &routed) || routed > kIndex31 || s->hidden > EIDM_I8_MAX_K || s->top_k > kMaxRouterTopK)
        return api_fail(EIDM_E_UNSUPPORTED, "m*top_k below 2^31, hidden <= %u and top_k <= %u are taken", EIDM_I8_MAX_K,
                        kMaxRouterTopK);
    return EIDM_OK;
}

// y null: no block, and the gate layout has no effect
NormArgs norm_args(const eidm_norm_shape* s, const float* y) {
    NormArgs a{};
    a.m = s->m;
    a.hidden = s->hidden;
    a.top_k = s->top_k;
    a.stream_dtype = s->stream_dtype;
    a.weight_dtype = s->weight_dtype;
    a.y = y;
    a.gate_layout = y ? s->gate_layout : EIDM_GATE_NONE;
    a.eps = (double)s->eps;
    a.per_value = 1.0 / (double)s->hidden;
    a.residual_scale = (double)s->residual_scale;
    return a;
}

int check_block(const eidm_norm_shape* s, const void* y, const void* slot_gates, const void* w_post, const void* gate) {
    if (!y && (slot_gates || w_post || gate))
        return api_fail(EIDM_E_INVALID, "without y there are no slot gates, no norm after the block and no gate");
    if (y && !slot_gates && s->top_k != 1) return api_fail(EIDM_E_INVALID, "top_k slots need their gates");
    if (y && (gate != nullptr) != (s->gate_layout != EIDM_GATE_NONE))
        return api_fail(EIDM_E_INVALID, "a gate is given exactly with a gate layout");
    return EIDM_OK;
}

constexpr int kBackBlock = 512;  // threads of a backward block, 1024 for rows of more than 4096 values

uint32_t back_rows(uint32_t hidden) { return hidden <= 512 ? kBackBlock / 64 : hidden <= 1024 ? kBackBlock / 256 : 1; }

constexpr uint32_t kLongLds = 144 * 1024;  // for the columns' sums of longer rows, beside the reductions' buffers

// Blocks that stay, one a compute unit: more would write as many more partial
// rows of the columns' sums.
constexpr uint32_t kBackBlocks = 256;

uint32_t back_blocks(const eidm_norm_shape* s) {
    const uint32_t rows = back_rows(s->hidden), need = (s->m + rows - 1) / rows;
    return need < kBackBlocks ? need : kBackBlocks;
}

// Rows that no block holds, which are read twice.
bool back_long(uint32_t hidden) { return hidden < kUnit || hidden > 4096; }

// Scratch: the blocks' column sums, then the rests of the rows that are read twice.
uint64_t back_sums_bytes(const eidm_norm_shape* s) { return round256((uint64_t)back_blocks(s) * 3 * s->hidden * 4); }
uint64_t back_scratch_bytes(const eidm_norm_shape* s) {
    return back_sums_bytes(s) + (back_long(s->hidden) ? round256((uint64_t)back_blocks(s) * s->hidden * 4) : 0);
}

}  // namespace
}  // namespace eidm

extern "C" {

using namespace eidm;

int eidm_block_norm(const eidm_norm_shape* shape, const void* x, const float* y, const float* slot_gates,
                    const void* w_post, const float* gate, void* out, const void* w_pre, float* normed, int8_t* q,
                    float* q_scales, void* stream) {
    ReceiptScope receipt;
    int rc = check_norm(shape);
    if (rc) return rc;
    if (!x) return api_fail(EIDM_E_INVALID, "x is NULL");
    if ((rc = check_block(shape, y, slot_gates, w_post, gate))) return rc;
    if ((y != nullptr) != (out != nullptr)) return api_fail(EIDM_E_INVALID, "out is given exactly with y");
    if (!y && !w_pre) return api_fail(EIDM_E_INVALID, "neither a block's output nor a norm is given");
    if ((q != nullptr) != (q_scales != nullptr)) return api_fail(EIDM_E_INVALID, "q and q_scales go together");
    if ((w_pre != nullptr) != (normed || q)) return api_fail(EIDM_E_INVALID, "normed or q is given exactly with w_pre");
    const uint32_t ss = scalar_bytes(shape->stream_dtype), sw = scalar_bytes(shape->weight_dtype);
    if (!is_aligned(x, ss) || !is_aligned(out, ss) || !is_aligned(w_post, sw) || !is_aligned(w_pre, sw) ||
        !is_aligned(y, 4) || !is_aligned(slot_gates, 4) || !is_aligned(gate, 4) || !is_aligned(normed, 4) ||
        !is_aligned(q_scales, 4))
        return api_fail(EIDM_E_ALIGN, "buffers must be aligned to their scalars");
    NormArgs a = norm_args(shape, y);
    a.x = x;
    a.slot_gates = slot_gates;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.out = out;
    a.normed = normed;
    a.q = q;
    a.q_scales = q_scales;
    const uint32_t h = a.hidden;
    auto go = [&](auto kernel, uint32_t block, uint32_t rows) {
        const uint32_t need = (a.m + rows - 1) / rows, most = (uint32_t)device_cus() * (1024 / block);
        const uint32_t grid = need < most ? need : most;
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(block), 0, static_cast<hipStream_t>(stream), a);
        return launched(EIDM_KERNEL_BLOCK_NORM, grid, block, 0);
    };
    auto by_length = [&](auto whole) {
        constexpr bool W = decltype(whole)::value;
        if (h < kUnit) return go(block_norm_long_kernel, kLongBlock, 1);
        if (h <= 256) return go(block_norm_kernel<64, 1, W>, 256, 4);
        if (h <= 512) return go(block_norm_kernel<64, 2, W>, 256, 4);
        if (h <= 1024) return go(block_norm_kernel<256, 1, W>, 256, 1);
        if (h <= 2048) return go(block_norm_kernel<512, 1, W>, 512, 1);
        if (h <= 4096) return go(block_norm_kernel<512, 2, W>, 512, 1);
        if (h <= 8192) return go(block_norm_kernel<1024, 2, W>, 1024, 1);
        return go(block_norm_long_kernel, kLongBlock, 1);
    };
    const hipError_t err = h % kUnit == 0 ? by_length(std::true_type{}) : by_length(std::false_type{});
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "norm launch: %s", hipGetErrorString(err));
    return api_ok();
}

uint64_t eidm_block_norm_backward_scratch_bytes(const eidm_norm_shape* shape) {
    if (check_norm(shape) != EIDM_OK) return 0;
    api_ok();
    return back_scratch_bytes(shape);
}

int eidm_block_norm_backward(const eidm_norm_shape* shape, const void* stream_rows, const float* y,
                             const float* slot_gates, const void* w_post, const float* gate, const void* w_pre,
                             const float* d_out, const float* d_normed, float* d_x, float* d_z, float* d_slot_gates,
                             float* d_gate, float* d_w_post, float* d_w_pre, void* scratch, uint64_t scratch_bytes,
                             void* stream) {
    ReceiptScope receipt;
    int rc = check_norm(shape);
    if (rc) return rc;
    if ((rc = check_block(shape, y, slot_gates, w_post, gate))) return rc;
    if (!d_x) return api_fail(EIDM_E_INVALID, "d_x is NULL");
    if (!d_out && !d_normed) return api_fail(EIDM_E_INVALID, "no gradient is given");
    if ((w_pre != nullptr) != (d_normed != nullptr)) return api_fail(EIDM_E_INVALID, "w_pre and d_normed go together");
    if (w_pre && !stream_rows) return api_fail(EIDM_E_INVALID, "the rows that the norm read are NULL");
    if ((y != nullptr) != (d_z != nullptr)) return api_fail(EIDM_E_INVALID, "d_z is given exactly with y");
    if ((d_slot_gates && !slot_gates) || (d_gate && !gate) || (d_w_post && !w_post) || (d_w_pre && !w_pre))
        return api_fail(EIDM_E_INVALID, "a gradient of an input that is not given");
    const uint32_t ss = scalar_bytes(shape->stream_dtype), sw = scalar_bytes(shape->weight_dtype);
    if (!is_aligned(stream_rows, ss) || !is_aligned(w_post, sw) || !is_aligned(w_pre, sw) || !is_aligned(y, 4) ||
        !is_aligned(slot_gates, 4) || !is_aligned(gate, 4) || !is_aligned(d_out, 4) || !is_aligned(d_normed, 4) ||
        !is_aligned(d_x, 4) || !is_aligned(d_z, 4) || !is_aligned(d_slot_gates, 4) || !is_aligned(d_gate, 4) ||
        !is_aligned(d_w_post, 4) || !is_aligned(d_w_pre, 4))
        return api_fail(EIDM_E_ALIGN, "buffers must be aligned to their scalars");
    const uint32_t blocks = back_blocks(shape);
    const uint64_t need = back_scratch_bytes(shape);
    if (!scratch || scratch_bytes < need)
        return api_fail(EIDM_E_SIZE, "the gradients need %llu bytes of scratch, got %llu", (unsigned long long)need,
                        (unsigned long long)(scratch ? scratch_bytes : 0));
    if (!is_aligned(scratch, 256)) return api_fail(EIDM_E_ALIGN, "scratch must be 256-byte aligned");
    NormArgs a = norm_args(shape, y);
    a.x = stream_rows;
    a.slot_gates = slot_gates;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.d_out = d_out;
    a.d_normed = d_normed;
    a.d_x = d_x;
    a.d_z = d_z;
    a.d_slot_gates = d_slot_gates;
    a.d_gate = d_gate;
    a.partial = static_cast<float*>(scratch);
    a.rest = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + back_sums_bytes(shape));
    const bool channel = d_gate && shape->gate_layout == EIDM_GATE_CHANNEL;
    a.sums = (d_w_pre ? kSumPre : 0) | (d_w_post ? kSumPost : 0) | (channel ? kSumGate : 0);
    hipStream_t st = static_cast<hipStream_t>(stream);
    const uint32_t h = a.hidden;
    uint32_t block = kBackBlock, lds = 0;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(block), lds, st, a); };
    auto read_twice = [&] {
        block = kLongBlock;
        lds = 3 * ((h + kUnit - 1) / kUnit) * (uint32_t)sizeof(float4);
        const bool in_lds = lds <= kLongLds;
        if (!in_lds) lds = 0;
        if (d_slot_gates) in_lds ? go(block_norm_backward_long_kernel<true, true>) : go(block_norm_backward_long_kernel<false, true>);
        else in_lds ? go(block_norm_backward_long_kernel<true, false>) : go(block_norm_backward_long_kernel<false, false>);
    };
    auto by_length = [&](auto whole) {
        constexpr bool W = decltype(whole)::value;
        if (back_long(h)) return read_twice();
        if (h <= 256) return go(block_norm_backward_kernel<64, kBackBlock, 1, W>);
        if (h <= 512) return go(block_norm_backward_kernel<64, kBackBlock, 2, W>);
        if (h <= 1024) return go(block_norm_backward_kernel<256, kBackBlock, 1, W>);
        if (h <= 2048) return go(block_norm_backward_kernel<512, kBackBlock, 1, W>);
        go(block_norm_backward_kernel<512, kBackBlock, 2, W>);
    };
    if (h % kUnit == 0) by_length(std::true_type{});
    else by_length(std::false_type{});
    hipError_t err = launched(EIDM_KERNEL_BLOCK_NORM_BACKWARD, blocks, block, lds);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "norm gradient launch: %s", hipGetErrorString(err));
    if (a.sums) {
        const uint32_t grid = (h + 63) / 64;
        hipLaunchKernelGGL(column_sums_kernel, dim3(grid, 3), dim3(256), 0, st, a.partial, blocks, h, d_w_pre, d_w_post,
                           channel ? d_gate : nullptr);
        err = launched(EIDM_KERNEL_COLUMN_SUMS, grid * 3, 256, 0);
        if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "column sum launch: %s", hipGetErrorString(err));
    }
    return api_ok();
}

}  // extern "C"
