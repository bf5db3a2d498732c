// rows16.hpp -- a block of four wavefronts: 16*RT activation rows times 16*CT
// weight rows (output columns), both streamed from memory, in the library's
// fixed reduction order; used by the adapters' and the shared projection's
// products of a few rows.
//
// The step is v_mfma_f32_16x16x1_4b_f32: four independent 16x16 blocks, one
// product per output.  A 128-element round is four sub-rounds of 32; wavefront
// j takes sub-round j of every round, lane 16s+i holding granule 4j+s of
// activation row i and of weight row i, so block s is slice 4j+s of the fixed
// order and the 16 slices lie in four wavefronts: a product's k is split four
// ways without touching the order.  Per 32 elements a lane loads 32 bytes of
// activations per row tile and 16 (32 for f32) of weights, a quarter of the
// registers in flight that the 4x4x1 step needs for as many rows.  Output
// register 4s+v of lane l is slice 4j+s, row 4*(l/16)+v, column l%16; the
// wavefronts' sums meet in LDS, where wavefront v takes the rows 4*(l/16)+v.
#pragma once

#include "eidm_device.hpp"
#include "few_rows.hpp"

namespace eidm {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileWaves = 4;

// Tiles whose sums meet in LDS at once: up to four (64 KB), else half of them.
constexpr int rows16_part(int tiles) { return tiles > 4 ? tiles / 2 : tiles; }
// LDS floats of rows16_product
constexpr uint32_t rows16_lds(int tiles) { return (uint32_t)rows16_part(tiles) * kTileWaves * 16 * 64; }

// D rounds are in flight, 4 for up to two tiles and 2 beyond: what a unit's
// cache holds of misses bounds the loads, and more rounds than that only push
// its lines out (64 x 1536 x 4096 bf16, two tiles: 20.1 us with 4, 20.9 with 6,
// 20.9 with 8, 24.3 with 2; 512 x 1024 x 2048, four tiles: 29.9 with 2, 31.0
// with 4, 34.9 with 6).
//
// wrow[c]: this lane's weight row (row l%16 of column tile c), xrow[t]: its
// activation row of row tile t; lanes without one repeat a valid row.  On
// return total[t][c] of lane l of wavefront v is (row 4*(l/16)+v of tile t,
// column l%16 of tile c).  The block's four wavefronts call it together; xs
// (rows16_lds(RT*CT) floats) may be reused after the next barrier.
template <int DT, int RT, int CT, int D>
__device__ __forceinline__ void rows16_product(const uint8_t* const (&wrow)[CT], const float* const (&xrow)[RT], int k,
                                               float* xs, float (&total)[RT][CT]) {
    constexpr int S = DtypeSize<DT>::value;
    constexpr int NP = S / 2;
    const int lane = threadIdx.x & 63, s = lane >> 4;
    const int j = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int full = k / kRoundK;

    f32x16 acc[RT][CT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[t][c] = f32x16{};

    struct Slot {
        fr_u32x4 w[CT][NP];
        f32x4 x[RT][2];
    };
    const int at0 = j * 32 + s * kGranule;  // this lane's elements of a round
    auto fetch = [&](int r, Slot& t) {
        const size_t at = (size_t)r * kRoundK + at0;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < NP; ++i)
                t.w[c][i] = *reinterpret_cast<const fr_u32x4_a2*>(wrow[c] + at * S + 16 * i);
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            t.x[u][0] = *reinterpret_cast<const fr_f32x4_a4*>(xrow[u] + at);
            t.x[u][1] = *reinterpret_cast<const fr_f32x4_a4*>(xrow[u] + at + 4);
        }
    };
    auto consume = [&](const Slot& t, bool partial = false) {
        float w[CT][kGranule], x[RT][kGranule];
        partial = partial && k >= kGranule;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            few_widen<DT>(t.w[c], w[c]);
            if (partial) few_shift(w[c], full * kRoundK + at0, k);
        }
#pragma unroll
        for (int u = 0; u < RT; ++u) {
#pragma unroll
            for (int i = 0; i < kGranule; ++i) x[u][i] = t.x[u][i / 4][i % 4];
            if (partial) few_shift(x[u], full * kRoundK + at0, k);
        }
#pragma unroll
        for (int i = 0; i < kGranule; ++i)
#pragma unroll
            for (int u = 0; u < RT; ++u)
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    acc[u][c] = __builtin_amdgcn_mfma_f32_16x16x1f32(x[u][i], w[c][i], acc[u][c], 0, 0, 0);
    };

    Slot ring[D];
    if (full > 0) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            fetch(min(d, full - 1), ring[d]);  // past the end: the last round again, never consumed
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    Slot tail{};  // the partial last round: zeros past k
    const int kk = full * kRoundK + at0;
    if (full * kRoundK < k) {
        if (k >= kGranule) {
            const size_t at = (size_t)few_clamp(kk, k);
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    tail.w[c][i] = *reinterpret_cast<const fr_u32x4_a2*>(wrow[c] + at * S + 16 * i);
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                tail.x[u][0] = *reinterpret_cast<const fr_f32x4_a4*>(xrow[u] + at);
                tail.x[u][1] = *reinterpret_cast<const fr_f32x4_a4*>(xrow[u] + at + 4);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kGranule; ++i)
                if (kk + i < k) {
#pragma unroll
                    for (int u = 0; u < RT; ++u) tail.x[u][i / 4][i % 4] = xrow[u][kk + i];
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        if constexpr (S == 4)
                            tail.w[c][i / 4][i % 4] = *reinterpret_cast<const uint32_t*>(wrow[c] + (size_t)(kk + i) * 4);
                        else
                            tail.w[c][0][i / 2] |=
                                (uint32_t)*reinterpret_cast<const uint16_t*>(wrow[c] + (size_t)(kk + i) * 2) << (i % 2 * 16);
                    }
                }
        }
    }
    // every slot is refilled unconditionally, so each wait counts the same loads
    int r = 0;
    for (; r + D < full; r += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            consume(ring[d]);
            fetch(min(r + d + D, full - 1), ring[d]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (full > 0) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (r + d < full) consume(ring[d]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (full * kRoundK < k) consume(tail, true);

    // pairs (slice, slice^8), then ^4: the wavefronts; ^2, ^1: the blocks
    constexpr int T = RT * CT, P = rows16_part(T);
#pragma unroll
    for (int t0 = 0; t0 < T; t0 += P) {
        __syncthreads();  // xs is free
        f32x4* mine = reinterpret_cast<f32x4*>(xs) + (size_t)j * P * 4 * 64 + lane;
#pragma unroll
        for (int t = 0; t < P; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) {  // the four blocks' sums of one output together
                const f32x16& e = acc[(t0 + t) / CT][(t0 + t) % CT];
                mine[(t * 4 + v) * 64] = f32x4{e[v], e[4 + v], e[8 + v], e[12 + v]};
            }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < P; ++t) {
            const f32x4* p = reinterpret_cast<const f32x4*>(xs) + (t * 4 + j) * 64 + lane;
            constexpr int W = P * 4 * 64;
            const f32x4 a = p[0], b = p[W], c = p[2 * W], d = p[3 * W];
            f32x4 q;
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = (a[i] + c[i]) + (b[i] + d[i]);
            total[(t0 + t) / CT][(t0 + t) % CT] = (q[0] + q[2]) + (q[1] + q[3]);
        }
    }
}

}  // namespace eidm
