// rows16.hpp -- one wavefront's product of 16 activation rows with 16*NB
// weight rows (output columns), both streamed from memory, in the library's
// fixed reduction order; used by the adapters' products where several rows
// share a weight.
//
// The step is v_mfma_f32_16x16x1_4b_f32: four independent 16x16 blocks, one
// product per output.  A 128-element round is four sub-rounds j; lane 16s+i
// holds granule 4j+s of activation row i and of weight row i, so block s of
// sub-round j is slice 4j+s of the fixed order and each sub-round has its own
// accumulator set.  Per 32 elements a lane loads 32 bytes of activations and
// 16 (32 for f32) of each weight row for 16x16 outputs per slice, a quarter of
// the registers in flight that the 4x4x1 step needs for as many rows.  Output
// register 4s+v of lane l is slice set s, row 4*(l/16)+v, column l%16, so all
// 16 slices of an output sit in one lane and the pairing needs no exchange.
#pragma once

#include "eidm_device.hpp"
#include "few_rows.hpp"

namespace eidm {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileRows = 16;

// wrow[c]: this lane's weight row (row l%16 of tile c), xrow: its activation
// row; lanes without one repeat a valid row.  total[c][v]: row 4*(l/16)+v,
// column l%16 of tile c.
template <int DT, int NB, int D, bool NT>
__device__ __forceinline__ void rows16_product(const uint8_t* const (&wrow)[NB], const float* xrow, int k,
                                               f32x4 (&total)[NB]) {
    static_assert(D % 4 == 0, "a slot keeps its sub-round");
    constexpr int S = DtypeSize<DT>::value;
    constexpr int NP = S / 2;
    const int s = (threadIdx.x & 63) >> 4;
    const int full = k / kRoundK * 4;  // whole sub-rounds

    f32x16 acc[4][NB];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < NB; ++c) acc[j][c] = f32x16{};

    struct Slot {
        fr_u32x4 w[NB][NP];
        f32x4 x[2];
    };
    auto fetch = [&](int r, Slot& t) {  // sub-round r: elements 32r + 8s ..
        const size_t at = (size_t)r * 32 + (size_t)s * kGranule;
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const fr_u32x4_a2* p = reinterpret_cast<const fr_u32x4_a2*>(wrow[c] + at * S + 16 * i);
                t.w[c][i] = NT ? __builtin_nontemporal_load(p) : *p;
            }
        t.x[0] = *reinterpret_cast<const fr_f32x4_a4*>(xrow + at);
        t.x[1] = *reinterpret_cast<const fr_f32x4_a4*>(xrow + at + 4);
    };
    auto consume = [&](f32x16 (&a)[NB], const Slot& t) {
        float w[NB][kGranule];
#pragma unroll
        for (int c = 0; c < NB; ++c) few_widen<DT>(t.w[c], w[c]);
#pragma unroll
        for (int i = 0; i < kGranule; ++i)
#pragma unroll
            for (int c = 0; c < NB; ++c)
                a[c] = __builtin_amdgcn_mfma_f32_16x16x1f32(t.x[i / 4][i % 4], w[c][i], a[c], 0, 0, 0);
    };

    if (full > 0) {
        Slot ring[D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            fetch(min(d, full - 4 + d % 4), ring[d]);  // past the end: a sub-round again, never consumed
            __builtin_amdgcn_sched_barrier(0);
        }
        int r = 0;
        for (; r + 2 * D <= full; r += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                consume(acc[d % 4], ring[d]);
                fetch(r + d + D, ring[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int j = 0; j < 2 * D; ++j) {
            if (r + j < full) {
                consume(acc[j % 4], ring[j % D]);
                if (r + j + D < full) fetch(r + j + D, ring[j % D]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (full * 32 < k) {  // the partial last round: zeros past k
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Slot t{};
            const int kk = (full + j) * 32 + s * kGranule;
            if (kk + kGranule <= k) {
                fetch(full + j, t);
            } else if (kk < k) {
#pragma unroll
                for (int i = 0; i < kGranule; ++i)
                    if (kk + i < k) {
                        t.x[i / 4][i % 4] = xrow[kk + i];
#pragma unroll
                        for (int c = 0; c < NB; ++c) {
                            if constexpr (S == 4)
                                t.w[c][i / 4][i % 4] = *reinterpret_cast<const uint32_t*>(wrow[c] + (size_t)(kk + i) * 4);
                            else
                                t.w[c][0][i / 2] |=
                                    (uint32_t)*reinterpret_cast<const uint16_t*>(wrow[c] + (size_t)(kk + i) * 2) << (i % 2 * 16);
                        }
                    }
            }
            consume(acc[j], t);
        }
    }
    // pairs (slice, slice^8), then ^4: the sub-round sets; ^2, ^1: the blocks
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            float q[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int e = 4 * b + v;
                q[b] = (acc[0][c][e] + acc[2][c][e]) + (acc[1][c][e] + acc[3][c][e]);
            }
            total[c][v] = (q[0] + q[2]) + (q[1] + q[3]);
        }
}

}  // namespace eidm
