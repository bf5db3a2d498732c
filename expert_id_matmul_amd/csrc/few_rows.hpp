// few_rows.hpp -- one wavefront's product of a few activation rows with 4*C
// weight rows (output columns), in the library's fixed reduction order; used
// by the few-token expert layer and by the adapters' low-rank products.
//
// A weight row is read once for up to 16 activation rows.  The lane layout is
// that of the 4x4x1 matrix-core step (eidm_device.hpp): lane 4b+i holds, per
// 128-element round, granule b of weight row i of each column group and of
// activation row i of each row group, so one v_mfma_f32_4x4x1_16b_f32 does
// one product for 4 rows x 4 columns x 16 slices.  A single activation row
// takes the same step on the vector ALU (one lane per slice and column: half
// the issue cycles, the same bits).
//
// Rounds run through a ring of D register slots, as in direct_wave.hpp: all
// D rounds ahead are in flight, each wait is for the oldest slot only.
// Rows need no 16-byte alignment: the loads are declared with the scalar's
// alignment, which global loads take at any address; only the last, partial
// round is masked (per granule; a granule cut by k is read element-wise).
#pragma once

#include "eidm_device.hpp"

namespace eidm {

typedef unsigned int fr_u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any 2-byte (weights) or 4-byte (activations) boundary
typedef fr_u32x4 fr_u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 fr_f32x4_a4 __attribute__((aligned(4)));

template <int DT, int C, int RG>
struct FewSlot {
    fr_u32x4 w[C][DtypeSize<DT>::value / 2];
    f32x4 x[RG][2];
};

template <int DT>
__device__ __forceinline__ void few_widen(const fr_u32x4 (&p)[DtypeSize<DT>::value / 2], float (&w)[kGranule]) {
    if constexpr (DT == kDtypeF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __uint_as_float(p[0][i]);
            w[4 + i] = __uint_as_float(p[1][i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) widen_pair<DT>(p[0][i], w[2 * i], w[2 * i + 1]);
    }
}

// Accumulates acc[g][c] over k.  ONE: row group 0 holds one row, every lane
// of slice b passes that row, and acc[0][c][0] of lane 4b+i is column i's
// slice sum; else acc[g][c][v] of lane 4b+i is (row v, column i) of slice b.
// wrow[c], xrow[g]: this lane's weight row and activation row (the caller
// repeats a valid row for lanes that have none).  NT: weights are read once,
// so their loads are non-temporal.
template <int DT, int C, int RG, int D, bool ONE, bool NT = true>
__device__ __forceinline__ void few_rows_product(const uint8_t* const (&wrow)[C], const float* const (&xrow)[RG], int k,
                                                 f32x4 (&acc)[RG][C]) {
    constexpr int S = DtypeSize<DT>::value;
    constexpr int NP = S / 2;
    const int b = (threadIdx.x & 63) >> 2;
    const int full = k / kRoundK;

#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[g][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto fetch = [&](int r, FewSlot<DT, C, RG>& s) {
        const size_t at = (size_t)r * kRoundK + (size_t)b * kGranule;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const fr_u32x4_a2* p = reinterpret_cast<const fr_u32x4_a2*>(wrow[c] + at * S + 16 * i);
                s.w[c][i] = NT ? __builtin_nontemporal_load(p) : *p;
            }
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            s.x[g][0] = *reinterpret_cast<const fr_f32x4_a4*>(xrow[g] + at);
            s.x[g][1] = *reinterpret_cast<const fr_f32x4_a4*>(xrow[g] + at + 4);
        }
    };
    auto step = [&](const float (&w)[C][kGranule], const float (&x)[RG][kGranule]) {
#pragma unroll
        for (int i = 0; i < kGranule; ++i)
#pragma unroll
            for (int g = 0; g < RG; ++g)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if constexpr (ONE)
                        acc[g][c][0] = fma_step(x[g][i], w[c][i], acc[g][c][0]);
                    else
                        acc[g][c] = mfma_step(x[g][i], w[c][i], acc[g][c]);
                }
    };
    auto consume = [&](const FewSlot<DT, C, RG>& s) {
        float w[C][kGranule], x[RG][kGranule];
#pragma unroll
        for (int c = 0; c < C; ++c) few_widen<DT>(s.w[c], w[c]);
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[g][i] = s.x[g][0][i];
                x[g][4 + i] = s.x[g][1][i];
            }
        step(w, x);
    };

    if (full > 0) {
        FewSlot<DT, C, RG> ring[D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            fetch(min(d, full - 1), ring[d]);  // past the end: the last round again, never consumed
            __builtin_amdgcn_sched_barrier(0);
        }
        int r = 0;
        for (; r + 2 * D <= full; r += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                consume(ring[d]);
                fetch(r + d + D, ring[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int j = 0; j < 2 * D; ++j) {
            if (r + j < full) {
                consume(ring[j % D]);
                if (r + j + D < full) fetch(r + j + D, ring[j % D]);
            }
        }
    }
    if (full * kRoundK < k) {  // the partial last round
        const int kk = full * kRoundK + b * kGranule;
        float w[C][kGranule], x[RG][kGranule];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (kk + kGranule <= k) {
                fr_u32x4 p[NP];
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    p[i] = *reinterpret_cast<const fr_u32x4_a2*>(wrow[c] + (size_t)kk * S + 16 * i);
                few_widen<DT>(p, w[c]);
            } else {
                load_weight_granule<DT>(wrow[c], kk, k, true, false, w[c]);
            }
        }
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            if (kk + kGranule <= k) {
                const f32x4 a = *reinterpret_cast<const fr_f32x4_a4*>(xrow[g] + kk);
                const f32x4 c = *reinterpret_cast<const fr_f32x4_a4*>(xrow[g] + kk + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[g][i] = a[i];
                    x[g][4 + i] = c[i];
                }
            } else {
                load_input_granule(xrow[g], kk, k, true, false, x[g]);
            }
        }
        step(w, x);
    }
}

// The 16 slice sums of (row v, column i), v = 0..3, combined in the fixed
// pairing by recursive halving: two of the four rows go to each half of the
// slices, then one to each quarter, so a lane adds 2 + 1 + 1 + 1 sums in place
// of 4 times 4.  f32 addition is commutative, so both partners of a pair hold
// the same bits as the butterfly's.  Lane 4b+i returns the total of row
// few_row(b), column i (slices b and b^1, b^2, b^3 hold the same total).
__device__ __forceinline__ int few_row(int b) { return ((b >> 3) & 1) * 2 + ((b >> 2) & 1); }

__device__ __forceinline__ float few_rows_total(const f32x4& a) {
    const int b = (threadIdx.x & 63) >> 2;
    const bool hi = b & 8, mid = b & 4;
    // slices b and b^8: the half with bit 3 set keeps rows 2, 3
    float p = hi ? a[2] : a[0], q = hi ? a[3] : a[1];
    p += __shfl_xor(hi ? a[0] : a[2], 32);
    q += __shfl_xor(hi ? a[1] : a[3], 32);
    // slices b and b^4: bit 2 keeps the odd row
    float t = mid ? q : p;
    t += __shfl_xor(mid ? p : q, 16);
    t += __shfl_xor(t, 8);
    t += __shfl_xor(t, 4);
    return t;
}

}  // namespace eidm
