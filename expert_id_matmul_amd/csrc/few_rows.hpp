// few_rows.hpp -- one wavefront's product of a few activation rows, staged in
// LDS, with 4*C weight rows (output columns), in the library's fixed
// reduction order; used by the few-token expert layer and by the adapters.
//
// A weight row is read once for up to 16 activation rows.  The lane layout is
// that of the 4x4x1 matrix-core step (eidm_device.hpp): lane 4b+i holds, per
// 128-element round, granule b of weight row i of each column group and of
// activation row i of each row group, so one v_mfma_f32_4x4x1_16b_f32 does
// one product for 4 rows x 4 columns x 16 slices.  A single activation row
// takes the same step on the vector ALU (one lane per slice and column: half
// the issue cycles, the same bits).
//
// What bounds it is the weight stream, so the registers hold weights only: a
// ring of D rounds in flight, each wait for the oldest one, as in
// direct_wave.hpp.  With the activations in the ring too (8 registers a round
// for every four rows) the kernel spilled, and a spill's reload waits for the
// whole ring; in LDS they cost no register and no place in the load queue.
// Weight rows need no 16-byte alignment: the loads are declared with the
// scalar's alignment, which global loads take at any address; the last,
// partial round is read within the row and shifted into place.
#pragma once

#include "eidm_device.hpp"

namespace eidm {

typedef unsigned int fr_u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any 2-byte (weights) or 4-byte (activations) boundary
typedef fr_u32x4 fr_u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 fr_f32x4_a4 __attribute__((aligned(4)));

constexpr int kFewRows = 16;  // activation rows of one pass over a weight row

// An activation row in LDS: per 128-element round the first halves of its 16
// granules, then the second halves, zero past k; rows are 64 bytes off a
// multiple of the 256-byte bank span, so the four rows of a row group that a
// 16-byte read takes together fall on different banks.
__host__ __device__ constexpr uint32_t few_row_floats(uint32_t k) { return (k + 127) / 128 * 128 + 16; }

// Copies rows row_of(0 .. count-1) of k f32 elements (4-byte aligned) to LDS
// rows 0 .. count-1; the whole block takes part, each thread with kBatch loads
// in flight.  issue() requests the first of them, finish() stores those and
// copies the rest, so other work can stand between the two; a barrier must
// follow before the rows are read.
//
// A wavefront takes units of 64 consecutive 16-byte pieces of one row, so
// that all index arithmetic but a lane's own place is scalar (per thread it
// was hoisted out of the caller's loops and spilled there).
template <uint32_t kBatch, typename RowOf>
struct FewStage {
    float* xs;
    uint32_t count, k;
    RowOf row_of;
    f32x4 v[kBatch];

    __device__ __forceinline__ static uint32_t waves() { return blockDim.x >> 6; }
    __device__ __forceinline__ static uint32_t wave() {
        return (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    }
    __device__ __forceinline__ uint32_t pieces() const { return (k + 127) / 128 * 32; }  // of a row, zeros past k
    __device__ __forceinline__ uint32_t units() const { return (pieces() + 63) / 64; }   // of a row

    __device__ __forceinline__ void load(uint32_t u0) {
        const uint32_t per = units();
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j) {
            const uint32_t u = u0 + j * waves();
            if (u >= count * per) break;  // wave-uniform
            const uint32_t r = u / per, p = ((u - r * per) * 64 + (threadIdx.x & 63)) * 4;
            const float* src = row_of(r) + p;
            v[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (p + 4 <= k) {
                v[j] = *reinterpret_cast<const fr_f32x4_a4*>(src);
            } else {
#pragma unroll
                for (uint32_t e = 0; e < 3; ++e)
                    if (p + e < k) v[j][e] = src[e];
            }
        }
    }
    __device__ __forceinline__ void store(uint32_t u0) const {
        const uint32_t per = units(), stride = few_row_floats(k);
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j) {
            const uint32_t u = u0 + j * waves();
            if (u >= count * per) break;
            const uint32_t r = u / per, p = (u - r * per) * 64 + (threadIdx.x & 63);
            if (p < pieces())
                *reinterpret_cast<f32x4*>(xs + (size_t)r * stride + p / 32 * 128 + (p & 1) * 64 + p % 32 / 2 * 4) = v[j];
        }
    }
    __device__ __forceinline__ void issue() { load(wave()); }
    __device__ __forceinline__ void finish() {
        store(wave());
        for (uint32_t u0 = wave() + kBatch * waves(); u0 < count * units(); u0 += kBatch * waves()) {
            load(u0);
            store(u0);
        }
    }
};

template <uint32_t kBatch, typename RowOf>
__device__ __forceinline__ FewStage<kBatch, RowOf> few_stage(float* xs, uint32_t count, uint32_t k, RowOf row_of) {
    return FewStage<kBatch, RowOf>{xs, count, k, row_of, {}};
}

// Elements kk .. kk+7 of a row of k of which not all need exist (lane-varying
// kk, wave-uniform k): where the row has 8 elements they are loaded from
// min(kk, k - 8), so the load crosses no end and waits for no branch, and
// few_shift() moves them into place once they have arrived.
__device__ __forceinline__ int few_clamp(int kk, int k) { return min(kk, k - kGranule); }

// w: the elements from few_clamp(kk, k) on -> those from kk on, zeros past k.
__device__ __forceinline__ void few_shift(float (&w)[kGranule], int kk, int k) {
    const bool cut = kk < k && kk + kGranule > k, past = kk >= k;
    for (int s = (kGranule - k % kGranule) % kGranule; s > 0; --s) {  // the cut granule's distance, one for all lanes
#pragma unroll
        for (int i = 0; i < kGranule; ++i) w[i] = cut ? (i + 1 < kGranule ? w[i + 1] : 0.0f) : w[i];
    }
#pragma unroll
    for (int i = 0; i < kGranule; ++i) w[i] = past ? 0.0f : w[i];
}

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

// The weight stream of one wavefront: C weight rows per lane (4*C columns),
// D rounds in flight.
template <int DT, int C, int D, bool NT>
struct FewStream {
    static constexpr int S = DtypeSize<DT>::value;
    static constexpr int NP = S / 2;
    static constexpr int kColumns = C;
    using Rows = const uint8_t* const (&)[C];
    struct Slot {
        fr_u32x4 w[C][NP];
    };
    Slot ring[D];
    Slot tail;  // the partial last round

    __device__ __forceinline__ static int slice() { return (threadIdx.x & 63) >> 2; }

    // wrow[c]: this lane's weight row (lanes without one repeat a valid row)
    __device__ __forceinline__ static void fetch(const uint8_t* const (&wrow)[C], int r, Slot& s) {
        const size_t at = ((size_t)r * kRoundK + (size_t)slice() * kGranule) * S;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const fr_u32x4_a2* p = reinterpret_cast<const fr_u32x4_a2*>(wrow[c] + at + 16 * i);
                s.w[c][i] = NT ? __builtin_nontemporal_load(p) : *p;  // NT: weights that are read once
            }
    }

    __device__ __forceinline__ void fetch_tail(Rows wrow, int k) {
        const int full = k / kRoundK;
        if (full * kRoundK == k) return;
        const int kk = full * kRoundK + slice() * kGranule;
        if (k >= kGranule) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    tail.w[c][i] = *reinterpret_cast<const fr_u32x4_a2*>(wrow[c] + (size_t)few_clamp(kk, k) * S + 16 * i);
            return;
        }
        tail = Slot{};
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < kGranule; ++i)
                if (kk + i < k) {
                    if constexpr (S == 4)
                        tail.w[c][i / 4][i % 4] = *reinterpret_cast<const uint32_t*>(wrow[c] + (size_t)(kk + i) * 4);
                    else
                        tail.w[c][0][i / 2] |=
                            (uint32_t)*reinterpret_cast<const uint16_t*>(wrow[c] + (size_t)(kk + i) * 2) << (i % 2 * 16);
                }
    }

    // Requests the first rounds (and the partial one) of a product.
    __device__ __forceinline__ void start(const uint8_t* const (&wrow)[C], int k) {
        const int full = k / kRoundK;
        if (full > 0) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                fetch(wrow, min(d, full - 1), ring[d]);  // past the end: the last round again, never consumed
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        fetch_tail(wrow, k);
    }

    // The product of the rows that start() requested; with MORE, start(next)
    // has been done on return: its requests take the slots as the last rounds
    // free them.  RG row groups of four activation rows in LDS, xl[g] this
    // lane's row (row q of group g): acc[g][c][v] of lane 4b+i is (row v,
    // column i) of slice b.  RG = 0: one row, the same in every lane, and
    // acc[0][c][0] is column i's slice sum.
    //
    // Every slot is refilled unconditionally (past the end the last round is
    // requested again), so that each wait counts the same loads on every path.
    template <int RG, bool MORE>
    __device__ __forceinline__ void run(Rows wrow, Rows next, const float* const (&xl)[RG ? RG : 1], int k,
                                        f32x4 (&acc)[RG ? RG : 1][C]) {
        constexpr int G = RG ? RG : 1;
        const int b = slice();
        const int full = k / kRoundK;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int c = 0; c < C; ++c) acc[g][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        // the activations of a round (both halves of this lane's granule); with
        // at most four rows they are read one round ahead, since then a
        // wavefront's few steps do not cover the latency of an LDS read
        constexpr bool kAhead = RG <= 1;
        f32x4 ahead[G][2];
        auto read = [&](int r, int h, f32x4 (&x)[G]) {
#pragma unroll
            for (int g = 0; g < G; ++g) x[g] = *reinterpret_cast<const f32x4*>(xl[g] + r * kRoundK + h * 64 + b * 4);
        };
        auto read_ahead = [&](int r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4 x[G];
                read(r, h, x);
#pragma unroll
                for (int g = 0; g < G; ++g) ahead[g][h] = x[g];
            }
        };
        const int last = (k + kRoundK - 1) / kRoundK - 1;
        if constexpr (kAhead) read_ahead(0);
        auto consume = [&](int r, const Slot& s, bool partial = false) {
            f32x4 x[2][G];
            if constexpr (kAhead) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int g = 0; g < G; ++g) x[h][g] = ahead[g][h];
                read_ahead(min(r + 1, last));
            }
            float w[C][kGranule];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                few_widen<DT>(s.w[c], w[c]);
                if (partial && k >= kGranule) few_shift(w[c], r * kRoundK + b * kGranule, k);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (!kAhead) read(r, h, x[h]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            if constexpr (RG == 0)
                                acc[g][c][0] = fma_step(x[h][g][i], w[c][h * 4 + i], acc[g][c][0]);
                            else
                                acc[g][c] = mfma_step(x[h][g][i], w[c][h * 4 + i], acc[g][c]);
                        }
            }
        };

        int r = 0;
        for (; r + D < full; r += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                consume(r + d, ring[d]);
                fetch(wrow, min(r + d + D, full - 1), ring[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (full > 0) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (r + d < full) consume(r + d, ring[d]);
                if constexpr (MORE) fetch(next, min(d, full - 1), ring[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (full * kRoundK < k) {
            consume(full, tail, true);
            if constexpr (MORE) fetch_tail(next, k);
        }
    }
};

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

// `count` (1..16) staged rows, row i at xs + lds_row(i) * stride, times the
// 4*C weight rows that `w` has been started on (MORE: and is then started on
// `next`): emit(i, totals[C]) for every
// row, in lanes that hold the totals of column q = lane & 3 of each group.
template <int RG, bool MORE, typename Stream, typename LdsRow, typename Emit>
__device__ __forceinline__ void few_rows_tile(Stream& w, typename Stream::Rows wrow, typename Stream::Rows next,
                                              const float* xs, uint32_t stride, uint32_t count, int k, LdsRow lds_row,
                                              Emit emit) {
    constexpr int C = Stream::kColumns;
    constexpr int G = RG ? RG : 1;
    const int lane = threadIdx.x & 63;
    const int b = lane >> 2;
    const uint32_t q = lane & 3;
    const float* xl[G];
#pragma unroll
    for (int g = 0; g < G; ++g) xl[g] = xs + (size_t)lds_row(RG ? min(4 * g + q, count - 1) : 0) * stride;
    f32x4 acc[G][C];
    w.template run<RG, MORE>(wrow, next, xl, k, acc);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = RG ? few_rows_total(acc[g][c]) : slice_tree(acc[g][c][0]);
        const uint32_t r = RG ? 4 * g + few_row(b) : 0;
        if (RG ? ((b & 3) == 0 && r < count) : b == 0) emit(r, v);
    }
}

template <bool MORE, typename Stream, typename LdsRow, typename Emit>
__device__ __forceinline__ void few_rows_any(Stream& w, typename Stream::Rows wrow, typename Stream::Rows next,
                                             const float* xs, uint32_t stride, uint32_t count, int k, LdsRow lds_row,
                                             Emit emit) {
    if (count == 1) few_rows_tile<0, MORE>(w, wrow, next, xs, stride, count, k, lds_row, emit);
    else if (count <= 4) few_rows_tile<1, MORE>(w, wrow, next, xs, stride, count, k, lds_row, emit);
    else if (count <= 8) few_rows_tile<2, MORE>(w, wrow, next, xs, stride, count, k, lds_row, emit);
    else few_rows_tile<4, MORE>(w, wrow, next, xs, stride, count, k, lds_row, emit);
}

}  // namespace eidm
