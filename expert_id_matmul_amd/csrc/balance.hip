// balance.hip -- the router's balance loss with per-expert counts, and the
// gradient of its logits through the loss and through the gates.
//
// For a sequence q of T tokens, with s = sigmoid(logits) (the router's scores:
// route_wave.hpp) and p[t, e] = s[t, e] / sum_e s[t, e]:
//   counts[q, e] = picks of e by q's tokens
//   load[q, e]   = counts[q, e] * n_experts / (top_k * T)
//   mean[q, e]   = sum_t p[t, e] / T
//   loss         = coefficient / n_seqs * sum_q sum_e load[q, e] * mean[q, e]
// load is constant in the gradient.  With w = d_loss * coefficient / (n_seqs * T)
//   d_s[t, e]  = w * (load[q, e] - sum_e' load[q, e'] * p[t, e']) / sum_e s[t, e]
//              + (e is pick j) d_gates[t, j], or with renormalised gates
//                (d_gates[t, j] - sum_i d_gates[t, i] * gates[t, i]) / sum_i s[t, ids[t, i]]
//   d_logits   = d_s * s * (1 - s)
// Renormalised gates are ratios, of order one beside the smallest scores: those
// of tiny scores, and their gradients, come from the logits' differences.
//
// Bound by memory beyond a few thousand tokens (the logits once, their
// gradient once): a wavefront takes a token, its scores and its experts' sums
// over tokens stay in registers, 16 bytes a lane and load.  Sums over tokens go
// wavefront by wavefront and block by block in a fixed order, without floating
// atomics: the loss, counts and means are the same from run to run.  (A pick's
// gradient is added to its expert's by an atomic on the wavefront's own row of
// LDS: one each, since the router's ids of a token differ.)  Blocks take equal
// stretches of the batch, so that one long sequence keeps no block waiting
// (64 uneven sequences of 65536 tokens of 256 experts: 98 us by sequences).  The
// same batch now: parts 16.2 us (71 MB), their sums 7.4 (one trip to memory and
// the ticket), gradient 31.3 (141 MB, 4.5 TB/s).
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "api_checks.hpp"
#include "eidm.h"
#include "eidm_internal.hpp"
#include "route_wave.hpp"

namespace eidm {
namespace {

struct BalanceArgs {
    uint32_t m, n_experts, top_k, n_seqs, each;  // each: tokens of a part
    double coefficient;
    const float* logits;
    const uint32_t *ids, *seq_offsets;
    uint32_t* counts;
    float *mean_probs, *loss;
    // scratch
    uint32_t* part_counts;  // [parts + n_seqs][n_experts]
    float* part_probs;      // [parts + n_seqs][n_experts]
    double* part_loss;      // [n_seqs * expert tiles]
    uint32_t* ticket;
    // backward
    int renormalize;
    const float *d_gates, *d_loss;
    float* d_logits;
};

// Sequence q's tokens; offsets beyond m, or that go back, are cut.
__device__ __forceinline__ void seq_range(const BalanceArgs& a, uint32_t q, uint32_t& lo, uint32_t& hi) {
    lo = a.seq_offsets ? min(a.seq_offsets[q], a.m) : 0;
    hi = a.seq_offsets ? max(min(a.seq_offsets[q + 1], a.m), lo) : a.m;
}

// exp(x + rest), x <= 0 and rest a rounding of it: the argument's product with
// log2(e) in two parts, so that the error stays at an f32 rounding or two for
// any x (one product would lose |x| of them).  v_exp_f32 flushes what falls
// below 2^-126, an infinite x like -256; a NaN stays one.
__device__ __forceinline__ float exp_below(float x, float rest = 0.0f) {
    x = __builtin_elementwise_maximum(x, -256.0f);
    const float hi = x * 0x1.715476p+0f;
    const float lo = __builtin_fmaf(x, 0x1.4ae0cp-26f, __builtin_fmaf(x, 0x1.715476p+0f, -hi));
    const float e = __builtin_amdgcn_exp2f(hi);
    return __builtin_fmaf(e, __builtin_fmaf(lo, 0x1.62e43p-1f, rest), e);
}

// s = sigmoid(v) and s * (1 - s), without a difference that cancels.  Here and
// for the sums of scores the reciprocal is v_rcp_f32, an f32 step off at most
// where a division is half of one, in one instruction of about ten: the logits'
// gradient is 1.1e-7 from 64 bits (9.6e-8 by elementary f32 operations).
__device__ __forceinline__ void score(float v, float& s, float& slope) {
    const float t = exp_below(-fabsf(v)), r = __builtin_amdgcn_rcpf(1.0f + t);
    s = v >= 0.0f ? r : t * r;
    slope = t * r * r;
}

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}

__device__ __forceinline__ float lane_f(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

__device__ __forceinline__ float wave_sum_f(float v) {
    v += dpp_f<0xb1>(v);
    v += dpp_f<0x4e>(v);
    v += dpp_f<0x141>(v);
    v += dpp_f<0x140>(v);
    return (lane_f(v, 0) + lane_f(v, 16)) + (lane_f(v, 32) + lane_f(v, 48));
}

__device__ __forceinline__ float wave_max_f(float v) {  // a NaN is the largest
    v = __builtin_elementwise_maximum(v, dpp_f<0xb1>(v));
    v = __builtin_elementwise_maximum(v, dpp_f<0x4e>(v));
    v = __builtin_elementwise_maximum(v, dpp_f<0x141>(v));
    v = __builtin_elementwise_maximum(v, dpp_f<0x140>(v));
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(lane_f(v, 0), lane_f(v, 16)),
                                         __builtin_elementwise_maximum(lane_f(v, 32), lane_f(v, 48)));
}

// Where a sum of scores is below this, each is its logit's exponential (1 - s is
// 1 to 2^-28), and ratios of them are taken from the differences to the largest
// logit: the scores themselves are flushed below 2^-126.
constexpr float kTiny = 0x1p-28f;

// sigmoid(v) / sigmoid(most) for v <= most, both tiny; the difference's own rounding
// is added to it.
__device__ __forceinline__ float score_beside(float v, float most) {
    v = __builtin_elementwise_maximum(v, -512.0f);
    const float d = v - most;
    return exp_below(d, -most - (d - v));
}

// The largest logit whose score is 0 in f32: half of the smallest number, -150 ln 2.
constexpr float kNoScore = -0x1.9fe36ap+6f;
// The largest whose score is not above 2^-126, -126 ln 2.
constexpr float kLeastScore = -0x1.5d58ap+6f;

// Expert of a lane's slot v: runs of up to four neighbours, one load each.
template <int NV>
struct Experts {
    static constexpr int kRun = NV < 4 ? NV : 4;
    __device__ static uint32_t of(int v) { return (v / kRun) * 64 * kRun + (threadIdx.x & 63) * kRun + v % kRun; }
    __device__ static void load(const float* row, uint32_t n, float (&x)[NV]) {
#pragma unroll
        for (int g = 0; g < NV / kRun; ++g) {
            const uint32_t e = of(g * kRun);
            if (e + kRun <= n) __builtin_memcpy(&x[g * kRun], row + e, 4 * kRun);
            else
#pragma unroll
                for (int v = g * kRun; v < (g + 1) * kRun; ++v) x[v] = of(v) < n ? row[of(v)] : 0.0f;
        }
    }
    // Past the caches, which then keep the logits (65536 tokens of 256 experts: 62.9 -> 53.8 us).
    __device__ static void store(float* row, uint32_t n, const float (&x)[NV]) {
        typedef float Run __attribute__((ext_vector_type(kRun), aligned(4)));
#pragma unroll
        for (int g = 0; g < NV / kRun; ++g) {
            const uint32_t e = of(g * kRun);
            Run run;
            __builtin_memcpy(&run, &x[g * kRun], 4 * kRun);
            if (e + kRun <= n) __builtin_nontemporal_store(run, reinterpret_cast<Run*>(row + e));
            else
#pragma unroll
                for (int v = g * kRun; v < (g + 1) * kRun; ++v)
                    if (of(v) < n) row[of(v)] = x[v];
        }
    }
};

// A token's scores (0 past n_experts) and the factor that makes them
// probabilities.  Scores that are all tiny become their ratios to the largest,
// with a slope of the same (1 - s is 1): what follows takes them times that
// factor alone.  Where the largest itself is not above 2^-126 all are 0.
template <int NV>
__device__ __forceinline__ float scores(const float (&l)[NV], uint32_t n, float (&s)[NV], float (&slope)[NV]) {
    float total = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        score(l[v], s[v], slope[v]);
        if (n < 64 * NV && Experts<NV>::of(v) >= n) s[v] = slope[v] = 0.0f;
        total += s[v];
    }
    total = wave_sum_f(total);
    if (total < kTiny) {
        float most = -__builtin_inff();
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (Experts<NV>::of(v) < n) most = fmaxf(most, l[v]);
        most = wave_max_f(most);
        total = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            s[v] = most > kLeastScore && Experts<NV>::of(v) < n ? score_beside(l[v], most) : 0.0f;
            slope[v] = s[v];
            total += s[v];
        }
        total = wave_sum_f(total);
        if (total == 0.0f) return 0.0f;
    }
    return __builtin_amdgcn_rcpf(total);
}

constexpr int kWaves = 4;      // of a block of the gradient
constexpr int kPartWaves = 8;  // of a block of a part, half of them beyond 1024 experts (LDS)

// The last sequence that starts at or before token t (0 where none does): the
// wavefront looks at 64 offsets at a time, so that up to 64 sequences take one
// load's latency.
__device__ __forceinline__ uint32_t seq_of(const BalanceArgs& a, uint32_t t) {
    const uint32_t lane = threadIdx.x & 63;
    uint32_t lo = 0;
    for (uint32_t size = a.n_seqs; size > 1;) {
        const uint32_t step = (size + 63) / 64, at = lane * step;
        const uint32_t upto = (uint32_t)__popcll(__ballot(at < size && a.seq_offsets[lo + min(at, size - 1)] <= t));
        if (!upto) return lo;
        lo += (upto - 1) * step;
        size = min(step, size - (upto - 1) * step);
    }
    return lo;
}

// Block c: tokens c * each .. of the batch, whatever their sequences.  What it
// holds of sequence q goes to row c + q of the parts: a row of its own, since
// from one part to the next c or q (or both) grows.
template <int NV>
__global__ __launch_bounds__(64 * kPartWaves) void balance_part_kernel(BalanceArgs a) {
    extern __shared__ uint32_t hist[];  // [n_experts] counts, then [wavefronts][n_experts] sums
    float* sums = reinterpret_cast<float*>(hist + a.n_experts);
    const uint32_t lane = threadIdx.x & 63, n = a.n_experts, threads = blockDim.x, waves = threads >> 6;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;  // for the next kernel
    const uint32_t first = blockIdx.x * a.each, last = min(first + a.each, a.m);
    for (uint32_t t0 = first; t0 < last;) {
        const uint32_t q = a.seq_offsets ? seq_of(a, t0) : 0;
        uint32_t lo, hi;
        seq_range(a, q, lo, hi);
        if (t0 < lo || t0 >= hi) {  // no sequence's: on to where the next one starts
            const uint32_t next = t0 < lo ? lo : q + 1 < a.n_seqs ? a.seq_offsets[q + 1] : last;
            t0 = max(t0 + 1, min(next, last));
            continue;
        }
        const uint32_t end = min(hi, last);
        for (uint32_t e = threadIdx.x; e < n; e += threads) hist[e] = 0;
        __syncthreads();
        float acc[NV] = {};
        // the next token's logits and picks are requested while this one's are worked on
        float l[NV], next[NV];
        uint32_t id = n, next_id = n;
        auto request = [&](uint32_t t) {
            Experts<NV>::load(a.logits + (size_t)t * n, n, next);
            if (lane < a.top_k) next_id = a.ids[(size_t)t * a.top_k + lane];
        };
        if (t0 + wave < end) request(t0 + wave);
        for (uint32_t t = t0 + wave; t < end; t += waves) {
#pragma unroll
            for (int v = 0; v < NV; ++v) l[v] = next[v];
            id = next_id;
            if (t + waves < end) request(t + waves);
            if (id < n) atomicAdd(&hist[id], 1u);
            float s[NV], slope[NV];
            const float r = scores<NV>(l, n, s, slope);
#pragma unroll
            for (int v = 0; v < NV; ++v) acc[v] += s[v] * r;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (Experts<NV>::of(v) < n) sums[wave * n + Experts<NV>::of(v)] = acc[v];
        __syncthreads();
        const size_t row = (size_t)(blockIdx.x + q) * n;
        for (uint32_t e = threadIdx.x; e < n; e += threads) {
            a.part_counts[row + e] = hist[e];
            float p = 0.0f;
            for (uint32_t w = 0; w < waves; ++w) p += sums[w * n + e];
            a.part_probs[row + e] = p;
        }
        __syncthreads();
        t0 = end;
    }
}

constexpr uint32_t kFinish = 1024;  // threads of a block

// Block (expert tile, q): the parts' sums, GROUPS threads an expert; the last
// block to end adds the loss.  Few sequences have many parts each: 16 threads an
// expert.  Many have few: 4, since every block's turn at the ticket makes its
// XCD write its L2 back (2 us of 64 for 256 blocks).
template <uint32_t GROUPS>
__global__ __launch_bounds__(kFinish) void balance_finish_kernel(BalanceArgs a) {
    constexpr uint32_t TILE = kFinish / GROUPS, WAVES = TILE / 64;
    __shared__ double probs[GROUPS][TILE];
    __shared__ uint32_t picks[GROUPS][TILE];
    __shared__ double terms[kFinish / 64];
    __shared__ uint32_t last;
    const uint32_t lane = threadIdx.x & 63, in = threadIdx.x % TILE, group = threadIdx.x / TILE, n = a.n_experts;
    const uint32_t q = blockIdx.y, e = blockIdx.x * TILE + in;
    double p = 0.0;
    uint32_t c = 0;
    uint32_t lo, hi;
    seq_range(a, q, lo, hi);
    if (e < n && lo < hi) {
        const uint32_t from = lo / a.each, parts = (hi - 1) / a.each - from + 1;
#pragma unroll 8
        for (uint32_t i = group; i < parts; i += GROUPS) {
            const size_t at = (size_t)(from + i + q) * n + e;
            p += (double)a.part_probs[at];
            c += a.part_counts[at];
        }
    }
    probs[group][in] = p;
    picks[group][in] = c;
    __syncthreads();
    if (group == 0) {
#pragma unroll
        for (uint32_t i = 1; i < GROUPS; ++i) {
            p += probs[i][in];
            c += picks[i][in];
        }
        const double tokens = hi > lo ? (double)(hi - lo) : 1.0;
        const double mean = p / tokens;
        double term = 0.0;
        if (e < n) {
            a.counts[(size_t)q * n + e] = c;
            a.mean_probs[(size_t)q * n + e] = (float)mean;
            term = (double)c * mean * ((double)n / (a.top_k * tokens));
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) term += __shfl_xor(term, d);
        if (lane == 0) terms[in >> 6] = term;
    }
    __syncthreads();
    const uint32_t blocks = gridDim.x * gridDim.y, block = q * gridDim.x + blockIdx.x;
    if (threadIdx.x == 0) {
        double term = terms[0];
        for (uint32_t w = 1; w < WAVES; ++w) term += terms[w];
        __hip_atomic_store(&a.part_loss[block], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint32_t turn = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        last = turn + 1 == blocks;
    }
    __syncthreads();
    if (!last) return;
    // in the blocks' order, whichever came last
    double sum = 0.0;
    for (uint32_t i = threadIdx.x; i < blocks; i += kFinish)
        sum += __hip_atomic_load(&a.part_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) terms[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (uint32_t i = 1; i < kFinish / 64; ++i) sum += terms[i];
        *a.loss = (float)(sum * (a.coefficient / (double)a.n_seqs));
    }
}

// A wavefront takes a stretch of tokens, so that a sequence's loads are fetched once for all of it.
template <int NV>
__global__ __launch_bounds__(64 * kWaves) void route_backward_kernel(BalanceArgs a, uint32_t each) {
    __shared__ float picks[kWaves][64 * NV];  // a token's gradients of its picks' logits, zeros between tokens
    const uint32_t lane = threadIdx.x & 63, n = a.n_experts, k = a.top_k;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint64_t first = ((uint64_t)blockIdx.x * kWaves + wave) * each;
    if (first >= a.m) return;
    const uint32_t from = (uint32_t)first, to = (uint32_t)min(first + each, (uint64_t)a.m);
    uint32_t q = a.seq_offsets ? seq_of(a, from) : 0;
    uint32_t begin, end;
    seq_range(a, q, begin, end);
    const float d_loss = a.d_loss ? *a.d_loss : 0.0f;
    float* mine = picks[wave];
#pragma unroll
    for (int v = 0; v < NV; ++v) mine[v * 64 + lane] = 0.0f;
    // the loads' distances from 1: p adds up to 1, so that load - sum load * p is the same of them, and of nearly even
    // loads nothing cancels (even ones have exactly no gradient)
    float load[NV], w = 0.0f;
    auto fetch = [&] {
        const uint32_t tokens = end - begin;
        const double share = tokens ? 1.0 / (double)tokens : 0.0;
        w = (float)((double)d_loss * (a.coefficient / (double)a.n_seqs) * share);
        const double even = (double)k * (double)tokens, per = share / (double)k;  // even picks are even / n
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t e = Experts<NV>::of(v);
            load[v] = e < n ? (float)(((double)a.counts[(size_t)q * n + e] * (double)n - even) * per) : 0.0f;
        }
    };
    fetch();
    // the next token is requested while this one is worked on, of up to 512 experts (more fill the registers)
    constexpr bool AHEAD = NV <= 8;
    float next[NV], next_dg = 0.0f, next_logit = 0.0f;
    uint32_t next_id = 0xffffffffu;
    auto request = [&](uint32_t t) {
        Experts<NV>::load(a.logits + (size_t)t * n, n, next);
        if (a.d_gates && lane < k) {
            next_id = a.ids[(size_t)t * k + lane];
            next_dg = a.d_gates[(size_t)t * k + lane];
        }
    };
    if (AHEAD) request(from);
    for (uint32_t t = from; t < to; ++t) {
        if (!AHEAD) request(t);
        if (t >= end && q + 1 < a.n_seqs) {
            do {
                ++q;
                seq_range(a, q, begin, end);
            } while (t >= end && q + 1 < a.n_seqs);
            fetch();
        }
        float d[NV], l[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) l[v] = next[v];
        const uint32_t id = next_id;
        float dg = next_dg, picked = 0.0f;
        if (a.d_gates && id < n) next_logit = a.logits[(size_t)t * n + id];
        if (AHEAD && t + 1 < to) request(t + 1);
        if (t < begin || t >= end) {  // no sequence's
#pragma unroll
            for (int v = 0; v < NV; ++v) d[v] = 0.0f;
            Experts<NV>::store(a.d_logits + (size_t)t * n, n, d);
            continue;
        }
        float s[NV], slope[NV], by = 0.0f;  // by: what the pick's gradient comes to its logit with
        if (id < n) score(next_logit, picked, by);
        else dg = 0.0f;
        const float r = scores<NV>(l, n, s, slope);
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) dot += load[v] * s[v];
        dot = wave_sum_f(dot) * r;
#pragma unroll
        for (int v = 0; v < NV; ++v) d[v] = w * (load[v] - dot) * r * slope[v];
        if (a.d_gates) {
            if (a.renormalize) {
                const float of = wave_sum_f(picked);
                float gate = 0.0f;
                if (!(of < kTiny)) {
                    gate = __fdiv_rn(picked, of);
                    by *= __builtin_amdgcn_rcpf(of);
                } else {
                    const float most = wave_max_f(id < n ? next_logit : -__builtin_inff());
                    if (most > kNoScore) {
                        const float p = id < n ? score_beside(next_logit, most) : 0.0f;
                        gate = __fdiv_rn(p, wave_sum_f(p));
                    }
                    by = gate;
                }
                // by the differences from the gate that has most of the weight, if one has: its own gradient is small
                // beside d_gates, and the difference that leaves it would cancel
                if (const uint64_t large = __ballot(gate > 0.5f)) dg -= lane_f(dg, __builtin_ctzll(large));
                dg -= wave_sum_f(dg * gate);
            }
            // the wavefront's own LDS row, in program order: no barrier
            if (id < n) atomicAdd(&mine[id], dg * by);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int v = 0; v < NV; ++v) d[v] += mine[Experts<NV>::of(v)];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (id < n) mine[id] = 0.0f;
        }
        Experts<NV>::store(a.d_logits + (size_t)t * n, n, d);
    }
}

uint32_t finish_groups(const eidm_balance_shape* s) { return s->n_seqs >= 16 ? 4 : 16; }
uint32_t expert_tiles(const eidm_balance_shape* s) {
    const uint32_t tile = kFinish / finish_groups(s);
    return (s->n_experts + tile - 1) / tile;
}

// Tokens of a part: as few as still leave parts whose rows of counts and sums
// are a small share of the logits, and no more parts than fill the device.
uint32_t balance_each(uint32_t m) {
    const uint32_t most = 1024, each = (m + most - 1) / most;
    return each < 16 ? 16 : each;
}

struct BalancePlan {
    uint64_t counts = 0, probs = 0, loss = 0, ticket = 0, total = 0;
    uint32_t each = 0, parts = 0;
};

int check_balance(const eidm_balance_shape* s, BalancePlan* p) {
    if (!s) return api_fail(EIDM_E_INVALID, "shape is NULL");
    if (s->struct_size != sizeof(eidm_balance_shape))
        return api_fail(EIDM_E_INVALID, "shape.struct_size is %u, expected %zu", s->struct_size, sizeof(eidm_balance_shape));
    if (!s->m || !s->n_experts || !s->top_k || !s->n_seqs)
        return api_fail(EIDM_E_INVALID, "zero dimension (m=%u n_experts=%u top_k=%u n_seqs=%u)", s->m, s->n_experts,
                        s->top_k, s->n_seqs);
    if (s->n_experts > kMaxExperts || s->top_k > kMaxRouterTopK)
        return api_fail(EIDM_E_UNSUPPORTED, "n_experts <= %u and top_k <= %u are taken", kMaxExperts, kMaxRouterTopK);
    if ((uint64_t)s->m * s->top_k > kIndex31 || s->n_seqs > EIDM_BALANCE_MAX_SEQS)
        return api_fail(EIDM_E_UNSUPPORTED, "m*top_k below 2^31 and n_seqs <= %u are taken", EIDM_BALANCE_MAX_SEQS);
    if (!std::isfinite(s->coefficient)) return api_fail(EIDM_E_INVALID, "the coefficient must be finite");
    p->each = balance_each(s->m);
    p->parts = (s->m + p->each - 1) / p->each;
    const uint64_t rows = ((uint64_t)p->parts + s->n_seqs) * s->n_experts * 4;
    p->probs = round256(rows);
    p->loss = p->probs + round256(rows);
    p->ticket = p->loss + round256((uint64_t)s->n_seqs * expert_tiles(s) * 8);
    p->total = p->ticket + 256;
    return EIDM_OK;
}

template <typename Go>
hipError_t by_width(uint32_t n_experts, Go go) {
    const uint32_t nv = (n_experts + 63) / 64;
    if (nv <= 1) return go(std::integral_constant<int, 1>{});
    if (nv <= 2) return go(std::integral_constant<int, 2>{});
    if (nv <= 4) return go(std::integral_constant<int, 4>{});
    if (nv <= 8) return go(std::integral_constant<int, 8>{});
    if (nv <= 16) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
}

}  // namespace
}  // namespace eidm

extern "C" {

using namespace eidm;

uint64_t eidm_route_balance_scratch_bytes(const eidm_balance_shape* shape) {
    BalancePlan p;
    if (check_balance(shape, &p) != EIDM_OK) return 0;
    api_ok();
    return p.total;
}

int eidm_route_balance(const eidm_balance_shape* shape, const float* logits, const uint32_t* ids,
                       const uint32_t* seq_offsets, uint32_t* counts, float* mean_probs, float* loss, void* scratch,
                       uint64_t scratch_bytes, void* stream) {
    ReceiptScope receipt;
    BalancePlan p;
    const int rc = check_balance(shape, &p);
    if (rc) return rc;
    if (!logits || !ids || !counts || !mean_probs || !loss) return api_fail(EIDM_E_INVALID, "a buffer is NULL");
    if (!seq_offsets && shape->n_seqs != 1) return api_fail(EIDM_E_INVALID, "%u sequences need offsets", shape->n_seqs);
    if (!is_aligned(logits, 4) || !is_aligned(ids, 4) || !is_aligned(seq_offsets, 4) || !is_aligned(counts, 4) ||
        !is_aligned(mean_probs, 4) || !is_aligned(loss, 4))
        return api_fail(EIDM_E_ALIGN, "buffers must be 4-byte aligned");
    if (!scratch || scratch_bytes < p.total)
        return api_fail(EIDM_E_SIZE, "the balance needs %llu bytes of scratch, got %llu", (unsigned long long)p.total,
                        (unsigned long long)(scratch ? scratch_bytes : 0));
    if (!is_aligned(scratch, 256)) return api_fail(EIDM_E_ALIGN, "scratch must be 256-byte aligned");
    uint8_t* at = static_cast<uint8_t*>(scratch);
    BalanceArgs a{};
    a.m = shape->m;
    a.n_experts = shape->n_experts;
    a.top_k = shape->top_k;
    a.n_seqs = shape->n_seqs;
    a.each = p.each;
    a.coefficient = (double)shape->coefficient;
    a.logits = logits;
    a.ids = ids;
    a.seq_offsets = seq_offsets;
    a.counts = counts;
    a.mean_probs = mean_probs;
    a.loss = loss;
    a.part_counts = reinterpret_cast<uint32_t*>(at);
    a.part_probs = reinterpret_cast<float*>(at + p.probs);
    a.part_loss = reinterpret_cast<double*>(at + p.loss);
    a.ticket = reinterpret_cast<uint32_t*>(at + p.ticket);
    hipStream_t st = static_cast<hipStream_t>(stream);
    const uint32_t waves = a.n_experts <= 1024 ? kPartWaves : kPartWaves / 2;
    const uint32_t grid = p.parts, lds = (1 + waves) * a.n_experts * 4;
    hipError_t err = by_width(a.n_experts, [&](auto width) {
        hipLaunchKernelGGL((balance_part_kernel<decltype(width)::value>), dim3(grid), dim3(64 * waves), lds, st, a);
        return launched(EIDM_KERNEL_BALANCE_PART, grid, 64 * waves, lds);
    });
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "balance launch: %s", hipGetErrorString(err));
    const uint32_t tiles = expert_tiles(shape);
    const dim3 finish(tiles, a.n_seqs);
    if (finish_groups(shape) == 16) hipLaunchKernelGGL(balance_finish_kernel<16>, finish, dim3(kFinish), 0, st, a);
    else hipLaunchKernelGGL(balance_finish_kernel<4>, finish, dim3(kFinish), 0, st, a);
    err = launched(EIDM_KERNEL_BALANCE_FINISH, tiles * a.n_seqs, kFinish, 0);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "balance launch: %s", hipGetErrorString(err));
    return api_ok();
}

int eidm_route_backward(const eidm_balance_shape* shape, const float* logits, const uint32_t* ids,
                        const uint32_t* seq_offsets, const uint32_t* counts, const float* d_gates, int renormalize,
                        const float* d_loss, float* d_logits, void* stream) {
    ReceiptScope receipt;
    BalancePlan p;
    const int rc = check_balance(shape, &p);
    if (rc) return rc;
    if (!logits || !ids || !counts || !d_logits) return api_fail(EIDM_E_INVALID, "a buffer is NULL");
    if (!d_gates && !d_loss) return api_fail(EIDM_E_INVALID, "no gradient is given");
    if (!seq_offsets && shape->n_seqs != 1) return api_fail(EIDM_E_INVALID, "%u sequences need offsets", shape->n_seqs);
    if (!is_aligned(logits, 4) || !is_aligned(ids, 4) || !is_aligned(seq_offsets, 4) || !is_aligned(counts, 4) ||
        !is_aligned(d_gates, 4) || !is_aligned(d_loss, 4) || !is_aligned(d_logits, 4))
        return api_fail(EIDM_E_ALIGN, "buffers must be 4-byte aligned");
    BalanceArgs a{};
    a.m = shape->m;
    a.n_experts = shape->n_experts;
    a.top_k = shape->top_k;
    a.n_seqs = shape->n_seqs;
    a.coefficient = (double)shape->coefficient;
    a.logits = logits;
    a.ids = ids;
    a.seq_offsets = seq_offsets;
    a.counts = const_cast<uint32_t*>(counts);
    a.renormalize = renormalize;
    a.d_gates = d_gates;
    a.d_loss = d_loss;
    a.d_logits = d_logits;
    // stretches of up to 16 tokens, shorter while the device is not full (8 wavefronts a SIMD), longer
    // where the launch would have 2^32 threads
    const uint64_t fill = (uint64_t)device_cus() * 32, most = (1ull << 32) / 64 - kWaves;
    uint64_t each = (a.m + fill - 1) / fill;
    if (each > 16) each = 16;
    if ((a.m + each - 1) / each > most) each = (a.m + most - 1) / most;
    const uint64_t waves = (a.m + each - 1) / each, grid = (waves + kWaves - 1) / kWaves;
    const hipError_t err = by_width(a.n_experts, [&](auto width) {
        hipLaunchKernelGGL((route_backward_kernel<decltype(width)::value>), dim3((uint32_t)grid), dim3(64 * kWaves), 0,
                           static_cast<hipStream_t>(stream), a, (uint32_t)each);
        return launched(EIDM_KERNEL_ROUTE_BACKWARD, (uint32_t)grid, 64 * kWaves, 0);
    });
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "router gradient launch: %s", hipGetErrorString(err));
    return api_ok();
}

}  // extern "C"
