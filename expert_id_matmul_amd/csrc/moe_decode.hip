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
// chose it (up to 16 rows at a time); one token, and tokens that would read
// little again, run each by itself (each_token() below).
//
// What bounds it is the experts' bytes.  Measured (bf16, top 8): one token of
// 2048 x 768, gate/up 50 MB in 11.3 us and down 25 MB in 7.4 (a launch's start,
// the router's inputs and the last block's end, some 4 us, weigh as much as
// the stream); of 4096 x 1536, 201 MB in 31.8 us (6.3 TB/s) and 101 MB in 19.0
// (5.3); 8 tokens of 2048 x 768, about 325 MB in 60 us (5.4) and 162 MB in 36
// (4.5); 64 tokens with popular experts, 618 MB in 134 us (4.6) and 311 MB in
// 85 (3.7), the matrix core busy 27 % and 21 % of the time and wavefronts
// waiting 33 % and 43 % of theirs: neither the stream nor the products alone.
//
// Every product is in the library's fixed reduction order, routing, silu and
// the combine are the same operations as the separate kernels', so the
// results are bit for bit those of eidm_moe_ffn.
//
// cortiq-engine 0.7.7, src/mimo_moe.rs, Dynamic::run (route, one FFN per
// pick, weighted sum); hf2q dense_ffn_arena.rs, MoeFfnArena (gate, up, h, y).
#include <atomic>
#include <cmath>

#include "eidm_device.hpp"
#include "eidm_internal.hpp"
#include "few_map.hpp"
#include "few_rows.hpp"
#include "route_wave.hpp"

namespace eidm {
namespace {

constexpr int kWaves = 8;  // wavefronts per block of the many-token kernels
// LDS for staged activation rows: 16 rows of 2048, one of the longest k
// (kMaxDecodeRow)
constexpr uint32_t kRowBytes = 16 * few_row_floats(2048) * 4;
static_assert(few_row_floats(kMaxDecodeRow) * 4 <= kRowBytes);
static_assert(kMaxDecodeTokens * kMaxDecodeTopK <= kFewMapRows * 64 * kWaves);
static_assert(few_map_words(kMaxDecodeTokens * kMaxDecodeTopK, kMaxExperts) <= kFewMapUnits * 4 * 64 * kWaves);
constexpr uint32_t kRouteExperts = 256;  // experts a block routes itself (4 per lane)

// most rows of k elements staged at once
__host__ __device__ constexpr uint32_t row_cap(uint32_t k) { return kRowBytes / (few_row_floats(k) * 4); }

// Rounds in flight: `loads` 16-byte loads per lane (C weight rows per lane;
// one load each for 16-bit weights, two for f32).
template <int DT, int C>
constexpr int few_depth(int loads) {
    return 2 * loads / (C * DtypeSize<DT>::value);
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// ------------------------------------------------------- one token by itself
// A wavefront per slot; a block owns `cols` <= 4 columns of one token's h for
// every slot (so all compute units have the same share of each expert).
// Routing as in the fused decode step (moe_direct.hip): each expert's sigmoid
// by one thread, every wavefront runs the selection up to its own pick, the
// last one forms the gates.
template <int DT, int NV, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void gate_up_one_kernel(MoeDecodeArgs a, uint32_t cols, uint32_t blocks) {
    constexpr int S = DtypeSize<DT>::value;
    extern __shared__ __align__(16) float xs[];
    __shared__ float rs_s[64 * NV];
    __shared__ uint32_t rs_code[64 * NV];
    const uint32_t lane = threadIdx.x & 63, slot = threadIdx.x >> 6, q = lane & 3;
    const uint32_t token = blockIdx.x / blocks, block = blockIdx.x % blocks;
    RouteInputs<NV> rin;
    route_inputs_issue<NV>(a.logits + (size_t)token * a.n_experts, a.bias, a.n_experts, rin);
    __builtin_amdgcn_sched_barrier(0);  // the row's loads queue behind the router's
    auto stage = few_stage<8>(xs, 1, a.hidden, [&](uint32_t) { return a.x + (size_t)token * a.hidden; });
    stage.issue();
    __builtin_amdgcn_sched_barrier(0);
    route_inputs_score<NV>(rin, a.n_experts, rs_s, rs_code);
    stage.finish();
    __syncthreads();

    RouteScores<NV> sc;
    route_scores_lds<NV>(rs_s, rs_code, sc);
    uint32_t pick;
    float score;
    const float sum = route_select<NV>(sc, slot + 1, pick, score);
    if (block == 0 && slot == a.top_k - 1 && lane < a.top_k) {
        a.ids[token * a.top_k + lane] = pick;
        a.gates[token * a.top_k + lane] = a.renormalize ? __fdiv_rn(score, sum) : score;
    }
    const uint32_t e = (uint32_t)__builtin_amdgcn_readlane((int)pick, (int)slot);
    const uint32_t col0 = block * cols, end = min(col0 + cols, a.inter);
    const uint32_t col = col0 + q;
    const size_t at = (size_t)e * a.gate_up_stride + (size_t)(col < end ? col : col0) * a.hidden * S;
    const uint8_t* const wrow[2] = {a.w_gate + at, a.w_up + at};
    FewStream<DT, 2, few_depth<DT, 2>(MAXW > 8 ? 12 : 16), true> w;
    w.start(wrow, (int)a.hidden);
    few_rows_tile<0, false>(w, wrow, wrow, xs, 0, 1, (int)a.hidden, [](uint32_t) { return 0u; },
                            [&](uint32_t, const float (&t)[2]) {
                                if (col < end) a.h[(size_t)(token * a.top_k + slot) * a.inter + col] = silu_mul(t[0], t[1]);
                            });
}

// A wavefront per slot; a block owns `cols` <= 4*C output columns of a token,
// so the sum over the slots needs no second launch (a combine of its own costs
// 4.7 us).
template <int DT, int C, int LOADS, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void down_one_kernel(MoeDecodeArgs a, uint32_t cols, uint32_t blocks) {
    constexpr int S = DtypeSize<DT>::value;
    extern __shared__ __align__(16) float xs[];
    __shared__ float ys[MAXW][4 * C];
    const uint32_t lane = threadIdx.x & 63, slot = threadIdx.x >> 6, q = lane & 3;
    const uint32_t token = blockIdx.x / blocks, first = token * a.top_k;  // its first routed row
    const uint32_t e = uniform(a.ids[first + slot]);
    auto stage = few_stage<8>(xs, a.top_k, a.inter, [&](uint32_t r) { return a.h + (size_t)(first + r) * a.inter; });
    stage.issue();
    const uint32_t col0 = blockIdx.x % blocks * cols, end = min(col0 + cols, a.hidden);
    const uint8_t* wrow[C];
#pragma unroll
    for (uint32_t c = 0; c < C; ++c) {
        const uint32_t col = col0 + 4 * c + q;
        wrow[c] = a.w_down + (size_t)e * a.down_stride + (size_t)(col < end ? col : col0) * a.inter * S;
    }
    FewStream<DT, C, few_depth<DT, C>(LOADS), true> w;
    w.start(wrow, (int)a.inter);
    stage.finish();
    __syncthreads();
    few_rows_tile<0, false>(w, wrow, wrow, xs, few_row_floats(a.inter), 1, (int)a.inter, [&](uint32_t) { return slot; },
                            [&](uint32_t, const float (&t)[C]) {
#pragma unroll
                                for (int c = 0; c < C; ++c) ys[slot][4 * c + q] = t[c];
                            });
    __syncthreads();
    if (slot == 0 && col0 + lane < end) {
        float acc = 0.0f;
        for (uint32_t s = 0; s < a.top_k; ++s) acc = __builtin_fmaf(a.gates[first + s], ys[s][lane], acc);
        a.out[(size_t)token * a.hidden + col0 + lane] = acc;
    }
}

// --------------------------------------------------------- several tokens
// Relative time of one column-group job for an expert of `rows` rows, `most`
// of which are staged at once: the weights' stream alone for up to 4 rows,
// the products beyond (measured at 16 rounds of k: 1, 2-4, 5-8 and 9-16 rows).
__device__ __forceinline__ uint32_t job_cost(uint32_t rows, uint32_t most) {
    auto pass = [](uint32_t r) { return r == 0 ? 0u : r <= 4 ? 8u : r <= 8 ? 10u : 15u; };
    most = min(most, (uint32_t)kFewRows);
    return rows / most * pass(most) + pass(rows % most);
}

// Column-group jobs (expert u, group g) of all touched experts in order, cut
// into one contiguous range of equal cost per block, so that a block meets
// one or two experts; its wavefronts take the range's jobs in turn, each
// requesting its next job's weights while the last rounds of one run.
// Rows: when `staged`, every row already stands in LDS, at lds_of(routed
// row); else the block stages its experts' rows, in passes when they do not
// fit.  row_of(routed row): the activation row of k elements.
// weight_of(expert, group, wrow): this lane's weight rows.
// emit(routed row, group, totals).
template <int DT, int C, int D, typename RowOf, typename LdsOf, typename WeightOf, typename Emit>
__device__ __forceinline__ void expert_major(const FewMap& map, float* xs, bool staged, uint32_t groups, uint32_t k,
                                             RowOf row_of, LdsOf lds_of, WeightOf weight_of, Emit emit) {
    const uint32_t stride = few_row_floats(k);
    const uint32_t most = row_cap(k);
    const uint32_t per_expert = min(most, (uint32_t)kFewRows);
    const uint32_t cost = map.cost[*map.used] * groups, share = cost / gridDim.x, over = cost % gridDim.x;
    uint32_t pos = few_map_job(map, groups, share * blockIdx.x + min(blockIdx.x, over));
    const uint32_t last = few_map_job(map, groups, share * (blockIdx.x + 1) + min(blockIdx.x + 1, over));
    pos = uniform(pos);
    while (pos < last) {  // block-uniform
        uint32_t v = pos / groups;  // experts pos/groups .. v in this pass
        const uint32_t first = map.off[v];
        uint32_t end = map.off[v + 1];
        uint32_t passes = 1;
        if (staged) {
            v = (last - 1) / groups;
            end = map.off[v + 1];
        } else if (end - first > per_expert) {
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
            FewStream<DT, C, D, true> w;
            const uint8_t* wrow[C];
            auto weights_at = [&](uint32_t job, const uint8_t* (&to)[C]) {
                const uint32_t u = uniform(job / groups);
                weight_of(uniform(map.id[u]), uniform(job) - u * groups, to);
            };
            uint32_t job = pos + (threadIdx.x >> 6);
            auto stage = few_stage<8>(xs, staged ? 0 : limit - base, k,
                                      [&](uint32_t i) { return row_of(map.row[base + i]); });
            stage.issue();  // ahead of the weights: a thread's loads return in order
            // in every wavefront: behind a branch, the rows' wait would be for the weights too
            weights_at(min(job, stop - 1), wrow);
            w.start(wrow, (int)k);
            if (!staged) {
                __syncthreads();  // the rows of the pass before are done with
                stage.finish();
                __syncthreads();
            }
            while (job < stop) {  // wave-uniform
                const uint32_t u = uniform(job / groups), g = uniform(job) - u * groups;
                const uint32_t to = min(uniform(map.off[u + 1]), limit);
                for (uint32_t at = max(uniform(map.off[u]), base); at < to; at += kFewRows) {
                    // (one turn unless an expert's staged rows exceed 16)
                    const bool again = at + kFewRows < to;
                    const uint32_t count = min(to - at, (uint32_t)kFewRows);
                    auto lds_row = [&](uint32_t i) { return staged ? lds_of(map.row[at + i]) : at + i - base; };
                    auto emit_at = [&](uint32_t i, const float (&t)[C]) { emit(map.row[at + i], g, t); };
                    const uint8_t* next[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) next[c] = wrow[c];
                    if (again || job + kWaves < stop) {
                        if (!again) weights_at(job + kWaves, next);
                        few_rows_any<true>(w, wrow, next, xs, stride, count, (int)k, lds_row, emit_at);
#pragma unroll
                        for (int c = 0; c < C; ++c) wrow[c] = next[c];
                    } else {
                        few_rows_any<false>(w, wrow, next, xs, stride, count, (int)k, lds_row, emit_at);
                    }
                }
                job += kWaves;
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
    __shared__ uint32_t picks[ROUTE ? kWaves * kMaxDecodeTopK : 1];
    const uint32_t rows = a.m * a.top_k;
    const FewMap map = few_map_at(lds, rows, a.n_experts);
    float* xs = reinterpret_cast<float*>(lds + few_map_words(rows, a.n_experts));
    const bool staged = a.m <= row_cap(a.hidden);  // every token's row fits
    auto stage = few_stage<8>(xs, staged ? a.m : 0, a.hidden, [&](uint32_t t) { return a.x + (size_t)t * a.hidden; });
    FewIds ids;
    if constexpr (ROUTE) {
        const uint32_t t = threadIdx.x >> 6, lane = threadIdx.x & 63;
        RouteScores<kRouteExperts / 64> sc;
        if (t < a.m) route_scores<kRouteExperts / 64>(a.logits + (size_t)t * a.n_experts, a.bias, a.n_experts, sc);
        stage.issue();
        if (t < a.m) {
            uint32_t id;
            float score;
            const float sum = route_select<kRouteExperts / 64>(sc, a.top_k, id, score);
            if (lane < a.top_k) {
                picks[t * a.top_k + lane] = id;
                if (blockIdx.x == 0) {
                    a.ids[t * a.top_k + lane] = id;
                    a.gates[t * a.top_k + lane] = a.renormalize ? __fdiv_rn(score, sum) : score;
                }
            }
        }
        __syncthreads();
        ids = few_map_ids_load(picks, rows);
    } else {
        ids = few_map_ids_load(a.ids, rows);
        stage.issue();
    }
    const uint32_t most = row_cap(a.hidden);
    few_map_build(map, ids, rows, a.n_experts, [&](uint32_t r) { return job_cost(r, most); });
    if (blockIdx.x == 0) few_map_save(lds, few_map_words(rows, a.n_experts), a.map);
    stage.finish();
    __syncthreads();

    const uint32_t q = threadIdx.x & 3;
    expert_major<DT, 2, few_depth<DT, 2>(12)>(
        map, xs, staged, (a.inter + 3) / 4, a.hidden, [&](uint32_t r) { return a.x + (size_t)(r / a.top_k) * a.hidden; },
        [&](uint32_t r) { return r / a.top_k; },
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
template <int DT, int C, int LOADS>
__global__ __launch_bounds__(64 * kWaves) void down_kernel(MoeDecodeArgs a) {
    constexpr int S = DtypeSize<DT>::value;
    extern __shared__ __align__(16) uint32_t lds[];
    const uint32_t rows = a.m * a.top_k;
    const FewMap map = few_map_at(lds, rows, a.n_experts);
    float* xs = reinterpret_cast<float*>(lds + few_map_words(rows, a.n_experts));
    FewMapCopy copy;  // (an expert's rows cost alike in both products but for the rows that fit in LDS)
    copy.load(a.map, few_map_words(rows, a.n_experts));
    copy.store(lds, few_map_words(rows, a.n_experts));
    __syncthreads();
    const uint32_t q = threadIdx.x & 3;
    expert_major<DT, C, few_depth<DT, C>(LOADS)>(
        map, xs, false, (a.hidden + 4 * C - 1) / (4 * C), a.inter,
        [&](uint32_t r) { return a.h + (size_t)r * a.inter; }, [](uint32_t) { return 0u; },
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
// every token, its wavefronts take the touched experts in turn.  At 65 rows of
// 363 (f32, 31 experts, 45 MB) 32 us: 13 for the map and the staged rows, which
// every block reads (24 MB in all), 14 for the products, four short streams a
// wavefront.
template <int DT, int C, int LOADS>
__global__ __launch_bounds__(64 * kWaves) void down_combine_kernel(MoeDecodeArgs a, uint32_t cols) {
    constexpr int S = DtypeSize<DT>::value;
    extern __shared__ __align__(16) uint32_t lds[];
    const uint32_t rows = a.m * a.top_k;
    const FewMap map = few_map_at(lds, rows, a.n_experts);
    float* ys = reinterpret_cast<float*>(lds + few_map_words(rows, a.n_experts));  // [rows][4*C]
    float* xs = ys + rows * 4 * C;
    auto stage = few_stage<8>(xs, rows, a.inter, [&](uint32_t r) { return a.h + (size_t)r * a.inter; });
    FewMapCopy copy;
    copy.load(a.map, few_map_words(rows, a.n_experts));
    stage.issue();
    copy.store(lds, few_map_words(rows, a.n_experts));
    __syncthreads();

    const uint32_t q = threadIdx.x & 3;
    const uint32_t col0 = blockIdx.x * cols, end = min(col0 + cols, a.hidden);
    const uint32_t used = *map.used;
    auto weights_at = [&](uint32_t u, const uint8_t* (&to)[C]) {
#pragma unroll
        for (uint32_t c = 0; c < C; ++c) {
            const uint32_t col = col0 + 4 * c + q;
            to[c] = a.w_down + (size_t)uniform(map.id[u]) * a.down_stride + (size_t)(col < end ? col : col0) * a.inter * S;
        }
    };
    FewStream<DT, C, few_depth<DT, C>(LOADS), true> w;
    const uint8_t* wrow[C];
    uint32_t u = uniform(threadIdx.x >> 6);
    weights_at(min(u, used - 1), wrow);
    w.start(wrow, (int)a.inter);
    stage.finish();
    __syncthreads();
    for (; u < used; u += kWaves) {
        const uint32_t to = uniform(map.off[u + 1]);
        for (uint32_t at = uniform(map.off[u]); at < to; at += kFewRows) {
            const bool again = at + kFewRows < to;
            const uint32_t count = min(to - at, (uint32_t)kFewRows), stride = few_row_floats(a.inter);
            auto lds_row = [&](uint32_t i) { return map.row[at + i]; };
            auto emit = [&](uint32_t i, const float (&t)[C]) {
#pragma unroll
                for (int c = 0; c < C; ++c) ys[map.row[at + i] * (4 * C) + 4 * c + q] = t[c];
            };
            const uint8_t* next[C];
#pragma unroll
            for (int c = 0; c < C; ++c) next[c] = wrow[c];
            if (again || u + kWaves < used) {
                if (!again) weights_at(u + kWaves, next);
                few_rows_any<true>(w, wrow, next, xs, stride, count, (int)a.inter, lds_row, emit);
#pragma unroll
                for (int c = 0; c < C; ++c) wrow[c] = next[c];
            } else {
                few_rows_any<false>(w, wrow, next, xs, stride, count, (int)a.inter, lds_row, emit);
            }
        }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < a.m * 4 * C; i += blockDim.x) {
        const uint32_t t = i / (4 * C), c = i % (4 * C);
        if (col0 + c < end) {
            float acc = 0.0f;
            for (uint32_t s = 0; s < a.top_k; ++s) {
                const uint32_t r = t * a.top_k + s;
                acc = __builtin_fmaf(a.gates[r], ys[r * (4 * C) + c], acc);
            }
            a.out[(size_t)t * a.hidden + col0 + c] = acc;
        }
    }
}

// ---------------------------------------------------------------- launches
// Allows a kernel as much dynamic LDS as its static LDS leaves of a compute
// unit's (the runtime refuses more), once per device.
constexpr uint32_t kUnitLds = 160 * 1024;
hipError_t allow_lds(const void* kernel, std::atomic<uint64_t>& done) {
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    hipFuncAttributes of{};
    err = hipFuncGetAttributes(&of, kernel);
    if (err == hipSuccess)
        err = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)(kUnitLds - of.sharedSizeBytes));
    if (err == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    else (void)hipGetLastError();  // reported here, not by the caller's next HIP call
    return err;
}

template <auto Kernel, typename... Args>
hipError_t launch_one(int receipt, uint32_t grid, uint32_t threads, uint32_t lds, hipStream_t stream, Args... args) {
    if (lds > 48 * 1024) {
        static std::atomic<uint64_t> done{0};
        const hipError_t err = allow_lds(reinterpret_cast<const void*>(Kernel), done);
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(Kernel, dim3(grid), dim3(threads), lds, stream, args...);
    return launched(receipt, grid, threads, lds);
}

// Columns per block in [most/2, most]: the width whose blocks, spread over
// the compute units, give the busiest one the fewest columns; the widest on
// ties.
uint32_t block_columns(uint32_t n, uint32_t most, uint32_t cus) {
    uint32_t best = most;
    uint64_t least = ~0ull;
    for (uint32_t c = most; c >= (most + 1) / 2; --c) {
        const uint64_t blocks = (n + c - 1) / c, cost = (blocks + cus - 1) / cus * c;
        if (cost < least) {
            least = cost;
            best = c;
        }
    }
    return best;
}

// 12 loads in flight where they hold the whole product, or cut it into whole
// rings where 16 do not; else 16.
bool twelve_loads(int dtype, uint32_t k, uint32_t weight_rows) {
    const uint32_t rounds = k / kRoundK, per = weight_rows * (dtype == kDtypeF32 ? 2 : 1);
    return rounds <= 12 / per || (rounds % (16 / per) && rounds % (12 / per) == 0);
}

template <int DT>
hipError_t launch_each_token(const MoeDecodeArgs& a, uint32_t cus, hipStream_t stream) {
    const uint32_t threads = 64 * a.top_k;
    const uint32_t up = block_columns(a.inter, 4, cus), down = block_columns(a.hidden, 8, cus);
    const uint32_t ub = (a.inter + up - 1) / up, db = (a.hidden + down - 1) / down;  // blocks per token
    const uint32_t up_lds = few_row_floats(a.hidden) * 4, down_lds = a.top_k * few_row_floats(a.inter) * 4;
    constexpr int U = EIDM_KERNEL_DECODE_GATE_UP_ONE, W = EIDM_KERNEL_DECODE_DOWN_ONE;
    const bool wide = a.top_k > 8;
    hipError_t err;
    if (a.n_experts <= 256)
        err = wide ? launch_one<gate_up_one_kernel<DT, 4, 16>>(U, ub * a.m, threads, up_lds, stream, a, up, ub)
                   : launch_one<gate_up_one_kernel<DT, 4, 8>>(U, ub * a.m, threads, up_lds, stream, a, up, ub);
    else
        err = wide ? launch_one<gate_up_one_kernel<DT, 32, 16>>(U, ub * a.m, threads, up_lds, stream, a, up, ub)
                   : launch_one<gate_up_one_kernel<DT, 32, 8>>(U, ub * a.m, threads, up_lds, stream, a, up, ub);
    if (err != hipSuccess) return err;
    if (wide) return launch_one<down_one_kernel<DT, 2, 12, 16>>(W, db * a.m, threads, down_lds, stream, a, down, db);
    if (down <= 4) return launch_one<down_one_kernel<DT, 1, 12, 8>>(W, db * a.m, threads, down_lds, stream, a, down, db);
    return twelve_loads(DT, a.inter, 2)
               ? launch_one<down_one_kernel<DT, 2, 12, 8>>(W, db * a.m, threads, down_lds, stream, a, down, db)
               : launch_one<down_one_kernel<DT, 2, 16, 8>>(W, db * a.m, threads, down_lds, stream, a, down, db);
}

// Each token by itself when it is the only one, or when what that repeats costs
// less than the map and the passes of the several-token form, which weigh as
// 100 MB of weights: the shared experts' bytes, and their blocks (a turn of the
// device's, 16 wavefronts a compute unit, as 5 MB); above kRouteExperts also
// the routing that every block does, 40 MB a turn. There are no ids to go by:
// picks are counted as evenly spread.
// Over 340 layers (2-64 tokens, 4-2048 experts, 1-12 slots, rows of 16-24000,
// spread and popular picks) the chosen form takes 4 % more than the better one
// on average and at most twice as long (4 tokens with the same 8 of 128 experts
// of 232 x 3856: 90 us, together 45). One by one : together, us, bf16, top 8:
// 128 experts of 2048 x 768, 2 tokens 29 : 38 (the same picks 27 : 29), 4 tokens
// 53 : 64 (50 : 30), 8 tokens 103 : 102; 128 of 256 x 128, 16 tokens 29 : 48, 64
// tokens 99 : 39; 2048 of 256 x 128, 16 tokens 50 : 85, 32 tokens 94 : 66.
bool each_token(const MoeDecodeArgs& a, uint32_t cus) {
    if (a.top_k > row_cap(a.inter)) return false;
    if (a.m == 1) return true;
    const double e = a.n_experts, rows = (double)a.m * a.top_k;
    const double again = rows - e * (1.0 - std::pow(1.0 - a.top_k / e, (double)a.m));  // rows whose expert is read before
    const double expert = 3.0 * a.hidden * a.inter * (a.dtype == kDtypeF32 ? 4 : 2);
    const uint32_t up = block_columns(a.inter, 4, cus), down = block_columns(a.hidden, 8, cus);
    const uint32_t ub = (a.inter + up - 1) / up, db = (a.hidden + down - 1) / down;  // wavefronts per row
    const double turn = 16.0 * cus;
    double cost = again * (expert + 5e6 * (ub + db) / turn);
    if (a.n_experts > kRouteExperts) cost += 40e6 * rows * ub / turn;
    return cost < 100e6;
}

template <int DT>
hipError_t launch_dt(const MoeDecodeArgs& a, int device_cus, hipStream_t stream) {
    const uint32_t cus = device_cus > 0 ? (uint32_t)device_cus : 256;
    const uint32_t rows = a.m * a.top_k;
    if (each_token(a, cus)) return launch_each_token<DT>(a, cus, stream);
    const uint32_t touched = few_map_ids(rows, a.n_experts);  // at most
    const uint32_t map_bytes = few_map_words(rows, a.n_experts) * 4;
    auto blocks_of = [&](uint32_t groups) {
        const uint64_t jobs = (uint64_t)touched * groups;
        return (uint32_t)(jobs < cus ? jobs : cus);
    };
    auto staged = [&](uint32_t count, uint32_t k) { return (count < row_cap(k) ? count : row_cap(k)) * few_row_floats(k) * 4; };
    constexpr int U = EIDM_KERNEL_DECODE_GATE_UP, W = EIDM_KERNEL_DECODE_DOWN, WC = EIDM_KERNEL_DECODE_DOWN_COMBINE;
    constexpr uint32_t threads = 64 * kWaves;
    const bool route = a.m <= (uint32_t)kWaves && a.n_experts <= kRouteExperts;
    hipError_t err = hipSuccess;
    if (!route) {
        err = launch_route(a.logits, a.bias, a.m, a.n_experts, a.top_k, a.renormalize, a.ids, a.gates, stream);
        if (err != hipSuccess) return err;
    }
    const uint32_t up_blocks = blocks_of((a.inter + 3) / 4), up_lds = map_bytes + staged(rows, a.hidden);
    err = route ? launch_one<gate_up_kernel<DT, true>>(U, up_blocks, threads, up_lds, stream, a)
                : launch_one<gate_up_kernel<DT, false>>(U, up_blocks, threads, up_lds, stream, a);
    if (err != hipSuccess) return err;
    if (rows <= row_cap(a.inter)) {  // every row of h fits beside the map and the output rows
        const uint32_t cols = block_columns(a.hidden, 8, cus), blocks = (a.hidden + cols - 1) / cols;
        const uint32_t lds = map_bytes + rows * 32 + staged(rows, a.inter);
        return cols <= 4 ? launch_one<down_combine_kernel<DT, 1, 12>>(WC, blocks, threads, lds, stream, a, cols)
                         : launch_one<down_combine_kernel<DT, 2, 12>>(WC, blocks, threads, lds, stream, a, cols);
    }
    const uint32_t blocks = blocks_of((a.hidden + 7) / 8), lds = map_bytes + staged(rows, a.inter);
    err = launch_one<down_kernel<DT, 2, 12>>(W, blocks, threads, lds, stream, a);
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

// scratch: the id -> row map | h [m*top_k][inter] | y [m*top_k][hidden]
uint64_t align256(uint64_t v) { return (v + 255) & ~uint64_t(255); }
uint64_t map_bytes(const eidm_ffn_shape* f) { return align256(few_map_words(f->m * f->top_k, f->n_experts) * 4); }
uint64_t h_bytes(const eidm_ffn_shape* f) { return align256((uint64_t)f->m * f->top_k * f->inter * 4); }

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
    *scratch = map_bytes(f) + h_bytes(f) + (uint64_t)f->m * f->top_k * f->hidden * 4;
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
    uint8_t* ws = static_cast<uint8_t*>(scratch);
    a.map = reinterpret_cast<uint32_t*>(ws);
    a.h = reinterpret_cast<float*>(ws + eidm::map_bytes(shape));
    a.y = reinterpret_cast<float*>(ws + eidm::map_bytes(shape) + eidm::h_bytes(shape));
    a.out = out;
    const hipError_t err = eidm::launch_moe_decode(a, eidm::device_cus(), st);
    if (err != hipSuccess) return api_fail(EIDM_E_DEVICE, "decode FFN launch: %s", hipGetErrorString(err));
    return eidm::api_ok();
}

}  // extern "C"
