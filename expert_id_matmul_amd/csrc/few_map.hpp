// few_map.hpp -- the id -> row map of a few routed rows, built in LDS by one
// block: the ids that occur, ascending, each with its list of rows.
//
// Rows of one id stand in no fixed order (their slots come from LDS
// atomics): a row's result does not depend on which rows share its tile, so
// no output does either.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace eidm {

struct FewMap {
    uint32_t* start;  // [n_ids] working counts, then next free slots
    uint32_t* id;     // [min(n_ids, rows)] the ids that occur
    uint32_t* off;    // [min(n_ids, rows) + 1] where each id's rows start in row[]
    uint32_t* cost;   // [min(n_ids, rows) + 1] cost units of the ids before each
    uint32_t* row;    // [rows]
    uint32_t* used;   // [1] how many ids occur
};

__host__ __device__ constexpr uint32_t few_map_ids(uint32_t rows, uint32_t n_ids) { return n_ids < rows ? n_ids : rows; }

// LDS words of a map of `rows` rows over n_ids ids, whole 16-byte units: what
// follows is read 16 bytes at a time (off that boundary such a read is several)
__host__ __device__ constexpr uint32_t few_map_words(uint32_t rows, uint32_t n_ids) {
    return (n_ids + 3 * few_map_ids(rows, n_ids) + 3 + rows + 3) / 4 * 4;
}

__device__ __forceinline__ FewMap few_map_at(uint32_t* lds, uint32_t rows, uint32_t n_ids) {
    FewMap f;
    const uint32_t u = few_map_ids(rows, n_ids);
    f.start = lds;
    f.id = f.start + n_ids;
    f.off = f.id + u;
    f.cost = f.off + u + 1;
    f.used = f.cost + u + 1;
    f.row = f.used + 1;
    return f;
}

// Inclusive sum over the wavefront's lanes.
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// The whole block takes part; ids that are >= n_ids have no list.  The map
// is ready for every thread on return.  cost_of(rows of an id): its cost.
template <typename CostOf>
__device__ __forceinline__ void few_map_build(const FewMap& f, const uint32_t* ids, uint32_t rows, uint32_t n_ids,
                                              CostOf cost_of) {
    const uint32_t tid = threadIdx.x, nt = blockDim.x;
    for (uint32_t e = tid; e < n_ids; e += nt) f.start[e] = 0;
    __syncthreads();
    for (uint32_t r = tid; r < rows; r += nt) {
        const uint32_t e = ids[r];
        if (e < n_ids) atomicAdd(&f.start[e], 1u);
    }
    __syncthreads();
    if (tid < 64) {  // one wavefront scans the counts, 64 ids at a time
        uint32_t used = 0, at = 0, spent = 0;
        for (uint32_t e0 = 0; e0 < n_ids; e0 += 64) {
            const uint32_t e = e0 + tid;
            const uint32_t c = e < n_ids ? f.start[e] : 0;
            const uint64_t hit = __ballot(c != 0);
            if (!hit) continue;
            const uint32_t mine = c ? cost_of(c) : 0;
            const uint32_t inc = wave_prefix(c), sum = wave_prefix(mine);
            if (c) {
                const uint32_t u = used + (uint32_t)__popcll(hit & ((1ull << tid) - 1));
                f.id[u] = e;
                f.off[u] = at + inc - c;
                f.cost[u] = spent + sum - mine;
                f.start[e] = at + inc - c;
            }
            used += (uint32_t)__popcll(hit);
            at += (uint32_t)__builtin_amdgcn_readlane((int)inc, 63);
            spent += (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
        }
        if (tid == 0) {
            f.off[used] = at;
            f.cost[used] = spent;
            *f.used = used;
        }
    }
    __syncthreads();
    for (uint32_t r = tid; r < rows; r += nt) {
        const uint32_t e = ids[r];
        if (e < n_ids) f.row[atomicAdd(&f.start[e], 1u)] = r;
    }
    __syncthreads();
}

// The first job at or past `at` of jobs (id u, part g < parts) in order, each
// of which costs cost[u+1] - cost[u] units, counted by part from cost[u] *
// parts: jobs cut at such points have near equal costs.
__device__ __forceinline__ uint32_t few_map_job(const FewMap& f, uint32_t parts, uint64_t at) {
    uint32_t lo = 0, hi = *f.used;
    while (lo < hi) {  // the last id that starts at or before `at`
        const uint32_t mid = (lo + hi + 1) / 2;
        if ((uint64_t)f.cost[mid] * parts <= at) lo = mid;
        else hi = mid - 1;
    }
    if (lo == *f.used) return lo * parts;
    const uint32_t each = f.cost[lo + 1] - f.cost[lo];
    return lo * parts + (uint32_t)((at - (uint64_t)f.cost[lo] * parts + each - 1) / each);
}

}  // namespace eidm
