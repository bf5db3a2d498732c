// few_map.hpp -- the id -> row map of a few routed rows, built in LDS by one
// block: the ids that occur, ascending, each with its list of rows.
//
// Rows of one id stand in no fixed order (their slots come from LDS
// atomics): a row's result does not depend on which rows share its tile, so
// no output does either.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

// Inclusive sum over the wavefront's lanes: within rows of 16 by shifts, then
// the rows' totals by broadcasts (DPP: no LDS latency).
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
    auto add = [&](auto ctrl, auto rows) {
        v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
    };
    using std::integral_constant;
    add(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr:1
    add(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});  // row_shr:2
    add(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});  // row_shr:4
    add(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});  // row_shr:8
    add(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});  // row_bcast:15 into rows 1, 3
    add(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});  // row_bcast:31 into rows 2, 3
    return v;
}

constexpr uint32_t kFewMapRows = 2;   // most rows per thread
constexpr uint32_t kFewMapUnits = 4;  // most 16-byte units per thread of a map's copy

// This thread's rows' ids, requested before anything that the map is not for.
struct FewIds {
    uint32_t e[kFewMapRows];
};

__device__ __forceinline__ FewIds few_map_ids_load(const uint32_t* ids, uint32_t rows) {
    FewIds f;
#pragma unroll
    for (uint32_t j = 0; j < kFewMapRows; ++j) f.e[j] = ids[min(threadIdx.x + j * blockDim.x, rows - 1)];
    return f;
}

// The whole block takes part (rows <= kFewMapRows * blockDim.x); ids that are
// >= n_ids have no list.  The map is ready for every thread on return.
// cost_of(rows of an id): its cost.
template <typename CostOf>
__device__ __forceinline__ void few_map_build(const FewMap& f, const FewIds& ids, uint32_t rows, uint32_t n_ids,
                                              CostOf cost_of) {
    const uint32_t tid = threadIdx.x, nt = blockDim.x;
    for (uint32_t e = tid; e < n_ids; e += nt) f.start[e] = 0;
    __syncthreads();
#pragma unroll
    for (uint32_t j = 0; j < kFewMapRows; ++j)
        if (tid + j * nt < rows && ids.e[j] < n_ids) atomicAdd(&f.start[ids.e[j]], 1u);
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
#pragma unroll
    for (uint32_t j = 0; j < kFewMapRows; ++j)
        if (tid + j * nt < rows && ids.e[j] < n_ids) f.row[atomicAdd(&f.start[ids.e[j]], 1u)] = tid + j * nt;
    __syncthreads();
}

// A built map to memory, and from there into another kernel's LDS: load()
// requests it, store() writes it (a barrier must follow).
__device__ __forceinline__ void few_map_save(const uint32_t* lds, uint32_t words, uint32_t* to) {
    for (uint32_t i = threadIdx.x; i < words / 4; i += blockDim.x)
        reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(lds)[i];
}

struct FewMapCopy {
    uint4 v[kFewMapUnits];
    __device__ __forceinline__ void load(const uint32_t* from, uint32_t words) {
#pragma unroll
        for (uint32_t j = 0; j < kFewMapUnits; ++j)
            v[j] = reinterpret_cast<const uint4*>(from)[min(threadIdx.x + j * blockDim.x, words / 4 - 1)];
    }
    __device__ __forceinline__ void store(uint32_t* lds, uint32_t words) const {
#pragma unroll
        for (uint32_t j = 0; j < kFewMapUnits; ++j)
            reinterpret_cast<uint4*>(lds)[min(threadIdx.x + j * blockDim.x, words / 4 - 1)] = v[j];
    }
};

// The first job at or past `at` of jobs (id u, part g < parts) in order, each
// of which costs cost[u+1] - cost[u] units, counted by part from cost[u] *
// parts: jobs cut at such points have near equal costs.  (At most 1024 rows of
// 8 units and 8192 parts: 32 bits suffice.)  Every lane takes part.
__device__ __forceinline__ uint32_t few_map_job(const FewMap& f, uint32_t parts, uint32_t at) {
    const uint32_t used = *f.used, lane = threadIdx.x & 63;
    uint32_t before = 0;  // ids that start at or before `at`: id 0 does
    for (uint32_t u0 = 0; u0 < used; u0 += 64) {
        const uint32_t u = u0 + lane;
        before += (uint32_t)__popcll(__ballot(u < used && f.cost[min(u, used - 1)] * parts <= at));
    }
    const uint32_t u = (uint32_t)__builtin_amdgcn_readfirstlane((int)before) - 1;
    if (at >= f.cost[used] * parts) return used * parts;
    const uint32_t each = f.cost[u + 1] - f.cost[u];
    return u * parts + (at - f.cost[u] * parts + each - 1) / each;
}

}  // namespace eidm
