// i8_args.hpp -- the 8-bit products' kernel arguments, launchers and epilogue.
#pragma once

#include "eidm_internal.hpp"

namespace eidm {

__device__ __forceinline__ float scaled_sum(int acc, float sx, float sw) { return ((float)acc * sx) * sw; }

// silu(g) * u, the f32 number nearest to the 64-bit value: h is quantised, and
// a rounding that depended on how exp() is computed would move its whole
// numbers by one here and there.
__device__ __forceinline__ float silu_mul(float g, float u) {
    const double d = (double)g;
    return (float)(d / (1.0 + exp(-d)) * (double)u);
}

// One projection, or (w2 given) gate and up of an FFN with h = silu(gate) * up.
struct I8Args {
    uint32_t m, n, k, top_k, n_experts;
    uint64_t stride;
    bool slotted;
    const int8_t *w, *w2;        // [n_experts][n][k]; w2: the up projection
    const float *ws, *ws2;       // [n_experts][n]
    const int8_t* x;             // [m or m*top_k][k]
    const float* xs;             // [m or m*top_k]
    const uint32_t* ids;         // [m*top_k], null: one weight for all rows
    const uint32_t *offsets, *rows;  // the id -> row map (tiles, with ids)
    float* out;                  // [m*top_k][n]
};

// The shape's own checks (the entry point's error codes), and the id -> row map
// in a scratch of eidm_matmul_id_i8_scratch_bytes(shape) bytes (a valid shape).
int check_i8_shape(const eidm_i8_shape* shape);
MapBuffers i8_map_at(const eidm_i8_shape* shape, void* scratch);

// Rows by themselves or tiles, by what is read: sharing saves the reads of every
// routed row beyond its expert's first, and costs the map and more launches,
// the time of reading some 64 MB.  (Experts are counted as if picks were even.)
// row_bytes: what a row's reads cost by themselves, where a load is a whole
// wavefront's however short k is.
uint64_t i8_row_bytes(uint32_t n, uint32_t k);
bool i8_rows_by_themselves(uint32_t m, uint32_t top_k, uint32_t n_experts, uint64_t expert_bytes, uint64_t row_bytes);
// The same with one weight for all rows, which stays in the caches.
bool i8_dense_rows_by_themselves(uint32_t m, uint32_t n, uint32_t k, bool whole_units);
// Rows by themselves read their weights past the caches: most are read once, and more than the caches keep to the next call.
bool i8_read_once(uint32_t m, uint32_t top_k, uint32_t n_experts, uint64_t expert_bytes);

hipError_t launch_i8_rows(const I8Args& a, hipStream_t stream);
hipError_t launch_i8_tiles(const I8Args& a, int device_cus, hipStream_t stream);

// Gate and up of a few tokens with the routing: a.x (8 bits, with a.xs) or x (f32).
struct I8OneArgs {
    I8Args a;
    const float *x, *logits, *bias;
    int renormalize;
    uint32_t* ids;
    float* gates;
};
constexpr uint32_t kI8OneRow = 8192;  // longest row of x
bool i8_one_supported(const I8Args& a, int device_cus);
hipError_t launch_i8_gate_up_one(const I8OneArgs& o, hipStream_t stream);

// The down projection of a few tokens' h rows [m*top_k][k] f32, quantised as
// they are read, and the combine.
struct I8DownArgs {
    uint32_t m, n, k, top_k, n_experts;
    uint64_t stride;
    const int8_t* w;
    const float* ws;
    const float* h;
    const uint32_t* ids;
    const float* gates;
    float* out;
};
constexpr uint32_t kI8DownTopK = 16;  // a wavefront per slot in one block
hipError_t launch_i8_down_combine(const I8DownArgs& a, hipStream_t stream);

hipError_t launch_quantize_rows(int dtype, const void* x, uint32_t rows, uint32_t k, int8_t* q, float* scales,
                                hipStream_t stream);

}  // namespace eidm
