// eidm_internal.hpp -- kernel launchers behind the C ABI (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "eidm.h"

namespace eidm {

// Largest expert count the kernels take (router state per lane, map tables).
constexpr uint32_t kMaxExperts = 2048;

// Largest top_k the router takes (one pick per lane).
constexpr uint32_t kMaxRouterTopK = 64;
// fused route -> Direct -> combine: one wavefront per slot in a block
constexpr uint32_t kMaxMoeDirectTopK = 16;
// the few-token expert FFN: its id -> row map and its output rows sit in LDS
constexpr uint32_t kMaxDecodeTokens = EIDM_DECODE_MAX_TOKENS;
constexpr uint32_t kMaxDecodeTopK = 16;
constexpr uint32_t kMaxDecodeRow = 32768;
constexpr uint32_t kMaxLoraRank = EIDM_LORA_MAX_RANK;

struct MatmulArgs {
    int dtype;
    uint32_t m, n, k, top_k, n_experts;
    uint64_t stride;
    int layout;                 // 0 shared per token, 1 slotted
    const void* weights;
    const float* input;
    const uint32_t* ids;
    float* output;
    bool vec;                   // 16-byte aligned rows: vector loads allowed
    int arith;                  // eidm_arith
    uint16_t* xsplit;           // SPLIT16: the split activations (scratch), else null
};

// Device pointers into a Grouped scratch buffer.
struct MapBuffers {
    uint32_t* hist;     // [blocks][n_experts+1]
    uint32_t* counts;   // [n_experts+1]
    uint32_t* offsets;  // [n_experts+2]
    uint32_t* rows;     // [m*top_k]
};

uint32_t map_waves(uint32_t n_experts);
uint32_t map_blocks(uint64_t routed_rows, uint32_t n_experts);
uint64_t map_hist_elements(uint64_t routed_rows, uint32_t n_experts);

// error state of the C ABI (thread-local message; see eidm_last_error)
int api_fail(int code, const char* fmt, ...);
int api_ok();

// The dispatch receipt (see eidm_last_dispatch): each public entry point
// starts a new one on the calling thread; every kernel launch is noted.
// The outermost scope on a thread starts the receipt; nested entry points
// (a library call made by another one) add to it.
struct ReceiptScope {
    ReceiptScope();
    ~ReceiptScope();
    ReceiptScope(const ReceiptScope&) = delete;
    ReceiptScope& operator=(const ReceiptScope&) = delete;
};
void receipt_route(int route);
void note_launch(int kernel, uint32_t grid, uint32_t block, uint32_t lds_bytes);
// hipGetLastError() after a launch; the launch goes on the receipt only when
// it was accepted.
hipError_t launched(int kernel, uint32_t grid, uint32_t block, uint32_t lds_bytes);

hipError_t launch_route(const float* logits, const float* bias, uint32_t m, uint32_t n_experts,
                        uint32_t top_k, int renormalize, uint32_t* ids, float* gates,
                        hipStream_t stream);
hipError_t launch_map(const uint32_t* ids, uint32_t routed_rows, uint32_t n_experts,
                      const MapBuffers& buf, hipStream_t stream);
// eidm_matmul_id for a sequence of calls over one set of ids (and one
// scratch): a Grouped call skips the id -> row map when *map_ready says an
// earlier Grouped call of the sequence left it in the scratch, and sets
// *map_ready when it builds it.
int matmul_id_shared_map(const eidm_shape* shape, int route, const void* weights, uint64_t weight_bytes,
                         const float* input, const uint32_t* ids, float* output, void* scratch,
                         uint64_t scratch_bytes, hipStream_t stream, bool* map_ready, int* route_taken);
hipError_t launch_direct(const MatmulArgs& a, hipStream_t stream);
hipError_t launch_grouped(const MatmulArgs& a, const MapBuffers& buf, int device_cus,
                          hipStream_t stream);
// The Grouped kernel on the 16x16x1 matrix-core step (16-bit weights, vector
// rows, at least two rounds, 32-bit offsets); launch_grouped picks it when
// grouped16_supported says so.
bool grouped16_supported(const MatmulArgs& a);
hipError_t launch_grouped16(const MatmulArgs& a, const MapBuffers& buf, int device_cus, hipStream_t stream);
// jobs of at most this many rounds of k run the build of the same kernel
// that keeps its accumulators in the accumulation registers
#ifndef EIDM_G16_ACC_ROUNDS
#define EIDM_G16_ACC_ROUNDS 12
#endif
constexpr uint32_t kG16AccRounds = EIDM_G16_ACC_ROUNDS;
hipError_t launch_grouped16_acc(const MatmulArgs& a, const MapBuffers& buf, int device_cus, hipStream_t stream);
// The split-16 arithmetic: the activation split (input -> a.xsplit), then
// the Direct or the Grouped form.
// bytes of the split activations of in_rows rows of k elements
uint64_t split16_bytes(uint64_t in_rows, uint32_t k);
hipError_t launch_split16_x(const MatmulArgs& a, hipStream_t stream);
// the id -> row map (one-launch form) and the activation split in one launch,
// when the map fits that form
bool map_split16_x_fits(const MatmulArgs& a);
hipError_t launch_map_split16_x(const MatmulArgs& a, const MapBuffers& buf, hipStream_t stream);
hipError_t launch_direct_split16(const MatmulArgs& a, hipStream_t stream);
hipError_t launch_grouped_split16(const MatmulArgs& a, const MapBuffers& buf, int device_cus, hipStream_t stream);
// one expert's product of many rows in the split-16 arithmetic (a.xsplit:
// dense_split16_bytes(m, k) of scratch; a.ids is not read)
bool dense_split16_supported(uint32_t m, uint32_t n, uint32_t k, int device_cus);
uint64_t dense_split16_bytes(uint32_t m, uint32_t k);
hipError_t launch_dense_split16(const MatmulArgs& a, int device_cus, hipStream_t stream);
hipError_t launch_combine(uint32_t m, uint32_t top_k, uint32_t n, const float* y,
                          const float* gates, float* out, hipStream_t stream);
bool moe_direct_supported(uint32_t top_k, uint32_t n_experts);
// synchronous: waits for `stream`; *first_bad = smallest bad routed index or -1
hipError_t run_validate(const uint32_t* ids, uint32_t m, uint32_t top_k, uint32_t n_experts, int distinct,
                        hipStream_t stream, int* first_bad);
// The expert FFN of a few tokens (moe_decode.hip); h [m*top_k][inter] and
// y [m*top_k][hidden] are f32 scratch, map the first kernel's id -> row map.
struct MoeDecodeArgs {
    int dtype;
    uint32_t m, hidden, inter, top_k, n_experts;
    uint64_t gate_up_stride, down_stride;
    const uint8_t *w_gate, *w_up, *w_down;
    const float *x, *logits, *bias;
    int renormalize;
    uint32_t *ids, *map;
    float *gates, *h, *y, *out;
};
hipError_t launch_moe_decode(const MoeDecodeArgs& a, int device_cus, hipStream_t stream);
// compute units of the current device
int device_cus();
// Low-rank adapters (lora.hip): v [m][v_stride] f32 scratch; base may be
// output itself.
struct LoraArgs {
    int dtype;  // of the adapters
    uint32_t m, n, k, n_adapters, max_rank, v_stride;
    uint64_t a_stride, b_stride;
    const uint8_t *a, *b;
    const uint32_t *ranks, *ids;
    const float *scales, *x, *base;
    float *v, *out;
    uint32_t* zero_ids;  // [m] ids of the shared projection, written by the shrink (or null)
    // the id -> row map of the rows (null: the row forms)
    const uint32_t *offsets, *rows;
    uint32_t* tiles;  // the sorted rows in tiles of 16, written by the shrink
};
// rows up to which each reads its adapter by itself (a row that a block can
// stage); more are sorted by adapter when that is the faster form
constexpr uint32_t kLoraRowForm = 64;
bool lora_sorts_rows(uint32_t m, uint32_t n, uint32_t k, uint32_t n_adapters, uint32_t max_rank);
hipError_t launch_lora_shrink(const LoraArgs& a, int device_cus, hipStream_t stream);
// out = W x for up to some hundred rows (any alignment), and the shrink of them
bool lora_base_few_supported(const LoraArgs& a, int device_cus);
hipError_t launch_lora_base_few(const LoraArgs& a, int weight_dtype, const uint8_t* weights, int device_cus,
                                hipStream_t stream);
hipError_t launch_lora_expand(const LoraArgs& a, int device_cus, hipStream_t stream);
// a.ids is ignored: the kernel writes the picks to `ids` and reads them itself
hipError_t launch_moe_direct(const MatmulArgs& a, const float* logits, const float* bias, int renormalize,
                             uint32_t* ids, float* gates, float* out, int device_cus, hipStream_t stream);

}  // namespace eidm
