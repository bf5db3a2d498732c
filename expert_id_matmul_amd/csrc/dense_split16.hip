// dense_split16.hip -- one shared projection y = W x in the split-16
// arithmetic for many rows: the bits of eidm_matmul_id with one expert
// (matmul_split16.hip holds the arithmetic's definition), without ids, a map
// or gathered rows.
//
// A block of four wavefronts takes 128 rows by 128 columns, a wavefront 32
// rows by all 128 columns, so that
//   * the split activations, three parts a row and the larger operand, go
//     straight into the registers of the one wavefront that uses them, some
//     steps of 32 ahead; the split writes them in the order of the matrix
//     operand, so that such a load is 1 KB in a row (from the 48-byte chunks
//     of the gathered form a load touched 32 cache lines, and address
//     processing took as long as the products);
//   * the weights, which all four use, pass through LDS: 64 elements of k per
//     buffer, two buffers, one barrier per 96 products a wavefront.  A
//     column's four 16-byte chunks are stored permuted by its index, so the
//     16 columns that are read together fall on all banks.
// LDS then carries 40 KB per 32 of k (some 320 cycles) beside the 768 cycles
// of a wavefront's 48 matrix instructions; with the rows there too it would be
// 88 KB, as long as the products.
// Blocks run in groups of up to 64 tiles per XCD, near square, whose operands
// its L2 serves; fewer tiles make smaller groups, so that all XCDs have one
// (1024 x 4096 x 4096: 133 us, 189 with groups of 64 on half of them).
// Measured at 2048 x 4096 x 4096, bf16: 177-185 us, 1.11-1.16 PFLOP/s of 16-bit
// products (a large library product in bf16 reaches the same rate), and 16 us
// for the split.  The matrix core is busy 55 % of that time; wavefronts, two a
// SIMD, wait 30 % of their cycles and are ready but not issued 52 %.
//
// mlx-native 0.13.0, src/ops/dense_matmul_id_auto.rs: the value-independence
// theorem statement (one order, whichever rows are computed together).
#include "eidm_device.hpp"
#include "eidm_internal.hpp"
#include "split16.hpp"

namespace eidm {
namespace {

constexpr int kTile = 128;           // rows and columns of a block
constexpr int kWaveRows = 2;         // 16-row tiles per wavefront
constexpr int kColTiles = 8;         // 16-column tiles per wavefront
constexpr uint32_t kAhead = 2;       // steps of activations in registers
constexpr uint32_t kXcds = 8, kGroup = 64;  // XCDs; tiles of one XCD side by side
constexpr uint32_t kPartBytes = 1024;        // one part of 16 rows and 32 k: lane l's row l%16, chunk l/16

__host__ __device__ inline uint32_t split_steps(uint32_t k) { return (k + 127) / 128 * 4; }  // of 32, zeros past k

// The three parts of x (split16.hpp), one thread per (row, 8 elements).
template <int DT>
__global__ __launch_bounds__(256) void pack_split16_kernel(const float* __restrict__ x, uint32_t m, uint32_t k,
                                                           uint8_t* __restrict__ packed) {
    const uint32_t steps = split_steps(k), lane = threadIdx.x & 63;
    const uint64_t units = (uint64_t)((m + 15) / 16) * steps;  // of 16 rows and 32 k
    for (uint64_t unit = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < units; unit += (uint64_t)gridDim.x * 4) {
        const uint32_t row = (uint32_t)(unit / steps) * 16 + (lane & 15);
        const uint32_t kk = (uint32_t)(unit % steps) * 32 + (lane >> 4) * 8;
        uint32_t p[3][8] = {};
        if (row < m && kk < k) {  // k is a multiple of 8
            const f32x4* src = reinterpret_cast<const f32x4*>(x + (size_t)row * k + kk);
            const f32x4 a = src[0], b = src[1];
#pragma unroll
            for (int i = 0; i < 8; ++i) s16_split<DT>(i < 4 ? a[i % 4] : b[i % 4], p[0][i], p[1][i], p[2][i]);
        }
        uint8_t* to = packed + unit * 3 * kPartBytes + lane * 16;
#pragma unroll
        for (int q = 0; q < 3; ++q)
            *reinterpret_cast<s16u32x4*>(to + q * kPartBytes) =
                s16u32x4{p[q][0] | p[q][1] << 16, p[q][2] | p[q][3] << 16, p[q][4] | p[q][5] << 16,
                         p[q][6] | p[q][7] << 16};
    }
}

// A column's chunks stand xor-ed with 0, 2, 3, 1 by its four-column group: the
// 16 columns of one chunk fall on all 64 banks, and so do 8 columns each of
// two neighbouring chunks, in which the 16-byte reads are served.
__device__ __forceinline__ uint32_t place(uint32_t col) {
    const uint32_t a = col >> 2 & 3;
    return a >> 1 | ((a ^ a >> 1) & 1) << 1;
}

// group_rows x group_cols tiles form one XCD's group.
template <int DT>
__global__ __launch_bounds__(256, 2) void dense_split16_kernel(const uint8_t* __restrict__ packed,
                                                               const uint8_t* __restrict__ weights, uint32_t m,
                                                               uint32_t n, uint32_t k, uint32_t group_rows,
                                                               uint32_t group_cols, uint32_t groups_down,
                                                               float* __restrict__ out) {
    __shared__ s16u32x4 buf[2][2][kTile][4];  // [buffer][step of 32][column][chunk, permuted]
    const uint32_t tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
    // block -> XCD, group of that XCD, tile of the group
    const uint32_t tiles = group_rows * group_cols;
    const uint32_t xcd = blockIdx.x % kXcds, at = blockIdx.x / kXcds;
    const uint32_t group = at / tiles * kXcds + xcd, in = at % tiles;
    const uint32_t row0 = (group % groups_down * group_rows + in % group_rows) * kTile;
    const uint32_t col0 = (group / groups_down * group_cols + in / group_rows) * kTile;
    if (row0 >= m || col0 >= n) return;  // block-uniform

    const uint32_t chunks = k / 8;         // of a weight row
    const uint32_t steps = split_steps(k);  // a multiple of 4
    const uint8_t* xrow[kWaveRows];
#pragma unroll
    for (int t = 0; t < kWaveRows; ++t)
        xrow[t] = packed + (size_t)min(row0 / 16 + wave * 2 + t, (m - 1) / 16) * steps * 3 * kPartBytes + lane * 16;
    // weights: thread -> column tid/2, half tid%2 of its 8 chunks per buffer
    const uint32_t wcol = tid >> 1, whalf = tid & 1;
    const uint8_t* wsrc = weights + (size_t)min(col0 + wcol, n - 1) * k * 2;

    struct Parts {
        s16u32x4 p[kWaveRows][3];
    };
    auto load_x = [&](uint32_t step, Parts& x) {  // step past the end: the last one again
        const size_t off = (size_t)min(step, steps - 1) * 3 * kPartBytes;
#pragma unroll
        for (int t = 0; t < kWaveRows; ++t)
#pragma unroll
            for (int p = 0; p < 3; ++p) x.p[t][p] = *reinterpret_cast<const s16u32x4*>(xrow[t] + off + p * kPartBytes);
    };
    s16u32x4 w[4];
    auto load_w = [&](uint32_t pair) {  // steps 2*pair, 2*pair+1; this thread's step is whalf
        const uint32_t c0 = min(pair, steps / 2 - 1) * 8 + whalf * 4;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c)
            w[c] = *reinterpret_cast<const s16u32x4*>(wsrc + (size_t)min(c0 + c, chunks - 1) * 16);
    };
    auto store_w = [&](uint32_t pair, uint32_t b) {
        const uint32_t c0 = pair * 8 + whalf * 4;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c)
            buf[b][whalf][wcol][c ^ place(wcol)] = c0 + c < chunks ? w[c] : s16u32x4{0, 0, 0, 0};  // zeros past k
    };

    f32x4 hi[kWaveRows][kColTiles], lo[kWaveRows][kColTiles];
#pragma unroll
    for (int t = 0; t < kWaveRows; ++t)
#pragma unroll
        for (int c = 0; c < kColTiles; ++c) hi[t][c] = lo[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    Parts x[kAhead];
    load_w(0);
#pragma unroll
    for (uint32_t s = 0; s < kAhead; ++s) load_x(s, x[s]);
    store_w(0, 0);
    load_w(1);
    __syncthreads();
    for (uint32_t first = 0; first < steps; first += 4)  // steps come in fours
#pragma unroll
    for (uint32_t half = 0; half < 2; ++half) {
        const uint32_t pair = first / 2 + half, b = half;
        store_w(pair + 1, b ^ 1);  // (past the end: never read)
        load_w(pair + 2);
#pragma unroll
        for (uint32_t h2 = 0; h2 < 2; ++h2) {
            const uint32_t s = (2 * half + h2) % kAhead;
#pragma unroll
            for (int h = 0; h < kColTiles; h += 4) {
                s16u32x4 wt[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) wt[c] = buf[b][h2][(h + c) * 16 + i][g ^ place(i)];
#pragma unroll
                for (int t = 0; t < kWaveRows; ++t)
#pragma unroll
                    for (int c = 0; c < 4; ++c) hi[t][h + c] = s16_mfma<DT>(x[s].p[t][0], wt[c], hi[t][h + c]);
#pragma unroll
                for (int p = 1; p < 3; ++p)
#pragma unroll
                    for (int t = 0; t < kWaveRows; ++t)
#pragma unroll
                        for (int c = 0; c < 4; ++c) lo[t][h + c] = s16_mfma<DT>(x[s].p[t][p], wt[c], lo[t][h + c]);
            }
            load_x(2 * pair + h2 + kAhead, x[s]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < kWaveRows; ++t)
#pragma unroll
        for (uint32_t v = 0; v < 4; ++v) {
            const uint32_t r = row0 + wave * 32 + t * 16 + 4 * g + v;
#pragma unroll
            for (int c = 0; c < kColTiles; ++c) {
                const uint32_t col = col0 + c * 16 + i;
                if (r < m && col < n) out[(size_t)r * n + col] = hi[t][c][v] + lo[t][c][v];
            }
        }
}

}  // namespace

// The tiles fill half the device; nine sixteenths of it with k above 2048, all
// of it where the tiles themselves are far from full (up to 64 rows) or each
// split row serves few columns. Up to 32 rows are one row tile of
// eidm_matmul_id's kernels, which then read the weights once as well.
// Over 330 products (m 1 - 32768, n 64 - 131072, k 128 - 4096) the chosen one
// takes 0.6 % more than the better one on average, 16 % at most. Whole calls,
// bf16, us, this : those: 1 x 16384 x 4096 121 : 46, 64 x 16384 x 4096 133 : 77,
// 96 x 16384 x 4096 140 : 117, 32 x 65536 x 512 49 : 45, 64 x 65536 x 512 58 : 69,
// 1024 x 2048 x 4096 135 : 126, 1024 x 2048 x 1024 56 : 59, 1500 x 1500 x 4096
// 147 : 175, 1024 x 4096 x 4096 140 : 222, 12000 x 200 x 4096 351 : 309.
bool dense_split16_supported(uint32_t m, uint32_t n, uint32_t k, int device_cus) {
    const uint64_t cus = device_cus > 0 ? (uint64_t)device_cus : 256;
    if (m <= 32) return false;
    const uint64_t tiles = (uint64_t)((m + kTile - 1) / kTile) * ((n + kTile - 1) / kTile);
    const bool whole = m <= 64 || (uint64_t)n * 8 <= k;
    return tiles * 16 >= cus * (whole ? 16 : k > 2048 ? 9 : 8);
}

uint64_t dense_split16_bytes(uint32_t m, uint32_t k) {
    return (uint64_t)(m + 15) / 16 * split_steps(k) * 3 * kPartBytes;
}

template <int DT>
static hipError_t launch_dense(const MatmulArgs& a, int device_cus, hipStream_t stream) {
    uint8_t* packed = reinterpret_cast<uint8_t*>(a.xsplit);
    const uint64_t units = (uint64_t)(a.m + 15) / 16 * split_steps(a.k), most = (uint64_t)device_cus * 32;
    const uint32_t pack_grid = (uint32_t)((units + 3) / 4 < most ? (units + 3) / 4 : most);
    hipLaunchKernelGGL(pack_split16_kernel<DT>, dim3(pack_grid), dim3(256), 0, stream, a.input, a.m, a.k, packed);
    hipError_t err = launched(EIDM_KERNEL_SPLIT_X, pack_grid, 256, 0);
    if (err != hipSuccess) return err;
    const uint32_t down = (a.m + kTile - 1) / kTile, across = (a.n + kTile - 1) / kTile;
    // 8 x 8, half that while XCDs would be left without a group; no taller than the tiles are
    uint32_t group = kGroup, group_rows = 8;
    while (group > 8 && (uint64_t)group * kXcds > (uint64_t)down * across) group /= 2;
    while (group_rows > 1 && (group_rows / 2 >= down || group_rows * group_rows > group)) group_rows /= 2;
    const uint32_t group_cols = group / group_rows;
    const uint64_t groups_down = (down + group_rows - 1) / group_rows;
    const uint64_t groups = groups_down * ((across + group_cols - 1) / group_cols);
    const uint64_t grid = (groups + kXcds - 1) / kXcds * kXcds * group;
    if (grid > 0x7fffffffull) return hipErrorInvalidValue;
    hipLaunchKernelGGL(dense_split16_kernel<DT>, dim3((uint32_t)grid), dim3(256), 0, stream, packed,
                       static_cast<const uint8_t*>(a.weights), a.m, a.n, a.k, group_rows, group_cols,
                       (uint32_t)groups_down, a.output);
    return launched(EIDM_KERNEL_DENSE_SPLIT16, (uint32_t)grid, 256, 0);
}

hipError_t launch_dense_split16(const MatmulArgs& a, int device_cus, hipStream_t stream) {
    return a.dtype == kDtypeF16 ? launch_dense<kDtypeF16>(a, device_cus, stream)
                                : launch_dense<kDtypeBF16>(a, device_cus, stream);
}

}  // namespace eidm
