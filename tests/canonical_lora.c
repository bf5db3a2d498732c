/* CPU evaluation of the adapters' documented order, test infrastructure only:
 * u = fma chain over i ascending from +0 of B[j, i] * v[i], out =
 * fma(scale, u, base).  v is f32 [m][v_stride] (the shrink's results), b the
 * adapters' B already widened to f32 [n_adapters][n][max_rank]. */
#include <math.h>
#include <stdint.h>

void canonical_lora_expand(uint32_t m, uint32_t n, uint32_t n_adapters, uint32_t max_rank, uint32_t v_stride,
                           const float* base, const float* b, const uint32_t* ranks, const float* scales,
                           const float* v, const uint32_t* ids, float* out) {
    for (uint64_t t = 0; t < m; ++t) {
        const uint32_t id = ids[t];
        uint32_t rank = 0;
        if (id < n_adapters) rank = ranks && ranks[id] < max_rank ? ranks[id] : max_rank;
        for (uint64_t j = 0; j < n; ++j) {
            float y = base[t * n + j];
            if (rank) {
                float u = 0.0f;
                for (uint32_t i = 0; i < rank; ++i)
                    u = fmaf(b[((uint64_t)id * n + j) * max_rank + i], v[t * v_stride + i], u);
                y = fmaf(scales ? scales[id] : 1.0f, u, y);
            }
            if (id >= n_adapters && id != 0xffffffffu) y = NAN;
            out[t * n + j] = y;
        }
    }
}
