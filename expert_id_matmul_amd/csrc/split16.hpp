// split16.hpp -- the split-16 arithmetic's two steps, an f32 activation as
// three 16-bit parts and the matrix instruction that multiplies them; every
// kernel of that arithmetic has them from here, so their products agree bit
// for bit (matmul_split16.hip holds the order of the products).
#pragma once

#include "eidm_device.hpp"

namespace eidm {

typedef __bf16 s16_bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 s16_f16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int s16u32x4 __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ f32x4 s16_mfma(const s16u32x4& a, const s16u32x4& b, f32x4 c) {
    if constexpr (DT == kDtypeF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(s16_f16x8, a),
                                                      __builtin_bit_cast(s16_f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(s16_bf16x8, a),
                                                       __builtin_bit_cast(s16_bf16x8, b), c, 0, 0, 0);
}

// f32 -> 16-bit, round to nearest even; the value back in f32
template <int DT> __device__ __forceinline__ uint32_t s16_round(float v);
template <> __device__ __forceinline__ uint32_t s16_round<kDtypeBF16>(float v) {
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7f800000u) == 0x7f800000u) return (u >> 16) | ((u & 0xffffu) ? 0x40u : 0u);  // inf, NaN stay
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}
template <> __device__ __forceinline__ uint32_t s16_round<kDtypeF16>(float v) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v);
}
template <int DT> __device__ __forceinline__ float s16_value(uint32_t h);
template <> __device__ __forceinline__ float s16_value<kDtypeBF16>(uint32_t h) { return __uint_as_float(h << 16); }
template <> __device__ __forceinline__ float s16_value<kDtypeF16>(uint32_t h) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// x = p1 + p2 + p3: p1 = rn(x), p2 = rn(x - p1), p3 = rn(x - p1 - p2); the
// differences are exact in f32.  A non-finite x keeps p1 = rn(x), p2 = p3 = 0.
template <int DT>
__device__ __forceinline__ void s16_split(float v, uint32_t& p1, uint32_t& p2, uint32_t& p3) {
    p1 = s16_round<DT>(v);
    const float f1 = s16_value<DT>(p1);
    if (!__builtin_isfinite(v) || !__builtin_isfinite(f1)) {
        p2 = p3 = 0;
        return;
    }
    const float r1 = v - f1;
    p2 = s16_round<DT>(r1);
    const float r2 = r1 - s16_value<DT>(p2);
    p3 = s16_round<DT>(r2);
}

}  // namespace eidm
