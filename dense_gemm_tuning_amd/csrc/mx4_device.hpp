// mx4_device.hpp -- device pieces shared by the kernels that multiply
// microscaled 4-bit weights with few rows (k_mx4_skinny.hip, k_mx4_rows.hip).
#pragma once

#include <utility>

#include "mx4.hpp"

namespace dgt {
namespace mx4 {

// The format of A.
enum class Kind { MX4, BF16, F16 };

typedef int intx8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ intx8 widen(u32x4 x) {
    return intx8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
}

// f(0), .., f(n-1) with compile-time arguments.
template <int... I, typename F>
__device__ __forceinline__ void static_for(std::integer_sequence<int, I...>, F&& f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    static_for(std::make_integer_sequence<int, N>{}, f);
}

// The 8 values of a dword of codes under scale byte s, as BF16 bits.
__device__ __forceinline__ u32x4 decode8(uint32_t q, float sc) {
    return u32x4{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 0)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 1)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 2)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 3))};
}

// ... and as unscaled FP16 bits (every magnitude is exact).
__device__ __forceinline__ u32x4 decode8_f16(uint32_t q) {
    return u32x4{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 0)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 1)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 2)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 3))};
}

// Scale byte b of a dword as the number it stands for: the value of code 2
// (1.0) under it.
__device__ __forceinline__ float scale_number(uint32_t s, int b) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(0x22u, scale_bits((s >> (8 * b)) & 255u), 0)[0];
}

// Weights under FP16 activations: acc += scale * (a * w) with the block's
// codes unscaled, since the scale's range does not fit FP16; the four lane
// groups hold the same block (8 of its k each), so a column's scale is one
// number for the whole product.
__device__ __forceinline__ floatx4 scaled_product_f16(u32x4 a, u32x4 w, float scale, floatx4 acc) {
    const floatx4 d = mfma16x16x32<In::F16>(a, w, floatx4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(scale, d[r], acc[r]);
    return acc;
}

}  // namespace mx4
}  // namespace dgt
