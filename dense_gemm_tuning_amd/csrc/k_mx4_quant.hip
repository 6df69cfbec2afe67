// k_mx4_quant.hip -- quantising to microscaled 4-bit blocks, and reading
// them back.
#include "mx4.hpp"

namespace dgt {
namespace mx4 {

namespace {

constexpr int NT = 256;

// One lane per scale byte (a block, or a pad byte past the last block).
template <In T, bool TR>
__global__ __launch_bounds__(NT) void quantize_kernel(const void* Xv, int64_t ldx, int M, int K,
                                                      uint8_t* Q, int64_t ldq, uint8_t* S,
                                                      int64_t lds, int nb, int slots) {
    using E = typename InFmt<T>::S;
    const E* X = static_cast<const E*>(Xv);
    const int64_t total = (int64_t)M * slots;
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * NT) {
        const int row = (int)(TR ? e % M : e / slots), kb = (int)(TR ? e / M : e % slots);
        uint8_t* srow = S + (int64_t)row * lds + kb;
        if (kb >= nb) {
            *srow = 127;
            continue;
        }
        float x[kBlock];
        uint32_t top = 0;  // largest magnitude's bits (NaN and infinity on top)
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            const int k = kb * kBlock + i;
            x[i] = k >= K ? 0.0f
                          : load_in<T>(TR ? X + (int64_t)k * ldx + row : X + (int64_t)row * ldx + k);
            top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
        }
        // exponent field of floor(log2(amax)) - 2, not below 0
        const uint32_t field = top >> 23;
        const uint32_t s = field == 255 ? 255 : field > 2 ? field - 2 : 0;
        u32x4 q = {0u, 0u, 0u, 0u};
        if (s != 255) {
            const float sc = scale_bits(s);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t v = 0;
                v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[8 * w], x[8 * w + 1], sc, 0);
                v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[8 * w + 2], x[8 * w + 3], sc, 1);
                v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[8 * w + 4], x[8 * w + 5], sc, 2);
                v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[8 * w + 6], x[8 * w + 7], sc, 3);
                q[w] = v;
            }
        }
        *reinterpret_cast<u32x4*>(Q + (int64_t)row * ldq + (int64_t)kb * kChunk) = q;
        *srow = (uint8_t)s;
    }
}

template <In T>
__device__ __forceinline__ void store_out(typename InFmt<T>::S* y, float v) {
    if constexpr (T == In::F32) *y = v;
    else if constexpr (T == In::BF16) *y = __builtin_bit_cast(uint16_t, (__bf16)v);
    else *y = __builtin_bit_cast(uint16_t, (_Float16)v);
}

// One lane per byte of codes.
template <In T>
__global__ __launch_bounds__(NT) void dequantize_kernel(const uint8_t* Q, int64_t ldq,
                                                        const uint8_t* S, int64_t lds, int M,
                                                        int K, void* Yv, int64_t ldy) {
    using E = typename InFmt<T>::S;
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const int per_row = (K + 1) / 2;
    const int64_t total = (int64_t)M * per_row;
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * NT) {
        const int64_t row = e / per_row;
        const int byte = (int)(e % per_row);
        const uint32_t q = Q[row * ldq + byte], s = S[row * lds + byte / kChunk];
        const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale_bits(s), 0);
        E* y = static_cast<E*>(Yv) + row * ldy + 2 * byte;
        store_out<T>(y, v[0]);
        if (2 * byte + 1 < K) store_out<T>(y + 1, v[1]);
    }
}

unsigned grid_for(int64_t items) {
    const int64_t g = (items + NT - 1) / NT;
    return (unsigned)(g < 65536 ? g : 65536);  // grid-stride loops cover the rest
}

}  // namespace

hipError_t launch_quantize(In t, bool trans, int M, int K, const void* X, int64_t ldx, uint8_t* Q,
                           int64_t ldq, uint8_t* S, int64_t lds, hipStream_t s) {
    const int nb = blocks(K), slots = (int)scale_pitch(K);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid_for((int64_t)M * slots)), dim3(NT), 0, s, X, ldx, M, K,
                           Q, ldq, S, lds, nb, slots);
        return hipGetLastError();
    };
    if (t == In::F32) return trans ? go(quantize_kernel<In::F32, true>) : go(quantize_kernel<In::F32, false>);
    if (t == In::BF16) return trans ? go(quantize_kernel<In::BF16, true>) : go(quantize_kernel<In::BF16, false>);
    return trans ? go(quantize_kernel<In::F16, true>) : go(quantize_kernel<In::F16, false>);
}

hipError_t launch_dequantize(In t, int M, int K, const uint8_t* Q, int64_t ldq, const uint8_t* S,
                             int64_t lds, void* Y, int64_t ldy, hipStream_t s) {
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid_for((int64_t)M * ((K + 1) / 2))), dim3(NT), 0, s, Q,
                           ldq, S, lds, M, K, Y, ldy);
        return hipGetLastError();
    };
    return t == In::F32    ? go(dequantize_kernel<In::F32>)
           : t == In::BF16 ? go(dequantize_kernel<In::BF16>)
                           : go(dequantize_kernel<In::F16>);
}

}  // namespace mx4
}  // namespace dgt
