// w4.hpp -- weights in 4 bits with a 16-bit scale (and a zero point) per group:
// the layout shared by the kernels (k_w4_*.hip) and their entry points
// (gated_api.cpp).
//
// A row of K elements is ceil(K/group) groups of `group` (32, 64 or 128)
// consecutive k with one scale s and one zero point z (8 where none is stored); element
// k is s * (q - z), q its code 0 .. 15.  Codes are stored as MX4's are: 16
// bytes per 32 k, the even k in a byte's low half.
#pragma once

#include "gated.hpp"
#include "mx4.hpp"

namespace dgt {
namespace w4 {

// An operand of rows x K.
struct Weight {
    const uint8_t* Q;
    int64_t ldq;         // bytes
    const uint16_t* S;   // BF16 or FP16 bits
    int64_t lds;         // elements
    const uint8_t* Z;    // optional
    int64_t ldz;         // bytes
    bool s_bf16;
    int log_group;       // 5, 6 or 7
};

inline int groups(int K, int log_group) {
    return (int)(((int64_t)K + (1 << log_group) - 1) >> log_group);
}

struct Product {  // C <- alpha*A*W^T + beta*C + bias; K > 0, as in Gated
    int M, N, K;
    float alpha, beta;
    const uint16_t* A;
    int64_t lda;  // elements
    Weight w;
    float* C;
    int64_t ldc;
    const float* bias;
};

struct Gated {  // H <- act(X*W[:N]^T + bg) * (X*W[N:]^T + bu)
    gated::Act act;
    int M, N, K;
    const uint16_t* X;
    int64_t ldx;
    Weight w;  // 2N rows
    const float *bg, *bu;
    uint16_t* H;
    int64_t ldh;
};

// A scale's value.
__device__ __forceinline__ float scale_value(uint32_t bits, bool bf16) {
    return bf16 ? bf16_bits_to_f32(bits)
                : (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

hipError_t launch_quantize(In t, int M, int K, const void* X, int64_t ldx, uint8_t* Q, int64_t ldq,
                           uint16_t* S, int64_t lds, uint8_t* Z, int64_t ldz, bool s_bf16,
                           int log_group, hipStream_t s);
hipError_t launch_dequantize(In t, int M, int K, const Weight& w, void* Y, int64_t ldy,
                             hipStream_t s);
hipError_t launch_product(In t, const Product& p, hipStream_t s);
hipError_t launch_gated(In t, const Gated& p, hipStream_t s);

}  // namespace w4
}  // namespace dgt
