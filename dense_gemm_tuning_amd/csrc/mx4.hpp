// mx4.hpp -- microscaled 4-bit operands: the layout shared by the kernels
// (k_mx4_*.hip) and their entry points (mx4_api.cpp).
//
// A row of K elements is ceil(K/32) blocks of 32 consecutive k.  Element k is
// value(code) * 2^(s - 127): code 4 bits (sign, then one of 0, 0.5, 1, 1.5,
// 2, 3, 4, 6; the even k in a byte's low half), s the block's scale byte
// (255: NaN).  So one 16-byte chunk of codes is one block with one scale,
// which is also what a lane of the matrix cores' scaled 4-bit products takes:
// 16 bytes of 32 consecutive k and one scale byte.
#pragma once

#include "gemm_common.hpp"

namespace dgt {
namespace mx4 {

constexpr int kBlock = 32;        // elements of a block
constexpr int kChunk = 16;        // bytes of its codes
constexpr int kScaleRow = 16;     // scale pitches are multiples of this many blocks

inline int blocks(int K) { return K / kBlock + (K % kBlock != 0); }
inline int64_t code_pitch(int K) { return (int64_t)kChunk * blocks(K); }
inline int64_t scale_pitch(int K) {
    return (int64_t)kScaleRow * ((blocks(K) + kScaleRow - 1) / kScaleRow);
}

// Whether one launch holds that many workgroups (fewer than 2^32 threads).
inline bool launchable(int64_t workgroups, int threads) {
    return workgroups < (int64_t(1) << 32) / threads;
}

struct Params {
    int M, N, K;
    float alpha, beta;
    const void* A;       // MX4 codes, or 16-bit elements
    const uint8_t* SA;   // scales of A (MX4)
    const uint8_t* B;
    const uint8_t* SB;
    int64_t lda;         // MX4: bytes; 16-bit: elements
    int64_t ldsa, ldb, ldsb;  // bytes
    float* C;
    int64_t ldc;
    const float* bias;
};

// (alpha*acc + beta*c) + bias[col]; C is read only when beta != 0.
__device__ __forceinline__ float epilogue(float acc, const Params& p, const float* c, int col) {
    const float r = p.beta == 0.0f ? p.alpha * acc : p.alpha * acc + p.beta * (*c);
    return p.bias ? r + p.bias[col] : r;
}

// Scale byte s as a float with the exponent field s: 2^(s-127), and for 0 and
// 255 the bit patterns that the scaled conversions read as 2^-127 and NaN
// (they take the exponent field alone).
__device__ __forceinline__ float scale_bits(uint32_t s) { return __uint_as_float(s << 23); }

hipError_t launch_quantize(In t, bool trans, int M, int K, const void* X, int64_t ldx, uint8_t* Q,
                           int64_t ldq, uint8_t* S, int64_t lds, hipStream_t s);
hipError_t launch_dequantize(In t, int M, int K, const uint8_t* Q, int64_t ldq, const uint8_t* S,
                             int64_t lds, void* Y, int64_t ldy, hipStream_t s);
// Products with MX4 and with 16-bit A (k_mx4_rows.hip, which chooses), and
// the forms chosen: tiles, and wave-private strips of rb blocks of 16 rows.
hipError_t launch_product(const Params& p, hipStream_t s);
hipError_t launch_product16(In t, const Params& p, hipStream_t s);
hipError_t launch_product_tile(const Params& p, hipStream_t s);
hipError_t launch_skinny(const Params& p, int rb, int cols, hipStream_t s);
hipError_t launch_skinny16(In t, const Params& p, int rb, int cols, hipStream_t s);

}  // namespace mx4
}  // namespace dgt
