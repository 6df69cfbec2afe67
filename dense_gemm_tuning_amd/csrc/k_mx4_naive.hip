// k_mx4_naive.hip -- products with microscaled 4-bit operands, one lane per
// output: C(i,j) = sum over blocks of (sum over the block of a*b), each
// operand decoded block by block, fp32 sums in block order.
#include "mx4.hpp"

namespace dgt {
namespace mx4 {

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// The block's 32 values.
__device__ __forceinline__ void decode(const uint8_t* q, uint32_t s, float (&v)[kBlock]) {
    const u32x4 c = *reinterpret_cast<const u32x4*>(q);
    const float sc = scale_bits(s);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[w], sc, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[w], sc, 1);
        const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[w], sc, 2);
        const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[w], sc, 3);
        v[8 * w + 0] = a[0]; v[8 * w + 1] = a[1]; v[8 * w + 2] = b[0]; v[8 * w + 3] = b[1];
        v[8 * w + 4] = d[0]; v[8 * w + 5] = d[1]; v[8 * w + 6] = e[0]; v[8 * w + 7] = e[1];
    }
}

// T: the format of A; kMx: A is MX4 (T unused).
template <bool kMx, In T>
__global__ __launch_bounds__(256) void mx4_naive_kernel(Params p, int tiles_n, int nb) {
    const int col = (int)(blockIdx.x % tiles_n) * 64 + threadIdx.x;
    const int row = (int)(blockIdx.x / tiles_n) * 4 + threadIdx.y;
    if (row >= p.M || col >= p.N) return;
    const uint8_t* b = p.B + (int64_t)col * p.ldb;
    const uint8_t* sb = p.SB + (int64_t)col * p.ldsb;
    float acc = 0.0f;
    for (int kb = 0; kb < nb; ++kb) {
        float x[kBlock], y[kBlock];
        decode(b + (int64_t)kb * kChunk, sb[kb], y);
        if constexpr (kMx) {
            decode(static_cast<const uint8_t*>(p.A) + (int64_t)row * p.lda + (int64_t)kb * kChunk,
                   p.SA[(int64_t)row * p.ldsa + kb], x);
        } else {
            const uint16_t* a = static_cast<const uint16_t*>(p.A) + (int64_t)row * p.lda;
#pragma unroll
            for (int i = 0; i < kBlock; ++i)
                x[i] = kb * kBlock + i < p.K ? load_in<T>(a + kb * kBlock + i) : 0.0f;
        }
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < kBlock; ++i) part = fmaf(x[i], y[i], part);
        acc += part;
    }
    float* c = p.C + (int64_t)row * p.ldc + col;
    *c = epilogue(acc, p, c, col);
}

template <bool kMx, In T>
hipError_t launch(const Params& p, hipStream_t s) {
    const int tiles_n = (p.N + 63) / 64;
    const int64_t wgs = (int64_t)tiles_n * ((p.M + 3) / 4);
    if (wgs > 0x7fffffff) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((mx4_naive_kernel<kMx, T>), dim3((unsigned)wgs), dim3(64, 4), 0, s, p,
                       tiles_n, blocks(p.K));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product(const Params& p, hipStream_t s) { return launch<true, In::BF16>(p, s); }

hipError_t launch_product16(In t, const Params& p, hipStream_t s) {
    return t == In::BF16 ? launch<false, In::BF16>(p, s) : launch<false, In::F16>(p, s);
}

}  // namespace mx4
}  // namespace dgt
