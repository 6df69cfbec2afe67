// k_mx4_quant.hip -- quantising to microscaled 4-bit blocks, and reading
// them back.  Bound by HBM: an element is read once (2 or 4 bytes) and 17/32
// of a byte written, or the other way round.
//
// Per block of 32 consecutive k: s = max(0, exponent field of the largest
// magnitude - 2) (the biased exponent of floor(log2(amax)) - 2; an infinity or
// NaN has field 255, which is the NaN scale), and each element the nearest
// code of x * 2^(127 - s), ties to even, at most 6: what the scaled FP4
// conversion computes from fp32, which holds every input exactly.
#include "mx4.hpp"

namespace dgt {
namespace mx4 {

namespace {

constexpr int NT = 256;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The scale byte of a block whose largest magnitude has the bits `top`.
__device__ __forceinline__ uint32_t scale_of(uint32_t top) {
    const uint32_t field = top >> 23;
    return field == 255 ? 255u : field > 2 ? field - 2 : 0u;
}

// Eight codes under scale byte s (zero codes in a NaN block).
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], uint32_t s) {
    const float sc = scale_bits(s);
    uint32_t v = 0;
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[0], x[1], sc, 0);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[2], x[3], sc, 1);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[4], x[5], sc, 2);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[6], x[7], sc, 3);
    return s == 255 ? 0u : v;
}

// Eight elements of a row as raw bits (fp32: two pieces), zeros past K.
template <In T>
struct Raw {
    static constexpr int N = T == In::F32 ? 2 : 1;
    u32x4 w[N];
    __device__ float get(int e) const {
        if constexpr (T == In::F32) return __uint_as_float(w[e / 4][e % 4]);
        else return InFmt<T>::widen((uint16_t)(w[0][e / 2] >> (16 * (e % 2))));
    }
};
template <In T>
__device__ __forceinline__ Raw<T> load_raw(const typename InFmt<T>::S* row, int k, int K,
                                           bool vec) {
    using E = typename InFmt<T>::S;
    Raw<T> r;
    if (vec && k + 8 <= K) {
#pragma unroll
        for (int i = 0; i < Raw<T>::N; ++i)
            r.w[i] = *reinterpret_cast<const u32x4*>(row + k + i * (16 / sizeof(E)));
        return r;
    }
#pragma unroll
    for (int i = 0; i < Raw<T>::N; ++i)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if constexpr (T == In::F32) {
                const int j = k + 4 * i + d;
                r.w[i][d] = j < K ? __float_as_uint(row[j]) : 0u;
            } else {
                const int j = k + 2 * d;
                const uint32_t lo = j < K ? row[j] : 0u, hi = j + 1 < K ? row[j + 1] : 0u;
                r.w[i][d] = lo | (hi << 16);
            }
        }
    return r;
}

// Rows: four lanes per block, 8 elements (16 or 32 bytes) each, so a wave
// reads 16 blocks in one run and writes their 256 code and 16 scale bytes.
// UN runs are loaded before the first is used.  A run is one 16-byte piece of scales:
// its blocks past the row's last one are the pad bytes.
template <In T, int UN>
__global__ __launch_bounds__(NT) void quantize_rows_kernel(const void* Xv, int64_t ldx, int64_t runs,
                                                           int runs_per_row, int K, int nb,
                                                           uint8_t* Q, int64_t ldq, uint8_t* S,
                                                           int64_t lds, bool vec) {
    using E = typename InFmt<T>::S;
    const E* X = static_cast<const E*>(Xv);
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * (NT / 64) + (threadIdx.x >> 6);
    const int64_t waves = (int64_t)gridDim.x * (NT / 64);
    for (int64_t r0 = wave; r0 < runs; r0 += waves * UN) {
        Raw<T> x[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t run = r0 + waves * i;
            if (run < runs)
                x[i] = load_raw<T>(X + run / runs_per_row * ldx,
                                   (int)(run % runs_per_row) * (16 * kBlock) + 8 * lane, K, vec);
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t run = r0 + waves * i;
            if (run >= runs) break;
            float v[8];
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = x[i].get(e);
                top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
            }
            top = max(top, (uint32_t)__shfl_xor((int)top, 1));
            top = max(top, (uint32_t)__shfl_xor((int)top, 2));
            const uint32_t s = scale_of(top);
            const int64_t row = run / runs_per_row;
            const int blk = (int)(run % runs_per_row) * 16 + lane / 4;
            if (blk < nb)
                *reinterpret_cast<uint32_t*>(Q + row * ldq + (int64_t)blk * kChunk +
                                             4 * (lane % 4)) = encode8(v, s);
            if (lane % 4 == 0) S[row * lds + blk] = (uint8_t)(blk < nb ? s : 127u);
        }
    }
}

// Stored transposed (X is K x M, rows of op(X) down its columns): a workgroup
// takes TCOLS columns x TBLK blocks, a wave one block of all columns, a lane two
// neighbouring columns of it, so each load reads 256 or 512 bytes of a stored row and
// all 32 are in flight.  Codes and scales go through LDS to leave as runs of
// the rows of Q and S (chunk c of LDS row r at c ^ (r/2 % TBLK): the lanes
// of a wave write one chunk of every second row).
constexpr int TCOLS = 128, TBLK = 8, TNT = 64 * TBLK;
template <In T>
__global__ __launch_bounds__(TNT) void quantize_columns_kernel(const void* Xv, int64_t ldx, int M,
                                                               int K, int nb, int slots,
                                                               int tiles_m, uint8_t* Q,
                                                               int64_t ldq, uint8_t* S,
                                                               int64_t lds, bool pairs) {
    using E = typename InFmt<T>::S;
    using W = typename std::conditional<T == In::F32, u32x2, uint32_t>::type;  // two elements
    const E* X = static_cast<const E*>(Xv);
    __shared__ __attribute__((aligned(16))) uint8_t codes[TCOLS * TBLK * kChunk];
    __shared__ __attribute__((aligned(16))) uint8_t scales[TCOLS * TBLK];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i0 = (int)(blockIdx.x % tiles_m) * TCOLS, b0 = (int)(blockIdx.x / tiles_m) * TBLK;
    const int col = i0 + 2 * lane;  // and col + 1
    const int blk = b0 + wave, k0 = blk * kBlock;
    const E* p = X + (int64_t)k0 * ldx + col;
    W w[kBlock];
    if (pairs && i0 + TCOLS <= M && k0 + kBlock <= K) {
#pragma unroll
        for (int e = 0; e < kBlock; ++e) w[e] = *reinterpret_cast<const W*>(p + (int64_t)e * ldx);
    } else {
#pragma unroll
        for (int e = 0; e < kBlock; ++e) {
            const bool in = k0 + e < K;
            const E a = in && col < M ? p[(int64_t)e * ldx] : E(0);
            const E b = in && col + 1 < M ? p[(int64_t)e * ldx + 1] : E(0);
            if constexpr (T == In::F32) w[e] = u32x2{__float_as_uint(a), __float_as_uint(b)};
            else w[e] = a | ((uint32_t)b << 16);
        }
    }
    auto value = [&](int e, int c) {
        if constexpr (T == In::F32) return __uint_as_float(w[e][c]);
        else return InFmt<T>::widen((uint16_t)(w[e] >> (16 * c)));
    };
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kBlock; ++e) top = max(top, __float_as_uint(value(e, c)) & 0x7fffffffu);
        const uint32_t s = scale_of(top);
        u32x4 q;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = value(8 * d + e, c);
            q[d] = encode8(x, s);
        }
        const int r = 2 * lane + c;
        *reinterpret_cast<u32x4*>(codes + (r * TBLK + (wave ^ (lane % TBLK))) * kChunk) = q;
        scales[r * TBLK + wave] = (uint8_t)(blk < nb ? s : 127u);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < TCOLS * TBLK / TNT; ++e) {
        const int at = e * TNT + threadIdx.x, r = at / TBLK, chunk = at % TBLK;
        if (i0 + r < M && b0 + chunk < nb)
            *reinterpret_cast<u32x4*>(Q + (int64_t)(i0 + r) * ldq + (int64_t)(b0 + chunk) * kChunk) =
                *reinterpret_cast<const u32x4*>(codes +
                                                (r * TBLK + (chunk ^ (r / 2 % TBLK))) * kChunk);
    }
    static_assert(kScaleRow % TBLK == 0 && TBLK == 8, "a tile's scales are one 8-byte piece");
    if (threadIdx.x < TCOLS && i0 + (int)threadIdx.x < M && b0 < slots)
        *reinterpret_cast<u32x2*>(S + (int64_t)(i0 + threadIdx.x) * lds + b0) =
            *reinterpret_cast<const u32x2*>(scales + threadIdx.x * TBLK);
}

// Reading back: 16 bytes of output per lane (8 or 4 elements, a dword or half of
// codes), so that a wave's store is one run; UN of them loaded before the first is
// used.
template <In T, int UN>
__global__ __launch_bounds__(NT) void dequantize_kernel(const uint8_t* Q, int64_t ldq,
                                                        const uint8_t* S, int64_t lds,
                                                        int64_t groups, int per_row, int K,
                                                        void* Yv, int64_t ldy, bool vec) {
    using E = typename InFmt<T>::S;
    using C = typename std::conditional<T == In::F32, uint16_t, uint32_t>::type;
    constexpr int EL = 16 / sizeof(E);
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    E* Y = static_cast<E*>(Yv);
    const int64_t step = (int64_t)gridDim.x * NT;
    for (int64_t g0 = (int64_t)blockIdx.x * NT + threadIdx.x; g0 < groups; g0 += step * UN) {
        uint32_t q[UN], s[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t g = g0 + step * i;
            if (g < groups) {
                const int64_t row = g / per_row;
                const int c = (int)(g % per_row);
                q[i] = *reinterpret_cast<const C*>(Q + row * ldq + (int64_t)sizeof(C) * c);
                s[i] = S[row * lds + c / (kBlock / EL)];
            }
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t g = g0 + step * i;
            if (g >= groups) break;
            const float sc = scale_bits(s[i]);
            float v[8];
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], sc, 0);
            const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], sc, 1);
            const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], sc, 2);
            const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], sc, 3);
            v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
            v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
            const int k = (int)(g % per_row) * EL;
            E* y = Y + g / per_row * ldy + k;
            E o[EL];
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                if constexpr (T == In::F32) {
                    o[e] = v[e];
                } else if constexpr (T == In::BF16) {
                    const __bf16 x = (__bf16)v[e];
                    o[e] = __builtin_bit_cast(uint16_t, x);
                } else {
                    const _Float16 x = (_Float16)v[e];
                    o[e] = __builtin_bit_cast(uint16_t, x);
                }
            }
            if (vec && k + EL <= K) {
                u32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (T == In::F32) w[e] = __float_as_uint(o[e]);
                    else w[e] = o[2 * e] | ((uint32_t)o[2 * e + 1] << 16);
                }
                __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(y));
            } else {
#pragma unroll
                for (int e = 0; e < EL; ++e)
                    if (k + e < K) y[e] = o[e];
            }
        }
    }
}

unsigned grid_for(int64_t items, int per_wg) {
    const int64_t g = (items + per_wg - 1) / per_wg;
    return (unsigned)(g < 16384 ? g : 16384);  // grid-stride loops cover the rest
}

template <In T>
hipError_t quantize(bool trans, int M, int K, const void* X, int64_t ldx, uint8_t* Q, int64_t ldq,
                    uint8_t* S, int64_t lds, hipStream_t s) {
    constexpr int esz = T == In::F32 ? 4 : 2;
    const int nb = blocks(K), runs_per_row = (int)(scale_pitch(K) / kScaleRow);
    if (trans) {
        const int tiles_m = (int)(((int64_t)M + TCOLS - 1) / TCOLS);
        const int slots = runs_per_row * kScaleRow;
        const int64_t wgs = (int64_t)tiles_m * (slots / TBLK);
        if (!launchable(wgs, TNT)) return hipErrorInvalidConfiguration;
        const bool pairs = reinterpret_cast<uintptr_t>(X) % (2 * esz) == 0 && ldx % 2 == 0;
        hipLaunchKernelGGL(quantize_columns_kernel<T>, dim3((unsigned)wgs), dim3(TNT), 0, s, X,
                           ldx, M, K, nb, slots, tiles_m, Q, ldq, S, lds, pairs);
        return hipGetLastError();
    }
    const int64_t runs = (int64_t)M * runs_per_row;
    const bool vec = rows_16b_aligned(X, ldx, esz);
    hipLaunchKernelGGL((quantize_rows_kernel<T, 4>), dim3(grid_for(runs, NT / 64)), dim3(NT), 0, s,
                       X, ldx, runs, runs_per_row, K, nb, Q, ldq, S, lds, vec);
    return hipGetLastError();
}

template <In T>
hipError_t dequantize(int M, int K, const uint8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds,
                      void* Y, int64_t ldy, hipStream_t s) {
    constexpr int EL = T == In::F32 ? 4 : 8;
    const int per_row = (K + EL - 1) / EL;
    const int64_t groups = (int64_t)M * per_row;
    const bool vec = rows_16b_aligned(Y, ldy, T == In::F32 ? 4 : 2);
    hipLaunchKernelGGL((dequantize_kernel<T, 4>), dim3(grid_for(groups, NT)), dim3(NT), 0, s, Q,
                       ldq, S, lds, groups, per_row, K, Y, ldy, vec);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(In t, bool trans, int M, int K, const void* X, int64_t ldx, uint8_t* Q,
                           int64_t ldq, uint8_t* S, int64_t lds, hipStream_t s) {
    return t == In::F32    ? quantize<In::F32>(trans, M, K, X, ldx, Q, ldq, S, lds, s)
           : t == In::BF16 ? quantize<In::BF16>(trans, M, K, X, ldx, Q, ldq, S, lds, s)
                           : quantize<In::F16>(trans, M, K, X, ldx, Q, ldq, S, lds, s);
}

hipError_t launch_dequantize(In t, int M, int K, const uint8_t* Q, int64_t ldq, const uint8_t* S,
                             int64_t lds, void* Y, int64_t ldy, hipStream_t s) {
    return t == In::F32    ? dequantize<In::F32>(M, K, Q, ldq, S, lds, Y, ldy, s)
           : t == In::BF16 ? dequantize<In::BF16>(M, K, Q, ldq, S, lds, Y, ldy, s)
                           : dequantize<In::F16>(M, K, Q, ldq, S, lds, Y, ldy, s);
}

}  // namespace mx4
}  // namespace dgt
