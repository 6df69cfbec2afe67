// k_w4_quant.hip -- quantising to 4 bits with a scale per group, and reading
// back.  Bound by HBM: an element is read once (2 or 4 bytes) and half a byte
// written, or the other way round.
//
// Per group, over its elements and zero: with zero points s = (max - min)/15 and z the
// whole number nearest to -min/s, at most 15 (s may have been rounded down); without,
// s = max(max/7, -min/8) and z = 8.
// The quotient that s is rounded from is taken in 64 bits; s is rounded to fp32, then
// to its 16-bit type (past that type's largest value: that value).  q = the
// whole number nearest to x/s, ties to even, plus z, within 0 .. 15.
#include "w4.hpp"

namespace dgt {
namespace w4 {

namespace {

constexpr int NT = 256;

// Eight elements of a row as raw bits (fp32: two pieces), zeros past K.
template <In T>
struct Raw {
    static constexpr int N = T == In::F32 ? 2 : 1;
    u32x4 w[N];
    __device__ float get(int e) const {
        if constexpr (T == In::F32) return __uint_as_float(w[e / 4][e % 4]);
        else return InFmt<T>::widen((uint16_t)(w[0][e / 2] >> (16 * (e % 2))));
    }
    __device__ void load(const typename InFmt<T>::S* row, int k, int K, bool vec) {
        if (vec && k + 8 <= K) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = *reinterpret_cast<const u32x4*>(row + k + i * (8 / N));
            return;
        }
#pragma unroll
        for (int e = 0; e < 4 * N; ++e) {
            if constexpr (T == In::F32) {
                w[e / 4][e % 4] = k + e < K ? __float_as_uint(row[k + e]) : 0u;
            } else {
                const uint32_t lo = k + 2 * e < K ? row[k + 2 * e] : 0u;
                const uint32_t hi = k + 2 * e + 1 < K ? row[k + 2 * e + 1] : 0u;
                w[0][e] = lo | (hi << 16);
            }
        }
    }
};

// The whole number nearest to x/s is q = rint(x * (1/s)) in fp32 unless x/s is half
// way between two whole numbers, or so near to it that fp32's product is on the
// other side.  What is left of x under q, rest, is exact (q has few bits and q*s is near x),
// and |rest| < s/2 says that q is right.  Otherwise this decides, ties to
// even.  Quotients past 16 need no care: the code is bounded there.
__device__ __forceinline__ float settle(float q, float rest, float half) {
    const bool odd = ((int)fminf(fmaxf(q, -32.0f), 32.0f) & 1) != 0;
    if (rest > half || (rest == half && odd)) q += 1.0f;
    else if (rest < -half || (rest == -half && odd)) q -= 1.0f;
    return q;
}

// A lane takes 8 neighbouring elements, group/8 lanes a group, a wavefront 512
// elements of a row (a run); UN runs are loaded before the first is used.
template <In T, int UN>
__global__ __launch_bounds__(NT) void quantize_kernel(const void* Xv, int64_t ldx, int64_t runs,
                                                      int runs_per_row, int K, uint8_t* Q,
                                                      int64_t ldq, uint16_t* S, int64_t lds,
                                                      uint8_t* Z, int64_t ldz, bool s_bf16,
                                                      int log_group, bool vec) {
    using E = typename InFmt<T>::S;
    const E* X = static_cast<const E*>(Xv);
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * (NT / 64) +
                         __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t waves = (int64_t)gridDim.x * (NT / 64);
    const int code_end = 32 * (K / 32 + (K % 32 != 0));
    // row and place in the row of the wavefront's next run, and their steps
    int64_t row_at = wave / runs_per_row;
    int at = (int)(wave % runs_per_row);
    const int64_t row_step = waves / runs_per_row;
    const int at_step = (int)(waves % runs_per_row);
    for (int64_t r0 = wave; r0 < runs; r0 += waves * UN) {
        Raw<T> x[UN];
        int64_t rows[UN];
        int ks[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            rows[i] = row_at;
            ks[i] = at * 512 + 8 * lane;
            if (r0 + waves * i < runs) x[i].load(X + row_at * ldx, ks[i], K, vec);
            row_at += row_step;
            at += at_step;
            if (at >= runs_per_row) at -= runs_per_row, ++row_at;
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            if (r0 + waves * i >= runs) break;
            const int64_t row = rows[i];
            const int k = ks[i];
            float v[8], top = 0.0f, low = 0.0f, bad = 0.0f;  // bad: NaN with an infinity or a NaN
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = x[i].get(e);
                top = fmaxf(top, v[e]);
                low = fminf(low, v[e]);
                bad = fmaf(v[e], 0.0f, bad);
            }
            for (int d = 1; d < 1 << (log_group - 3); d *= 2) {
                top = fmaxf(top, __shfl_xor(top, d));
                low = fminf(low, __shfl_xor(low, d));
                bad += __shfl_xor(bad, d);
            }
            const bool finite = bad == 0.0f;
            const double hi = top, lo = -(double)low;
            float wide = (float)(Z ? (hi + lo) / 15.0 : fmax(hi / 7.0, lo / 8.0));
            // two roundings, as documented: the compiler would join them into one
            asm("" : "+v"(wide));
            uint16_t bits = s_bf16 ? gated::to_bits<In::BF16>(wide) : gated::to_bits<In::F16>(wide);
            const uint16_t inf = s_bf16 ? 0x7f80 : 0x7c00;
            if (bits == inf) bits = inf - 1;
            const float s = scale_value(bits, s_bf16);
            const float unit = s > 0.0f ? s : 1.0f;  // a group of zeros, or below the type's least
            // the reciprocal of a scale below 2^-100 may be too large for fp32
            const float up = unit < 0x1p-100f ? 0x1p64f : 1.0f, su = up * unit;
            const float inv = __builtin_amdgcn_rcpf(su), half = 0.5f * su;
            float z = 8.0f;
            if (Z) {
                const float q = rintf(-low * up * inv);
                z = fminf(settle(q, fmaf(-q, su, -low * up), half), 15.0f);
            }
            if (!finite) bits = inf | 1;
            float q[8], most = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= up;
                q[e] = v[e] * inv;
                if constexpr (T == In::F32) {
                    q[e] = rintf(q[e]);
                    most = fmaxf(most, fabsf(fmaf(-q[e], su, v[e])));
                } else {
                    // Of 16-bit elements, half ways are common and everything
                    // else is 2^-19 or more away: with the quotient's error taken
                    // out they come out as they are.
                    q[e] = rintf(fmaf(fmaf(-q[e], su, v[e]), inv, q[e]));
                }
            }
            if (T == In::F32 && !(most < half)) {  // rare
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = settle(q[e], fmaf(-q[e], su, v[e]), half);
            }
            uint32_t codes = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                codes |= (uint32_t)fminf(fmaxf(q[e] + z, 0.0f), 15.0f) << (4 * e);
            if (!finite) codes = 0;
            if (k + 8 > K) codes &= k < K ? (1u << (4 * (K - k))) - 1u : 0u;
            if (k < code_end) *reinterpret_cast<uint32_t*>(Q + row * ldq + k / 2) = codes;
            if (k < K && (k & ((1 << log_group) - 1)) == 0) {
                S[row * lds + (k >> log_group)] = bits;
                if (Z) Z[row * ldz + (k >> log_group)] = finite ? (uint8_t)z : 0;
            }
        }
    }
}

// Reading back: 16 bytes of output per lane, so that a wave's store is one run;
// UN of them loaded before the first is used.
template <In T, int UN>
__global__ __launch_bounds__(NT) void dequantize_kernel(Weight w, int64_t pieces, int per_row, int K,
                                                        void* Yv, int64_t ldy, bool vec) {
    using E = typename InFmt<T>::S;
    using C = typename std::conditional<T == In::F32, uint16_t, uint32_t>::type;
    constexpr int EL = 16 / sizeof(E);
    E* Y = static_cast<E*>(Yv);
    const int64_t step = (int64_t)gridDim.x * NT;
    for (int64_t p0 = (int64_t)blockIdx.x * NT + threadIdx.x; p0 < pieces; p0 += step * UN) {
        uint32_t q[UN], s[UN], z[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t p = p0 + step * i;
            if (p < pieces) {
                const int64_t row = p / per_row;
                const int k = (int)(p % per_row) * EL;
                q[i] = *reinterpret_cast<const C*>(w.Q + row * w.ldq + k / 2);
                s[i] = w.S[row * w.lds + (k >> w.log_group)];
                z[i] = w.Z ? w.Z[row * w.ldz + (k >> w.log_group)] : 8u;
            }
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t p = p0 + step * i;
            if (p >= pieces) break;
            const int k = (int)(p % per_row) * EL;
            const float sc = scale_value(s[i], w.s_bf16);
            E* y = Y + p / per_row * ldy + k;
            E o[EL];
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                const float v = sc * (float)((int)((q[i] >> (4 * e)) & 15u) - (int)z[i]);
                if constexpr (T == In::F32) o[e] = v;
                else o[e] = gated::to_bits<T>(v);
            }
            if (vec && k + EL <= K) {
                u32x4 out;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (T == In::F32) out[e] = __float_as_uint(o[e]);
                    else out[e] = o[2 * e] | ((uint32_t)o[2 * e + 1] << 16);
                }
                __builtin_nontemporal_store(out, reinterpret_cast<u32x4*>(y));
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
hipError_t quantize(int M, int K, const void* X, int64_t ldx, uint8_t* Q, int64_t ldq, uint16_t* S,
                    int64_t lds, uint8_t* Z, int64_t ldz, bool s_bf16, int log_group,
                    hipStream_t s) {
    const int runs_per_row = (int)(((int64_t)K + 511) / 512);
    const int64_t runs = (int64_t)M * runs_per_row;
    const bool vec = rows_16b_aligned(X, ldx, T == In::F32 ? 4 : 2);
    hipLaunchKernelGGL((quantize_kernel<T, 4>), dim3(grid_for(runs, NT / 64)), dim3(NT), 0, s, X,
                       ldx, runs, runs_per_row, K, Q, ldq, S, lds, Z, ldz, s_bf16, log_group, vec);
    return hipGetLastError();
}

template <In T>
hipError_t dequantize(int M, int K, const Weight& w, void* Y, int64_t ldy, hipStream_t s) {
    constexpr int EL = T == In::F32 ? 4 : 8;
    const int per_row = (K + EL - 1) / EL;
    const int64_t pieces = (int64_t)M * per_row;
    const bool vec = rows_16b_aligned(Y, ldy, T == In::F32 ? 4 : 2);
    hipLaunchKernelGGL((dequantize_kernel<T, 4>), dim3(grid_for(pieces, NT)), dim3(NT), 0, s, w,
                       pieces, per_row, K, Y, ldy, vec);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(In t, int M, int K, const void* X, int64_t ldx, uint8_t* Q, int64_t ldq,
                           uint16_t* S, int64_t lds, uint8_t* Z, int64_t ldz, bool s_bf16,
                           int log_group, hipStream_t s) {
    auto go = [&](auto f) { return f(M, K, X, ldx, Q, ldq, S, lds, Z, ldz, s_bf16, log_group, s); };
    return t == In::F32 ? go(quantize<In::F32>) : t == In::BF16 ? go(quantize<In::BF16>)
                                                               : go(quantize<In::F16>);
}

hipError_t launch_dequantize(In t, int M, int K, const Weight& w, void* Y, int64_t ldy,
                             hipStream_t s) {
    return t == In::F32    ? dequantize<In::F32>(M, K, w, Y, ldy, s)
           : t == In::BF16 ? dequantize<In::BF16>(M, K, w, Y, ldy, s)
                           : dequantize<In::F16>(M, K, w, Y, ldy, s);
}

}  // namespace w4
}  // namespace dgt
