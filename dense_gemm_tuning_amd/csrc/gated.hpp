// gated.hpp -- gated projections of a feed-forward block and their gradient:
// what the kernels (k_gated_*.hip) and the entry points (gated_api.cpp) share.
//
//   g = X*Wg^T + bg,  u = X*Wu^T + bu,  H = act(g) * u        (weights N x K)
//   dh = dY*Wd,  dG = dh * u * act'(g),  dU = dh * act(g)     (Wd K x N)
//
// Products are summed in fp32, and everything between the sums and the stored
// 16-bit values is fp32.
#pragma once

#include "gemm_common.hpp"

namespace dgt {
namespace gated {

enum class Act { Silu, Gelu, GeluTanh, Relu, Sigmoid, Identity };

struct Forward {
    Act act;
    int M, N, K;
    const uint16_t *X, *Wg, *Wu;
    int64_t ldx, ldwg, ldwu;  // elements, as all pitches here
    const float *bg, *bu;     // optional
    uint16_t *H, *G, *U;      // G, U optional: the pre-activations
    int64_t ldh, ldg, ldu;
};

struct Grad {
    Act act;
    int M, N, K;
    const uint16_t *dY, *Wd, *G, *U;
    int64_t lddy, ldw, ldg, ldu;
    uint16_t *dG, *dU, *H;  // H optional: act(g) * u again; dG may be G and dU may be U
    int64_t lddg, lddu, ldh;
    // Column sums of dG and dU over runs of rows, for the biases' gradients
    // (optional): run r's sums of dG at parts + 2*r*N, of dU N floats later.
    float* parts;
};

// Rows whose column sums one part holds, at least (a wavefront's share of a
// tile), and the parts of M rows when tiles of `tile` rows are two
// wavefronts high.
constexpr int kPartRows = 64;
inline int64_t parts_for(int M, int tile) { return 2 * (((int64_t)M + tile - 1) / tile); }

// 16 bytes from wherever they start.
__device__ __forceinline__ u32x4 load16(const uint16_t* from) {
    u32x4 v;
    __builtin_memcpy(&v, from, 16);
    return v;
}

// Elements [at, at + 8) of a row of fewer than 8, zeros behind it (limit >= 1).
__device__ __forceinline__ u32x4 gather8(const uint16_t* row, int at, int limit) {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = row[min(at + i, limit - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = at + i < limit ? e[i] : 0u;
    return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
}

// The 8 elements from `past` (0 .. 8) on, zeros behind them.  A piece that crosses a row's end is
// the row's last 8 elements so shifted: its load needs no branch, behind which it would wait
// for the others.
__device__ __forceinline__ u32x4 shift_out(u32x4 v, int past) {
#pragma unroll
    for (int d = 0; d < 4; ++d)
        if (past & 1) v[d] = (v[d] >> 16) | (d < 3 ? v[(d + 1) % 4] << 16 : 0u);
#pragma unroll
    for (int d = 0; d < 4; ++d)
        if (past & 2) v[d] = d < 3 ? v[(d + 1) % 4] : 0u;
#pragma unroll
    for (int d = 0; d < 4; ++d)
        if (past & 4) v[d] = d < 2 ? v[(d + 2) % 4] : 0u;
#pragma unroll
    for (int d = 0; d < 4; ++d)
        if (past & 8) v[d] = 0u;
    return v;
}

// t = exp(-|x|) and the logistic function of x and of -x from it: no
// cancellation on either side.  The reciprocal is the hardware's, to 1 ulp like
// exp2, and the argument's rounding adds |x| * 2^-24: what is computed from
// them is stored in 16 bits, or summed over rows.
struct Logistic {
    float pos, neg;  // of x, of -x
};
__device__ __forceinline__ Logistic logistic(float x) {
    const float t = __builtin_exp2f(-1.44269504f * fabsf(x));  // keeps subnormal results
    const float r = __builtin_amdgcn_rcpf(1.0f + t), q = t * r;
    return x >= 0.0f ? Logistic{r, q} : Logistic{q, r};
}

constexpr float kTanhA = 1.59576912f;              // 2 * sqrt(2/pi)
constexpr float kTanhB = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228f;

// P(normal variable < x) and exp(-x^2/2).  The tail below -|x| is exp(-x^2/2)/2 times t
// times a polynomial in t = 1/(1 + 0.4|x|): a least-maximum fit of erfcx(|x|/sqrt 2)/t over
// 0 < t <= 1 in 64 bits.  Its relative error with the coefficients as fp32 holds them is 1.43e-7, and
// 4.0e-7 evaluated in fp32 with t rounded once (the hardware's reciprocal adds its ulp); the exponential's
// argument is rounded twice, which adds x^2 roundoffs (6e-8 x^2).  (A tail as 1 - P(x < |x|) would lose its
// digits.)
struct Normal {
    float below, bell;
};
__device__ __forceinline__ Normal normal(float x) {
    const float bell = __builtin_exp2f(-0.72134752f * (x * x));
    const float t = __builtin_amdgcn_rcpf(fmaf(0.4f, fabsf(x), 1.0f));
    float q = 0.046239819f;
    q = fmaf(q, t, -0.26906604f);
    q = fmaf(q, t, 0.59885973f);
    q = fmaf(q, t, -0.56983966f);
    q = fmaf(q, t, 0.12439930f);
    q = fmaf(q, t, -0.0086596236f);
    q = fmaf(q, t, 0.17206378f);
    q = fmaf(q, t, 0.26768470f);
    q = fmaf(q, t, 0.31916407f);
    q = fmaf(q, t, 0.31915379f);
    const float tail = 0.5f * bell * t * q;
    return Normal{x < 0.0f ? tail : 1.0f - tail, bell};
}

// act(x), and with kSlope its derivative.  A NaN stays one.
template <bool kSlope>
__device__ __forceinline__ float act_at(Act act, float x, float& slope) {
    switch (act) {
        case Act::Silu: {
            const Logistic s = logistic(x);
            if (kSlope) slope = s.pos * fmaf(x, s.neg, 1.0f);
            return x * s.pos;
        }
        case Act::Gelu: {
            const Normal n = normal(x);
            if (kSlope) slope = fmaf(x * kInvSqrt2Pi, n.bell, n.below);
            return x * n.below;
        }
        case Act::GeluTanh: {  // 0.5 * x * (1 + tanh(y/2)) = x * logistic(y)
            const float x2 = x * x;
            const Logistic s = logistic(kTanhA * x * fmaf(kTanhB, x2, 1.0f));
            if (kSlope) {  // x bounded: s.neg or s.pos is zero from |x| = 12 on, and products with x would overflow
                const float b = fminf(fmaxf(x, -64.0f), 64.0f);
                slope = s.pos * fmaf(b * s.neg, kTanhA * fmaf(3.0f * kTanhB, b * b, 1.0f), 1.0f);
            }
            return x * s.pos;
        }
        case Act::Relu:
            if (kSlope) slope = x > 0.0f ? 1.0f : 0.0f;
            return x < 0.0f ? 0.0f : x;
        case Act::Sigmoid: {
            const Logistic s = logistic(x);
            if (kSlope) slope = s.pos * s.neg;
            return s.pos;
        }
        default:
            if (kSlope) slope = 1.0f;
            return x;
    }
}
__device__ __forceinline__ float act_of(Act act, float x) {
    float unused;
    return act_at<false>(act, x, unused);
}

// An fp32 value as the bits of a 16-bit format, to nearest even.
template <In T>
__device__ __forceinline__ uint16_t to_bits(float x) {
    if constexpr (T == In::BF16) {
        const __bf16 y = (__bf16)x;
        return __builtin_bit_cast(uint16_t, y);
    } else {
        const _Float16 y = (_Float16)x;
        return __builtin_bit_cast(uint16_t, y);
    }
}

// dg, du and h of one element.
struct GradOut {
    float dg, du, h;
};
__device__ __forceinline__ GradOut grad_at(Act act, float dh, float g, float u) {
    float slope;
    const float a = act_at<true>(act, g, slope);
    return GradOut{dh * u * slope, dh * a, a * u};
}

// Launchers.  The register-staged ones take any operands; the grad ones say how
// many rows of parts they wrote.
template <In T> hipError_t launch_forward_regs(const Forward& p, hipStream_t s);
template <In T> hipError_t launch_grad_regs(const Grad& p, int64_t* parts, hipStream_t s);
// out[n] <- the sums over `parts` parts (either pointer may be null).
hipError_t launch_join(const float* parts, int64_t n_parts, int N, float* dbg, float* dbu,
                       hipStream_t s);
bool strip_eligible(const Forward& p);
template <In T> hipError_t launch_forward_strip(const Forward& p, hipStream_t s);
template <In T> hipError_t launch_forward(const Forward& p, hipStream_t s);
template <In T> hipError_t launch_grad(const Grad& p, int64_t* parts, hipStream_t s);

}  // namespace gated
}  // namespace dgt
