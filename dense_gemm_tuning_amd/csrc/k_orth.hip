// k_orth.hip -- orthogonalisation by Newton-Schulz steps.
//
//     X <- G / (|G|_F + eps);   steps times:  S = X X^T,  X <- a X + (b S + c S S) X
//
// (M <= N; for M > N the same from the right: S = X^T X, X <- a X + X (b S + c S S),
// so no matrix is transposed in memory).  The three products of a step run on
// the library's FP16 tile kernels with fp32 sums.
//
// Rounding.  The products' operands are FP16.  Each step multiplies what
// rounding X adds in the weak singular directions by up to a (3.4 with the
// usual coefficients, 484 over five steps), so rounding X itself to 16 bits
// costs a result normwise 2 to 4e-3 against 1.7e-3 that its own bf16 rounding costs.
// X is therefore kept as two halves hi + lo (22 bits); the products read hi,
// the term a X both.  What hi's rounding E adds through the products reaches the
// weak directions only as (b S + c S S) E, small where S is, and the result
// is 1.7 to 2.4e-3 off (matrices of 256 to 1024, normal, low-rank and 1/i spectra).
//
// FP16's range: |X| <= |X|_2, about 1, but its elements are near
// 1/sqrt(max(M, N)) and the Gram matrix's smaller still, so X is held times
// 2^x_exp near that root, S times 2^12 and the polynomial times 2^10 (both at most
// about 13 * 2^10 for singular values up to 1.3); powers of two, so only the
// range moves.
#include <cmath>

#include "orth.hpp"

namespace dgt {
namespace orth {

namespace {

constexpr int NT = 256;
constexpr float kGramScale = 4096.0f;  // 2^12
constexpr float kPolyScale = 1024.0f;  // 2^10

int scale_exp(const Plan& p) {  // round(log2(sqrt(max(M, N))))
    return (int)std::lround(0.5 * std::log2((double)(p.M > p.N ? p.M : p.N)));
}

// kNormParts partial sums of squares per matrix, in 64 bits: workgroup x of
// matrix blockIdx.y sums elements x*NT + t, + kNormParts*NT, ...
template <In T>
__global__ __launch_bounds__(NT) void norm_kernel(const typename InFmt<T>::S* G, int64_t ldg,
                                                  int64_t stride, int M, int N, double* parts) {
    G += blockIdx.y * stride;
    const int64_t total = (int64_t)M * N;
    double sum = 0.0;
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < total;
         e += (int64_t)kNormParts * NT) {
        const double v = load_in<T>(G + e / N * ldg + e % N);
        sum += v * v;
    }
    __shared__ double red[NT];
    red[threadIdx.x] = sum;
    __syncthreads();
    for (int h = NT / 2; h > 0; h /= 2) {
        if ((int)threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
        __syncthreads();
    }
    if (threadIdx.x == 0) parts[(int64_t)blockIdx.y * kNormParts + blockIdx.x] = red[0];
}

struct Halves {
    _Float16 hi, lo;
};
__device__ __forceinline__ Halves split(float x) {
    Halves h;
    h.hi = (_Float16)x;
    h.lo = (_Float16)(x - (float)h.hi);
    return h;
}

// X <- G * 2^x_exp / (|G| + eps) as two halves; zeros in the padding columns.
template <In T>
__global__ __launch_bounds__(NT) void init_kernel(const typename InFmt<T>::S* G, int64_t ldg,
                                                  int64_t stride, int M, int N, const double* parts,
                                                  double eps, double scale, _Float16* hi,
                                                  _Float16* lo, int64_t ldx) {
    const int64_t z = blockIdx.y;
    G += z * stride;
    hi += z * M * ldx;
    lo += z * M * ldx;
    double sum = 0.0;
    for (int i = 0; i < kNormParts; ++i) sum += parts[z * kNormParts + i];
    const double inv = scale / (sqrt(sum) + eps);
    const int64_t total = (int64_t)M * ldx;
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * NT) {
        const int64_t row = e / ldx;
        const int col = (int)(e % ldx);
        const Halves h =
            split(col < N ? (float)((double)load_in<T>(G + row * ldg + col) * inv) : 0.0f);
        hi[e] = h.hi;
        lo[e] = h.lo;
    }
}

// S <- the Gram matrix's sums times f, in FP16.
__global__ __launch_bounds__(NT) void gram_kernel(const float* C, _Float16* S, int64_t total,
                                                  float f) {
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * NT)
        S[e] = (_Float16)(C[e] * f);
}

// B <- fb * S + fc * (sums of S*S), in FP16.
__global__ __launch_bounds__(NT) void poly_kernel(const float* C, const _Float16* S, _Float16* B,
                                                  int64_t total, float fb, float fc) {
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * NT)
        B[e] = (_Float16)(fb * (float)S[e] + fc * C[e]);
}

// X' <- a * (hi + lo) + f * sums: two halves, or the result (times out_scale)
// in bf16.
template <bool kLast>
__global__ __launch_bounds__(NT) void update_kernel(const float* C, const _Float16* hi,
                                                    const _Float16* lo, int M, int N, int64_t ldx,
                                                    float a, float f, _Float16* hi2, _Float16* lo2,
                                                    uint16_t* O, int64_t ldo, int64_t stride_o,
                                                    float out_scale) {
    const int64_t z = blockIdx.y, base = z * M * ldx;
    const int64_t total = (int64_t)M * ldx;
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * NT) {
        const int64_t row = e / ldx;
        const int col = (int)(e % ldx);
        const float x = a * ((float)hi[base + e] + (float)lo[base + e]) + f * C[base + e];
        if constexpr (kLast) {
            if (col < N)
                O[z * stride_o + row * ldo + col] =
                    __builtin_bit_cast(uint16_t, (__bf16)(x * out_scale));
        } else {
            const Halves h = split(col < N ? x : 0.0f);
            hi2[base + e] = h.hi;
            lo2[base + e] = h.lo;
        }
    }
}

unsigned grid_for(int64_t items) {
    const int64_t g = (items + NT - 1) / NT;
    return (unsigned)(g < 16384 ? g : 16384);  // grid-stride loops cover the rest
}

// C <- op(A) op(B), FP16 operands of a batch.
hipError_t product(const Plan& p, int M, int N, int K, const void* A, int64_t lda, int64_t sa,
                   int ta, const void* B, int64_t ldb, int64_t sb, int tb, float* C, int64_t ldc,
                   int64_t sc, hipStream_t s) {
    GemmParams g = {};
    g.M = M; g.N = N; g.K = K;
    g.alpha = 1.0f;
    g.A = A; g.lda = lda; g.stride_a = sa * 2; g.ta = ta;
    g.B = B; g.ldb = ldb; g.stride_b = sb * 2; g.tb = tb;
    g.C = C; g.ldc = ldc; g.stride_c = sc;
    g.batch = p.batch;
    return launch_mfma16<In::F16>(g, s);
}

template <In T>
void launch_init(const Plan& p, const Call& c, hipStream_t s) {
    using E = typename InFmt<T>::S;
    const E* G = static_cast<const E*>(c.G);
    double* parts = reinterpret_cast<double*>(c.ws + p.parts);
    hipLaunchKernelGGL(norm_kernel<T>, dim3(kNormParts, p.batch), dim3(NT), 0, s, G, c.ldg,
                       c.stride_g, p.M, p.N, parts);
    hipLaunchKernelGGL(init_kernel<T>, dim3(grid_for(p.x_size), p.batch), dim3(NT), 0, s, G, c.ldg,
                       c.stride_g, p.M, p.N, parts, (double)c.eps, std::ldexp(1.0, scale_exp(p)),
                       reinterpret_cast<_Float16*>(c.ws + p.hi[0]),
                       reinterpret_cast<_Float16*>(c.ws + p.lo[0]), p.ldx);
}

}  // namespace

hipError_t launch(const Plan& p, const Call& c, hipStream_t s) {
    if (c.t == In::F32) launch_init<In::F32>(p, c, s);
    else if (c.t == In::BF16) launch_init<In::BF16>(p, c, s);
    else launch_init<In::F16>(p, c, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const bool tall = p.M > p.N;
    const int n = p.s, large = tall ? p.M : p.N;
    _Float16* hi[2] = {reinterpret_cast<_Float16*>(c.ws + p.hi[0]),
                       reinterpret_cast<_Float16*>(c.ws + p.hi[1])};
    _Float16* lo[2] = {reinterpret_cast<_Float16*>(c.ws + p.lo[0]),
                       reinterpret_cast<_Float16*>(c.ws + p.lo[1])};
    _Float16* S = reinterpret_cast<_Float16*>(c.ws + p.gram);
    _Float16* B = reinterpret_cast<_Float16*>(c.ws + p.poly);
    float* C = reinterpret_cast<float*>(c.ws + p.c32);
    const float xs = std::ldexp(1.0f, scale_exp(p));
    const int64_t s_total = p.batch * p.s_size;
    for (int i = 0; i < c.steps; ++i) {
        const int r = i & 1, w = 1 - r;
        // S: rows of X against rows (wide), columns against columns (tall)
        e = product(p, n, n, large, hi[r], p.ldx, p.x_size, tall, hi[r], p.ldx, p.x_size, !tall, C,
                    p.lds, p.s_size, s);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(gram_kernel, dim3(grid_for(s_total)), dim3(NT), 0, s, C, S, s_total,
                           kGramScale / (xs * xs));
        // S is symmetric: its rows serve as the columns
        e = product(p, n, n, n, S, p.lds, p.s_size, 0, S, p.lds, p.s_size, 1, C, p.lds, p.s_size, s);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(poly_kernel, dim3(grid_for(s_total)), dim3(NT), 0, s, C, S, B, s_total,
                           c.b * (kPolyScale / kGramScale),
                           c.c * (kPolyScale / (kGramScale * kGramScale)));
        if (tall)
            e = product(p, p.M, p.N, n, hi[r], p.ldx, p.x_size, 0, B, p.lds, p.s_size, 1, C, p.ldx,
                        p.x_size, s);
        else
            e = product(p, p.M, p.N, n, B, p.lds, p.s_size, 0, hi[r], p.ldx, p.x_size, 0, C, p.ldx,
                        p.x_size, s);
        if (e != hipSuccess) return e;
        const dim3 grid(grid_for(p.x_size), p.batch);
        if (i + 1 == c.steps)
            hipLaunchKernelGGL(update_kernel<true>, grid, dim3(NT), 0, s, C, hi[r], lo[r], p.M, p.N,
                               p.ldx, c.a, 1.0f / kPolyScale, nullptr, nullptr, c.O, c.ldo,
                               c.stride_o, 1.0f / xs);
        else
            hipLaunchKernelGGL(update_kernel<false>, grid, dim3(NT), 0, s, C, hi[r], lo[r], p.M, p.N,
                               p.ldx, c.a, 1.0f / kPolyScale, hi[w], lo[w], nullptr, 0, 0, 1.0f);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace orth
}  // namespace dgt
