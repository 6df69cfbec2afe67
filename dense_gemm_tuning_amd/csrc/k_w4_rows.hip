// k_w4_rows.hip -- products of few rows with a weight in 4 bits, plain and
// gated.  A wavefront takes one output column and up to MB rows, each lane 8
// consecutive k at a time (a dword of codes): x*q and x are summed apart for
// each lane's piece, which lies in one group, and s*(sum xq - z * sum x) is added up.
#include "w4.hpp"

namespace dgt {
namespace w4 {

namespace {

constexpr int NT = 256, MB = 4;

// Sums of rows m0 .. m0+rows-1 of A with row n of the weight, in every lane.
template <In T>
__device__ __forceinline__ void row_sums(const uint16_t* A, int64_t lda, int K, int m0, int rows,
                                         const Weight& w, int64_t n, int lane, float (&out)[MB]) {
#pragma unroll
    for (int m = 0; m < MB; ++m) out[m] = 0.0f;
    for (int64_t k = 8 * lane; k < K; k += 512) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(w.Q + n * w.ldq + k / 2);
        const float s = scale_value(w.S[n * w.lds + (k >> w.log_group)], w.s_bf16);
        const float z = w.Z ? (float)w.Z[n * w.ldz + (k >> w.log_group)] : 8.0f;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (m >= rows) break;
            const uint16_t* x = A + (int64_t)(m0 + m) * lda + k;
            float sum = 0.0f, sx = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = k + e < K ? load_in<T>(x + e) : 0.0f;
                sum = fmaf(v, (float)((q >> (4 * e)) & 15u), sum);
                sx += v;
            }
            out[m] = fmaf(s, fmaf(-z, sx, sum), out[m]);
        }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
        for (int d = 32; d > 0; d /= 2) out[m] += __shfl_xor(out[m], d);
}

template <In T>
__global__ __launch_bounds__(NT) void product_kernel(Product p) {
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * (NT / 64) + (threadIdx.x >> 6);
    if (n >= p.N) return;
    for (int64_t m0 = (int64_t)blockIdx.y * MB; m0 < p.M; m0 += (int64_t)gridDim.y * MB) {
        const int rows = (int)min((int64_t)MB, p.M - m0);
        float sum[MB];
        row_sums<T>(p.A, p.lda, p.K, (int)m0, rows, p.w, n, lane, sum);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (m >= rows || lane != m) continue;
            float* c = p.C + (m0 + m) * p.ldc + n;
            const float r = p.beta == 0.0f ? p.alpha * sum[m] : p.alpha * sum[m] + p.beta * *c;
            *c = p.bias ? r + p.bias[n] : r;
        }
    }
}

template <In T>
__global__ __launch_bounds__(NT) void gated_kernel(Gated p) {
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * (NT / 64) + (threadIdx.x >> 6);
    if (n >= p.N) return;
    for (int64_t m0 = (int64_t)blockIdx.y * MB; m0 < p.M; m0 += (int64_t)gridDim.y * MB) {
        const int rows = (int)min((int64_t)MB, p.M - m0);
        float g[MB], u[MB];
        row_sums<T>(p.X, p.ldx, p.K, (int)m0, rows, p.w, n, lane, g);
        row_sums<T>(p.X, p.ldx, p.K, (int)m0, rows, p.w, p.N + n, lane, u);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (m >= rows || lane != m) continue;
            const float gv = g[m] + (p.bg ? p.bg[n] : 0.0f), uv = u[m] + (p.bu ? p.bu[n] : 0.0f);
            p.H[(m0 + m) * p.ldh + n] = gated::to_bits<T>(gated::act_of(p.act, gv) * uv);
        }
    }
}

dim3 grid(int M, int N) {
    const int64_t blocks_m = ((int64_t)M + MB - 1) / MB;
    return dim3((unsigned)(((int64_t)N + NT / 64 - 1) / (NT / 64)),
                (unsigned)(blocks_m < 65535 ? blocks_m : 65535));
}

}  // namespace

hipError_t launch_product(In t, const Product& p, hipStream_t s) {
    if (t == In::BF16) hipLaunchKernelGGL(product_kernel<In::BF16>, grid(p.M, p.N), dim3(NT), 0, s, p);
    else hipLaunchKernelGGL(product_kernel<In::F16>, grid(p.M, p.N), dim3(NT), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_gated(In t, const Gated& p, hipStream_t s) {
    if (t == In::BF16) hipLaunchKernelGGL(gated_kernel<In::BF16>, grid(p.M, p.N), dim3(NT), 0, s, p);
    else hipLaunchKernelGGL(gated_kernel<In::F16>, grid(p.M, p.N), dim3(NT), 0, s, p);
    return hipGetLastError();
}

}  // namespace w4
}  // namespace dgt
