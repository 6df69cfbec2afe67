// gated_api.cpp -- the C entry points of the gated projections, their
// gradient, and the weights in 4 bits with group scales (include/dgt_gemm.h):
// host-side argument checks and the launch on the caller's stream.  Nothing
// here allocates, synchronises or keeps state, and the checks run before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_common.hpp"
#include "gated.hpp"
#include "w4.hpp"

namespace {

using namespace dgt::api;
namespace gated = dgt::gated;
namespace w4 = dgt::w4;

// Sizes stay clear of int's end by the kernels' tiles, and launches of the
// limit of 2^32 threads where they go by one size.
constexpr int kMaxDim = DGT_GEMM_GATED_MAX_DIM;

dgt::In in_of(DType t) {
    return t == DType::F32 ? dgt::In::F32 : t == DType::BF16 ? dgt::In::BF16 : dgt::In::F16;
}

bool dtype16_of(int dtype, DType& t) { return dtype_of(dtype, t) && t != DType::F32; }

bool act_of(int act, gated::Act& a) {
    if (act < GEMM_ACT_SILU || act > GEMM_ACT_IDENTITY) return false;
    a = static_cast<gated::Act>(act);
    return true;
}
static_assert((int)gated::Act::Silu == GEMM_ACT_SILU && (int)gated::Act::Gelu == GEMM_ACT_GELU &&
                  (int)gated::Act::GeluTanh == GEMM_ACT_GELU_TANH &&
                  (int)gated::Act::Relu == GEMM_ACT_RELU &&
                  (int)gated::Act::Sigmoid == GEMM_ACT_SIGMOID &&
                  (int)gated::Act::Identity == GEMM_ACT_IDENTITY,
              "the header's activations");

bool dims_ok(int M, int N, int K) {
    return M >= 0 && N >= 0 && K >= 0 && M <= kMaxDim && N <= kMaxDim && K <= kMaxDim;
}

// A row-major operand's memory: `rows` rows of `bytes` bytes, `pitch` apart.
struct Rows {
    uintptr_t at;
    int64_t rows, bytes, pitch;
};
Rows rows_of(const void* p, int rows, int64_t cols, int64_t ld, int esz) {
    return Rows{reinterpret_cast<uintptr_t>(p), p ? rows : 0, cols * esz, ld * esz};
}
// Whether two operands share a byte.  Operands of one pitch whose rows lie side
// by side (column ranges of one matrix) do not, though their ranges cross.
bool share(const Rows& a, const Rows& b) {
    if (a.rows == 0 || b.rows == 0 || a.bytes == 0 || b.bytes == 0) return false;
    const uint64_t a_end = a.at + (uint64_t)(a.rows - 1) * a.pitch + a.bytes;
    const uint64_t b_end = b.at + (uint64_t)(b.rows - 1) * b.pitch + b.bytes;
    if (a.at >= b_end || b.at >= a_end) return false;
    if (a.pitch != b.pitch) return true;
    const int64_t d = (int64_t)(b.at - a.at) % a.pitch, off = d < 0 ? d + a.pitch : d;
    return off < a.bytes || off + b.bytes > a.pitch;  // off: of b's rows after a's
}
bool same(const Rows& a, const Rows& b) {
    return a.at == b.at && (a.pitch == b.pitch || a.rows <= 1);
}

int status_of(hipError_t e) {
    return e == hipSuccess                      ? GEMM_OK
           : e == hipErrorInvalidConfiguration ? GEMM_ERR_DIM  // more workgroups than a launch holds
                                               : GEMM_ERR_LAUNCH;
}

// ---- 4-bit weights

int log_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : -1; }

bool scale_type(int t, bool& bf16) {
    bf16 = t == GEMM_DTYPE_BF16;
    return bf16 || t == GEMM_DTYPE_F16;
}

// Pitches of a weight of K columns (ldz is looked at where there are zero points).
bool pitches_ok(int K, int lg, int ldq, int lds, bool zeros, int ldz) {
    const int g = std::max(1, w4::groups(K, lg));
    return ldq >= std::max<int64_t>(1, dgt::mx4::code_pitch(K)) && ldq <= DGT_GEMM_MX4_MAX_PITCH &&
           lds >= g && (!zeros || ldz >= g);
}
bool aligned(const void* Q, int ldq, const void* S) {
    return (reinterpret_cast<uintptr_t>(Q) | (uintptr_t)ldq) % 16 == 0 &&
           reinterpret_cast<uintptr_t>(S) % 2 == 0;
}
struct WeightRows {
    Rows q, s, z;
};
WeightRows weight_rows(int rows, int K, int lg, const void* Q, int ldq, const void* S, int lds,
                       const void* Z, int ldz) {
    const int g = w4::groups(K, lg);
    return WeightRows{rows_of(Q, rows, dgt::mx4::code_pitch(K), ldq, 1), rows_of(S, rows, g, lds, 2),
                      rows_of(Z, rows, g, ldz, 1)};
}
bool share(const Rows& a, const WeightRows& w) { return share(a, w.q) || share(a, w.s) || share(a, w.z); }

w4::Weight weight_of(const uint8_t* Q, int ldq, const void* S, int lds, const uint8_t* Z, int ldz,
                     bool bf16, int lg) {
    return w4::Weight{Q, ldq, static_cast<const uint16_t*>(S), lds, Z, ldz, bf16, lg};
}

}  // namespace

extern "C" {

int gemm_gated(int dtype, int act, int M, int N, int K, const uint16_t* X, int ldx,
               const uint16_t* Wg, int ldwg, const uint16_t* Wu, int ldwu, const float* bias_g,
               const float* bias_u, uint16_t* H, int ldh, uint16_t* G, int ldg, uint16_t* U, int ldu,
               void* stream) {
    DType t;
    gated::Forward p;
    if (!dtype16_of(dtype, t) || !act_of(act, p.act)) return GEMM_ERR_ARG;
    if (!dims_ok(M, N, K)) return GEMM_ERR_DIM;
    const int k1 = std::max(1, K), n1 = std::max(1, N);
    if (ldx < k1 || ldwg < k1 || ldwu < k1 || ldh < n1 || (G && ldg < n1) || (U && ldu < n1))
        return GEMM_ERR_LD;
    if (M == 0 || N == 0) return GEMM_OK;
    if (H == nullptr || (K > 0 && (X == nullptr || Wg == nullptr || Wu == nullptr)))
        return GEMM_ERR_NULL;
    const Rows out[3] = {rows_of(H, M, N, ldh, 2), rows_of(G, M, N, ldg, 2), rows_of(U, M, N, ldu, 2)};
    const Rows in[5] = {rows_of(X, M, K, ldx, 2), rows_of(Wg, N, K, ldwg, 2),
                        rows_of(Wu, N, K, ldwu, 2), rows_of(bias_g, 1, N, N, 4),
                        rows_of(bias_u, 1, N, N, 4)};
    for (const Rows& o : out)
        for (const Rows& i : in)
            if (share(o, i)) return GEMM_ERR_OVERLAP;
    if (share(out[0], out[1]) || share(out[0], out[2]) || share(out[1], out[2]))
        return GEMM_ERR_OVERLAP;
    p.M = M; p.N = N; p.K = K;
    p.X = X; p.ldx = ldx;
    p.Wg = Wg; p.ldwg = ldwg;
    p.Wu = Wu; p.ldwu = ldwu;
    p.bg = bias_g; p.bu = bias_u;
    p.H = H; p.ldh = ldh;
    p.G = G; p.ldg = ldg;
    p.U = U; p.ldu = ldu;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return status_of(t == DType::BF16 ? gated::launch_forward<dgt::In::BF16>(p, s)
                                      : gated::launch_forward<dgt::In::F16>(p, s));
}

int64_t gemm_gated_grad_workspace_size(int M, int N) {
    if (!dims_ok(M, N, 0)) return GEMM_ERR_DIM;
    if (M == 0 || N == 0) return 0;
    return gated::parts_for(M, 2 * gated::kPartRows) * 2 * N * (int64_t)sizeof(float);
}

int gemm_gated_grad(int dtype, int act, int M, int N, int K, const uint16_t* dY, int lddy,
                    const uint16_t* Wd, int ldw, const uint16_t* G, int ldg, const uint16_t* U,
                    int ldu, uint16_t* dG, int lddg, uint16_t* dU, int lddu, uint16_t* H, int ldh,
                    float* dbias_g, float* dbias_u, void* workspace, int64_t workspace_bytes,
                    void* stream) {
    DType t;
    gated::Grad p;
    if (!dtype16_of(dtype, t) || !act_of(act, p.act) || workspace_bytes < 0) return GEMM_ERR_ARG;
    if (!dims_ok(M, N, K)) return GEMM_ERR_DIM;
    const int k1 = std::max(1, K), n1 = std::max(1, N);
    if (lddy < k1 || ldw < n1 || ldg < n1 || ldu < n1 || lddg < n1 || lddu < n1 || (H && ldh < n1))
        return GEMM_ERR_LD;
    if (N == 0) return GEMM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool sums = dbias_g != nullptr || dbias_u != nullptr;
    const Rows bias[2] = {rows_of(dbias_g, 1, N, N, 4), rows_of(dbias_u, 1, N, N, 4)};
    if (share(bias[0], bias[1])) return GEMM_ERR_OVERLAP;
    if (M == 0)  // sums over no rows
        return sums ? status_of(gated::launch_join(nullptr, 0, N, dbias_g, dbias_u, s)) : GEMM_OK;
    if (G == nullptr || U == nullptr || dG == nullptr || dU == nullptr ||
        (K > 0 && (dY == nullptr || Wd == nullptr)))
        return GEMM_ERR_NULL;
    const int64_t need = sums ? gemm_gated_grad_workspace_size(M, N) : 0;
    if (sums && (workspace == nullptr || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
    if (sums && reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return GEMM_ERR_ALIGN;
    const Rows ws = Rows{reinterpret_cast<uintptr_t>(workspace), sums ? 1 : 0, need, need};
    const Rows out[5] = {rows_of(dG, M, N, lddg, 2), rows_of(dU, M, N, lddu, 2),
                         rows_of(H, M, N, ldh, 2), bias[0], bias[1]};
    const Rows in[4] = {rows_of(G, M, N, ldg, 2), rows_of(U, M, N, ldu, 2),
                        rows_of(dY, M, K, lddy, 2), rows_of(Wd, K, N, ldw, 2)};
    for (int o = 0; o < 5; ++o) {
        for (int i = 0; i < 4; ++i)
            if (share(out[o], in[i]) && !(i < 2 && o == i && same(out[o], in[i])))  // dG on G, dU on U
                return GEMM_ERR_OVERLAP;
        for (int q = 0; q < o; ++q)
            if (share(out[o], out[q])) return GEMM_ERR_OVERLAP;
        if (share(out[o], ws)) return GEMM_ERR_OVERLAP;
    }
    for (const Rows& i : in)
        if (share(i, ws)) return GEMM_ERR_OVERLAP;
    p.M = M; p.N = N; p.K = K;
    p.dY = dY; p.lddy = lddy;
    p.Wd = Wd; p.ldw = ldw;
    p.G = G; p.ldg = ldg;
    p.U = U; p.ldu = ldu;
    p.dG = dG; p.lddg = lddg;
    p.dU = dU; p.lddu = lddu;
    p.H = H; p.ldh = ldh;
    p.parts = sums ? static_cast<float*>(workspace) : nullptr;
    int64_t parts = 0;
    const hipError_t e = t == DType::BF16 ? gated::launch_grad<dgt::In::BF16>(p, &parts, s)
                                          : gated::launch_grad<dgt::In::F16>(p, &parts, s);
    if (e != hipSuccess || !sums) return status_of(e);
    return status_of(gated::launch_join(p.parts, parts, N, dbias_g, dbias_u, s));
}

int gemm_w4_quantize(int dtype, int group, int scale_dtype, int M, int K, const void* X, int ldx,
                     uint8_t* Q, int ldq, void* S, int lds, uint8_t* Z, int ldz, void* stream) {
    DType t;
    bool bf16;
    const int lg = log_of(group);
    if (!dtype_of(dtype, t) || lg < 0 || !scale_type(scale_dtype, bf16)) return GEMM_ERR_ARG;
    if (!dims_ok(M, 0, K)) return GEMM_ERR_DIM;
    if (ldx < std::max(1, K) || !pitches_ok(K, lg, ldq, lds, Z != nullptr, ldz)) return GEMM_ERR_LD;
    if (M == 0 || K == 0) return GEMM_OK;
    if (X == nullptr || Q == nullptr || S == nullptr) return GEMM_ERR_NULL;
    if (!aligned(Q, ldq, S)) return GEMM_ERR_ALIGN;
    const Rows x = rows_of(X, M, K, ldx, elem_size(t));
    const WeightRows w = weight_rows(M, K, lg, Q, ldq, S, lds, Z, ldz);
    if (share(x, w) || share(w.q, w.s) || share(w.q, w.z) || share(w.s, w.z))
        return GEMM_ERR_OVERLAP;
    return status_of(w4::launch_quantize(in_of(t), M, K, X, ldx, Q, ldq, static_cast<uint16_t*>(S),
                                         lds, Z, ldz, bf16, lg, static_cast<hipStream_t>(stream)));
}

int gemm_w4_dequantize(int dtype, int group, int scale_dtype, int M, int K, const uint8_t* Q,
                       int ldq, const void* S, int lds, const uint8_t* Z, int ldz, void* Y, int ldy,
                       void* stream) {
    DType t;
    bool bf16;
    const int lg = log_of(group);
    if (!dtype_of(dtype, t) || lg < 0 || !scale_type(scale_dtype, bf16)) return GEMM_ERR_ARG;
    if (!dims_ok(M, 0, K)) return GEMM_ERR_DIM;
    if (!pitches_ok(K, lg, ldq, lds, Z != nullptr, ldz) || ldy < std::max(1, K)) return GEMM_ERR_LD;
    if (M == 0 || K == 0) return GEMM_OK;
    if (Q == nullptr || S == nullptr || Y == nullptr) return GEMM_ERR_NULL;
    if (!aligned(Q, ldq, S)) return GEMM_ERR_ALIGN;
    if (share(rows_of(Y, M, K, ldy, elem_size(t)), weight_rows(M, K, lg, Q, ldq, S, lds, Z, ldz)))
        return GEMM_ERR_OVERLAP;
    return status_of(w4::launch_dequantize(in_of(t), M, K, weight_of(Q, ldq, S, lds, Z, ldz, bf16, lg),
                                           Y, ldy, static_cast<hipStream_t>(stream)));
}

int gemm_w4_a16(int dtype, int group, int scale_dtype, int M, int N, int K, float alpha,
                const uint16_t* A, int lda, const uint8_t* Q, int ldq, const void* S, int lds,
                const uint8_t* Z, int ldz, float beta, float* C, int ldc, const float* bias,
                void* stream) {
    DType t;
    bool bf16;
    const int lg = log_of(group);
    if (!dtype16_of(dtype, t) || lg < 0 || !scale_type(scale_dtype, bf16)) return GEMM_ERR_ARG;
    if (!dims_ok(M, N, K)) return GEMM_ERR_DIM;
    if (lda < std::max(1, K) || !pitches_ok(K, lg, ldq, lds, Z != nullptr, ldz) ||
        ldc < std::max(1, N))
        return GEMM_ERR_LD;
    if (M == 0 || N == 0) return GEMM_OK;
    const bool reads = alpha != 0.0f && K > 0;
    if (C == nullptr || (reads && (A == nullptr || Q == nullptr || S == nullptr)))
        return GEMM_ERR_NULL;
    const Rows c = rows_of(C, M, N, ldc, 4);
    if (reads) {
        if (!aligned(Q, ldq, S)) return GEMM_ERR_ALIGN;
        if (share(c, rows_of(A, M, K, lda, 2)) ||
            share(c, weight_rows(N, K, lg, Q, ldq, S, lds, Z, ldz)))
            return GEMM_ERR_OVERLAP;
    }
    if (share(c, rows_of(bias, 1, N, N, 4))) return GEMM_ERR_OVERLAP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!reads) {  // C <- beta*C (+ bias)
        dgt::GemmParams g = {};
        g.M = M; g.N = N;
        g.beta = beta;
        g.C = C; g.ldc = ldc;
        g.bias = bias;
        g.batch = 1;
        return status_of(dgt::launch_scale(g, s));
    }
    w4::Product p;
    p.M = M; p.N = N; p.K = K;
    p.alpha = alpha; p.beta = beta;
    p.A = A; p.lda = lda;
    p.w = weight_of(Q, ldq, S, lds, Z, ldz, bf16, lg);
    p.C = C; p.ldc = ldc;
    p.bias = bias;
    return status_of(w4::launch_product(in_of(t), p, s));
}

int gemm_w4_gated(int dtype, int act, int group, int scale_dtype, int M, int N, int K,
                  const uint16_t* X, int ldx, const uint8_t* Q, int ldq, const void* S, int lds,
                  const uint8_t* Z, int ldz, const float* bias_g, const float* bias_u, uint16_t* H,
                  int ldh, void* stream) {
    DType t;
    bool bf16;
    const int lg = log_of(group);
    w4::Gated p;
    if (!dtype16_of(dtype, t) || !act_of(act, p.act) || lg < 0 || !scale_type(scale_dtype, bf16))
        return GEMM_ERR_ARG;
    if (!dims_ok(M, N, K) || N > kMaxDim / 2) return GEMM_ERR_DIM;
    if (ldx < std::max(1, K) || !pitches_ok(K, lg, ldq, lds, Z != nullptr, ldz) ||
        ldh < std::max(1, N))
        return GEMM_ERR_LD;
    if (M == 0 || N == 0) return GEMM_OK;
    if (H == nullptr || (K > 0 && (X == nullptr || Q == nullptr || S == nullptr)))
        return GEMM_ERR_NULL;
    if (K > 0 && !aligned(Q, ldq, S)) return GEMM_ERR_ALIGN;
    const Rows h = rows_of(H, M, N, ldh, 2);
    if (share(h, rows_of(X, M, K, ldx, 2)) ||
        share(h, weight_rows(2 * N, K, lg, Q, ldq, S, lds, Z, ldz)) ||
        share(h, rows_of(bias_g, 1, N, N, 4)) || share(h, rows_of(bias_u, 1, N, N, 4)))
        return GEMM_ERR_OVERLAP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0) {  // the biases alone: no weights, whatever their type
        gated::Forward f = {};
        f.act = p.act;
        f.M = M; f.N = N;
        f.ldx = ldx; f.ldwg = f.ldwu = 1;
        f.bg = bias_g; f.bu = bias_u;
        f.H = H; f.ldh = ldh;
        return status_of(t == DType::BF16 ? gated::launch_forward<dgt::In::BF16>(f, s)
                                          : gated::launch_forward<dgt::In::F16>(f, s));
    }
    p.M = M; p.N = N; p.K = K;
    p.X = X; p.ldx = ldx;
    p.w = weight_of(Q, ldq, S, lds, Z, ldz, bf16, lg);
    p.bg = bias_g; p.bu = bias_u;
    p.H = H; p.ldh = ldh;
    return status_of(w4::launch_gated(in_of(t), p, s));
}

}  // extern "C"
