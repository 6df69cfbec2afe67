// mx4_api.cpp -- the C entry points of the microscaled 4-bit operators
// (include/dgt_gemm.h): host-side argument checks and the launch on the
// caller's stream.  Nothing here allocates, synchronises or keeps state, and
// the checks run before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_common.hpp"
#include "mx4.hpp"

namespace {

using namespace dgt::api;
namespace mx4 = dgt::mx4;

dgt::In in_of(DType t) {
    return t == DType::F32 ? dgt::In::F32 : t == DType::BF16 ? dgt::In::BF16 : dgt::In::F16;
}

// Pitches of an MX4 operand of K columns against their limits.
bool pitch_ok(int K, int ldq, int lds) {
    return ldq >= std::max<int64_t>(1, mx4::code_pitch(K)) && ldq <= DGT_GEMM_MX4_MAX_PITCH &&
           lds >= std::max<int64_t>(1, mx4::scale_pitch(K)) && lds <= DGT_GEMM_MX4_MAX_PITCH;
}

// 16-byte boundaries of an operand's codes and scales.
bool aligned(const void* Q, int ldq, const void* S, int lds) {
    return (reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(S) | (uintptr_t)ldq |
            (uintptr_t)lds) % 16 == 0;
}

Range rows_range(const void* base, int rows, int64_t row_bytes, int64_t pitch_bytes) {
    if (rows == 0 || row_bytes == 0) return batch_range(base, 0, 0, 0);
    return batch_range(base, (uint64_t)(rows - 1) * (uint64_t)pitch_bytes + (uint64_t)row_bytes, 0,
                       1);
}

int status_of(hipError_t e) {
    return e == hipSuccess                      ? GEMM_OK
           : e == hipErrorInvalidConfiguration ? GEMM_ERR_DIM  // more workgroups than a launch holds
                                               : GEMM_ERR_LAUNCH;
}

// The checks and the launch shared by the two products; t is the format of A
// (MX4 when mx is set).
int product(bool mx, DType t, int M, int N, int K, float alpha, const void* A, int lda,
            const uint8_t* SA, int ldsa, const uint8_t* B, int ldb, const uint8_t* SB, int ldsb,
            float beta, float* C, int ldc, const float* bias, void* stream) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_DIM;
    if (!pitch_ok(K, ldb, ldsb) || ldc < std::max(1, N)) return GEMM_ERR_LD;
    if (mx ? !pitch_ok(K, lda, ldsa) : lda < std::max(1, K)) return GEMM_ERR_LD;
    if (M == 0 || N == 0) return GEMM_OK;  // empty C: nothing to do
    const bool reads_ab = alpha != 0.0f && K > 0;
    if (C == nullptr) return GEMM_ERR_NULL;
    if (reads_ab && (A == nullptr || B == nullptr || SB == nullptr || (mx && SA == nullptr)))
        return GEMM_ERR_NULL;
    const Range rc = rows_range(C, M, (int64_t)N * 4, (int64_t)ldc * 4);
    if (reads_ab) {
        if (!aligned(B, ldb, SB, ldsb) || (mx && !aligned(A, lda, SA, ldsa))) return GEMM_ERR_ALIGN;
        if (overlaps(rc, rows_range(B, N, mx4::code_pitch(K), ldb)) ||
            overlaps(rc, rows_range(SB, N, mx4::scale_pitch(K), ldsb)))
            return GEMM_ERR_OVERLAP;
        if (mx ? overlaps(rc, rows_range(A, M, mx4::code_pitch(K), lda)) ||
                     overlaps(rc, rows_range(SA, M, mx4::scale_pitch(K), ldsa))
               : overlaps(rc, rows_range(A, M, (int64_t)K * 2, (int64_t)lda * 2)))
            return GEMM_ERR_OVERLAP;
    }
    if (bias && overlaps(rc, batch_range(bias, (uint64_t)N * 4, 0, 1))) return GEMM_ERR_OVERLAP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!reads_ab) {  // C <- beta*C (+ bias)
        dgt::GemmParams g = {};
        g.M = M; g.N = N;
        g.beta = beta;
        g.C = C; g.ldc = ldc;
        g.bias = bias;
        g.batch = 1;
        return status_of(dgt::launch_scale(g, s));
    }
    mx4::Params p;
    p.M = M; p.N = N; p.K = K;
    p.alpha = alpha; p.beta = beta;
    p.A = A; p.lda = lda;
    p.SA = SA; p.ldsa = ldsa;
    p.B = B; p.ldb = ldb;
    p.SB = SB; p.ldsb = ldsb;
    p.C = C; p.ldc = ldc;
    p.bias = bias;
    return status_of(mx ? mx4::launch_product(p, s) : mx4::launch_product16(in_of(t), p, s));
}

}  // namespace

extern "C" {

int64_t gemm_mx4_code_pitch(int K) { return K <= 0 ? 0 : mx4::code_pitch(K); }
int64_t gemm_mx4_scale_pitch(int K) { return K <= 0 ? 0 : mx4::scale_pitch(K); }

int gemm_mx4_quantize(int dtype, int trans, int M, int K, const void* X, int ldx, uint8_t* Q,
                      int ldq, uint8_t* S, int lds, void* stream) {
    DType t;
    if (!dtype_of(dtype, t) || !valid_flag(trans)) return GEMM_ERR_ARG;
    if (M < 0 || K < 0) return GEMM_ERR_DIM;
    if (ldx < std::max(1, trans ? M : K) || !pitch_ok(K, ldq, lds)) return GEMM_ERR_LD;
    if (M == 0 || K == 0) return GEMM_OK;
    if (X == nullptr || Q == nullptr || S == nullptr) return GEMM_ERR_NULL;
    if (!aligned(Q, ldq, S, lds)) return GEMM_ERR_ALIGN;
    const int esz = elem_size(t);
    const Range rx = batch_range(X, trans ? span_bytes(K, M, ldx, esz) : span_bytes(M, K, ldx, esz),
                                 0, 1);
    const Range rq = rows_range(Q, M, mx4::code_pitch(K), ldq);
    const Range rs = rows_range(S, M, mx4::scale_pitch(K), lds);
    if (overlaps(rx, rq) || overlaps(rx, rs) || overlaps(rq, rs)) return GEMM_ERR_OVERLAP;
    return status_of(mx4::launch_quantize(in_of(t), trans != 0, M, K, X, ldx, Q, ldq, S, lds,
                                          static_cast<hipStream_t>(stream)));
}

int gemm_mx4_dequantize(int dtype, int M, int K, const uint8_t* Q, int ldq, const uint8_t* S,
                        int lds, void* Y, int ldy, void* stream) {
    DType t;
    if (!dtype_of(dtype, t)) return GEMM_ERR_ARG;
    if (M < 0 || K < 0) return GEMM_ERR_DIM;
    if (!pitch_ok(K, ldq, lds) || ldy < std::max(1, K)) return GEMM_ERR_LD;
    if (M == 0 || K == 0) return GEMM_OK;
    if (Q == nullptr || S == nullptr || Y == nullptr) return GEMM_ERR_NULL;
    if (!aligned(Q, ldq, S, lds)) return GEMM_ERR_ALIGN;
    const int esz = elem_size(t);
    const Range ry = rows_range(Y, M, (int64_t)K * esz, (int64_t)ldy * esz);
    if (overlaps(ry, rows_range(Q, M, mx4::code_pitch(K), ldq)) ||
        overlaps(ry, rows_range(S, M, mx4::scale_pitch(K), lds)))
        return GEMM_ERR_OVERLAP;
    return status_of(mx4::launch_dequantize(in_of(t), M, K, Q, ldq, S, lds, Y, ldy,
                                            static_cast<hipStream_t>(stream)));
}

int gemm_mx4(int M, int N, int K, float alpha, const uint8_t* A, int lda, const uint8_t* SA,
             int ldsa, const uint8_t* B, int ldb, const uint8_t* SB, int ldsb, float beta, float* C,
             int ldc, const float* bias, void* stream) {
    return product(true, DType::F32, M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, beta, C,
                   ldc, bias, stream);
}

int gemm_mx4_a16(int dtype, int M, int N, int K, float alpha, const uint16_t* A, int lda,
                 const uint8_t* B, int ldb, const uint8_t* SB, int ldsb, float beta, float* C,
                 int ldc, const float* bias, void* stream) {
    DType t;
    if (!dtype_of(dtype, t) || t == DType::F32) return GEMM_ERR_ARG;
    return product(false, t, M, N, K, alpha, A, lda, nullptr, 0, B, ldb, SB, ldsb, beta, C, ldc,
                   bias, stream);
}

}  // extern "C"
