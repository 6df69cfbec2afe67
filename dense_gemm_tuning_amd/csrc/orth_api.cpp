// orth_api.cpp -- the C entry points of the Newton-Schulz orthogonalisation
// (include/dgt_gemm.h): host-side argument checks and the launches on the
// caller's stream.  Nothing here allocates, synchronises or keeps state.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api_common.hpp"
#include "orth.hpp"

namespace {

using namespace dgt::api;
namespace orth = dgt::orth;

constexpr int kMaxSteps = 64;
constexpr int kMaxBatch = 65535;  // one grid dimension

// Rows past the tiles' 32-bit copy offsets, columns past FP16's range
// (orth.hpp), or matrices whose padded size cannot be a workspace offset.
bool too_large(int M, int N, int batch) {
    return M > orth::kMaxRows || N > orth::kMaxCols ||
           (double)M * ((double)N + 64) * batch > (double)(int64_t(1) << 46);
}

}  // namespace

extern "C" {

int64_t gemm_orthogonalize_workspace_size(int M, int N, int batch) {
    if (batch < 0 || batch > kMaxBatch) return GEMM_ERR_ARG;
    if (M < 0 || N < 0 || too_large(M, N, batch)) return GEMM_ERR_DIM;
    if (M == 0 || N == 0 || batch == 0) return 0;
    return orth::workspace_bytes(M, N, batch);
}

int gemm_orthogonalize(int dtype, int M, int N, const void* G, int ldg, int64_t stride_g,
                       uint16_t* O, int ldo, int64_t stride_o, int batch, int steps, float a,
                       float b, float c, float eps, void* workspace, int64_t workspace_bytes,
                       void* stream) {
    DType t;
    if (!dtype_of(dtype, t) || batch < 0 || batch > kMaxBatch || steps < 1 || steps > kMaxSteps ||
        !std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !std::isfinite(eps) ||
        eps < 0.0f || workspace_bytes < 0 || !valid_stride(stride_g) || !valid_stride(stride_o))
        return GEMM_ERR_ARG;
    if (M < 0 || N < 0 || too_large(M, N, batch)) return GEMM_ERR_DIM;
    if (ldg < std::max(1, N) || ldo < std::max(1, N)) return GEMM_ERR_LD;
    if (M == 0 || N == 0 || batch == 0) return GEMM_OK;
    if (G == nullptr || O == nullptr) return GEMM_ERR_NULL;
    const int64_t need = orth::workspace_bytes(M, N, batch);
    if (workspace == nullptr || workspace_bytes < need) return GEMM_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return GEMM_ERR_ALIGN;
    const int esz = elem_size(t);
    const uint64_t o_span = span_bytes(M, N, ldo, 2);
    // the problems of a batch must not write over each other
    if (batch > 1 && (uint64_t)stride_o * 2 < o_span) return GEMM_ERR_OVERLAP;
    const Range rw = batch_range(workspace, (uint64_t)need, 0, 1);
    if (overlaps(rw, batch_range(G, span_bytes(M, N, ldg, esz), stride_g * esz, batch)) ||
        overlaps(rw, batch_range(O, o_span, stride_o * 2, batch)))
        return GEMM_ERR_OVERLAP;
    orth::Call call;
    call.t = t == DType::F32 ? dgt::In::F32 : t == DType::BF16 ? dgt::In::BF16 : dgt::In::F16;
    call.G = G; call.ldg = ldg; call.stride_g = stride_g;
    call.O = O; call.ldo = ldo; call.stride_o = stride_o;
    call.steps = steps;
    call.a = a; call.b = b; call.c = c; call.eps = eps;
    call.ws = static_cast<uint8_t*>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = orth::is_small(M, N, batch)
                             ? orth::launch_small(orth::make_small_plan(M, N, batch), call, s)
                             : orth::launch(orth::make_plan(M, N, batch), call, s);
    if (e == hipErrorInvalidConfiguration) return GEMM_ERR_DIM;  // more tiles than a grid holds
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
