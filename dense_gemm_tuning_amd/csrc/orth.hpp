// orth.hpp -- Newton-Schulz orthogonalisation: the plan shared by the entry
// point (orth_api.cpp) and the kernels (k_orth.hip).
#pragma once

#include "gemm_common.hpp"

namespace dgt {
namespace orth {

constexpr int kNormParts = 64;  // partial sums of squares per matrix

// Workspace of a batch of M x N matrices, byte offsets from its start.  X is
// kept as two FP16 halves (hi + lo), twice (a step reads one copy and writes
// the other); S and B are the s x s Gram matrix and step polynomial, s the
// smaller dimension; C the fp32 product before it is rounded.  Rows are
// padded to 64 elements (128 bytes).
struct Plan {
    int M, N, batch, s;
    int64_t ldx, lds;           // elements
    int64_t x_size, s_size;     // elements of one matrix
    int64_t hi[2], lo[2], gram, poly, c32, parts, bytes;
};

inline Plan make_plan(int M, int N, int batch) {
    Plan p;
    p.M = M; p.N = N; p.batch = batch;
    p.s = M < N ? M : N;
    p.ldx = (N + 63) / 64 * (int64_t)64;
    p.lds = (p.s + 63) / 64 * (int64_t)64;
    p.x_size = (int64_t)M * p.ldx;
    p.s_size = (int64_t)p.s * p.lds;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    p.parts = take((int64_t)batch * kNormParts * 8);
    for (int i = 0; i < 2; ++i) {
        p.hi[i] = take(batch * p.x_size * 2);
        p.lo[i] = take(batch * p.x_size * 2);
    }
    p.gram = take(batch * p.s_size * 2);
    p.poly = take(batch * p.s_size * 2);
    p.c32 = take(batch * (p.x_size > p.s_size ? p.x_size : p.s_size) * 4);
    p.bytes = at;
    return p;
}

struct Call {
    In t;
    const void* G;
    int64_t ldg, stride_g;  // elements
    uint16_t* O;
    int64_t ldo, stride_o;
    int steps;
    float a, b, c, eps;
    uint8_t* ws;
};

hipError_t launch(const Plan& p, const Call& c, hipStream_t s);

}  // namespace orth
}  // namespace dgt
