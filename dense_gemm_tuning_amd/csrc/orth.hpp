// orth.hpp -- Newton-Schulz orthogonalisation: the plan shared by the entry
// point (orth_api.cpp) and the kernels (k_orth.hip).
#pragma once

#include "gemm_common.hpp"

namespace dgt {
namespace orth {

constexpr int kNormParts = 256;  // partial sums of squares per matrix

// Workspace of a batch of M x N matrices, byte offsets from its start.  X is
// kept as two FP16 halves (hi + lo), twice (a step reads one copy and writes
// the other); S and B are the n x n Gram matrix and step polynomial, n the
// smaller dimension and k the larger.  Rows are padded to 64 elements (128 bytes).
struct Plan {
    int M, N, batch, n, k;
    int64_t ldx, lds;           // elements
    int64_t x_size, s_size;     // elements of one matrix
    // The Gram matrix's sums over k in `splits` parts of kc (the last one
    // shorter) of tiles of kGramTile, when more than one part is worthwhile.
    int splits, kc;
    int64_t hi[2], lo[2], gram, poly, partial, parts, bytes;
};

constexpr int kGramTile = 128;  // of a Gram matrix in parts

inline int64_t lower_tiles(int n, int R) {  // tiles on or below the diagonal
    const int64_t t = (n + R - 1) / R;
    return t * (t + 1) / 2;
}

inline Plan make_plan(int M, int N, int batch) {
    Plan p;
    p.M = M; p.N = N; p.batch = batch;
    p.n = M < N ? M : N;
    p.k = M < N ? N : M;
    p.ldx = ((int64_t)N + 63) / 64 * 64;
    p.lds = ((int64_t)p.n + 63) / 64 * 64;
    p.x_size = (int64_t)M * p.ldx;
    p.s_size = (int64_t)p.n * p.lds;
    // Few tiles and a long k leave compute units idle: enough parts to give
    // each one a tile, no part below 512 deep.
    p.splits = 1;
    p.kc = p.k;
    const int64_t tiles = lower_tiles(p.n, kGramTile) * batch;
    const int64_t want = tiles < 256 ? 256 / tiles : 1, most = p.k / 512;
    const int64_t parts = want < most ? want : most;
    if (parts > 1) {
        p.kc = (int)((p.k + parts - 1) / parts + 127) / 128 * 128;
        p.splits = (p.k + p.kc - 1) / p.kc;
    }
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
    p.partial = take(p.splits > 1 ? tiles * p.splits * kGramTile * kGramTile * 4 : 0);
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
