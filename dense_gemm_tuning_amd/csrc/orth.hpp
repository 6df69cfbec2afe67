// orth.hpp -- Newton-Schulz orthogonalisation: the plan shared by the entry
// point (orth_api.cpp) and the kernels (k_orth.hip).
#pragma once

#include <cmath>

#include "gemm_common.hpp"

namespace dgt {
namespace orth {

// Sizes.  A workgroup of the tile kernels copies up to 64 rows of X through one
// descriptor with 32-bit byte offsets (mfma16_tile.hpp), so a padded row is at
// most kMaxBufferPitch elements.  X is held times 2^scale_exp of the larger
// dimension, 2^13 up to 2^26: its elements, below 4 as its singular values are,
// stay below FP16's 65504 (2^14 would not).
constexpr int kMaxCols = (int)kMaxBufferPitch, kMaxRows = 1 << 26;

// Partial sums of squares of a matrix: a workgroup's 256 lanes take a few runs
// of 8 elements each.
constexpr int kMaxNormParts = 1024;
inline int norm_parts(int M, int N) {
    const int64_t runs = (int64_t)M * (((int64_t)N + 7) / 8), parts = (runs + 1023) / 1024;
    return (int)(parts < kMaxNormParts ? parts : kMaxNormParts);
}

// Workspace of a batch of M x N matrices, byte offsets from its start.  X is
// kept as two FP16 halves (hi + lo), twice (a step reads one copy and writes
// the other); S and B are the n x n Gram matrix and step polynomial, n the
// smaller dimension and k the larger; diag is what rounding to FP16 took from
// B's diagonal (n floats).  Rows are padded to 64 elements (128 bytes).
struct Plan {
    int M, N, batch, n, k;
    int64_t ldx, lds;           // elements
    int64_t x_size, s_size;     // elements of one matrix
    // The Gram matrix's sums over k in `splits` parts of kc (the last one
    // shorter) of tiles of kGramTile, when more than one part is worthwhile.
    int splits, kc;
    int64_t hi[2], lo[2], gram, poly, diag, partial, parts, bytes;
};

// Small matrices (k_orth_small.hip): every matrix padded with zeros to
// multiples of 64 in both dimensions, X held both ways round.
struct SmallPlan {
    int M, N, batch, n, k;      // n <= k: a tall G is taken transposed
    int n64, k64;
    int64_t x_size, s_size;     // elements of one matrix
    int64_t x[2], xt[2], lo[2], gram, poly, diag, parts, bytes;
};

// Whether a call takes them: products whose 32 x 32 tiles, a workgroup each,
// make three rounds of the compute units at most.  Measured, us (these / the tile
// kernels): 64^2 51 / 80, 256^2 60 / 109, 512^2 85 / 146, 768^2 194 / 188, 900^2 281 / 234,
// 1024^2 290 / 216, 256 x 1024 78 / 130, 640 x 1280 187 / 184, 256 x 4096 167 / 138,
// 4 x 256^2 69 / 112, 16 x 256^2 135 / 109.
inline bool is_small(int M, int N, int batch) {
    const int64_t n = ((M < N ? M : N) + 63ll) / 64 * 64, k = ((M < N ? N : M) + 63ll) / 64 * 64;
    return k <= 2048 && n * k / 1024 * batch <= 800;
}

inline SmallPlan make_small_plan(int M, int N, int batch) {
    SmallPlan p;
    p.M = M; p.N = N; p.batch = batch;
    p.n = M < N ? M : N;
    p.k = M < N ? N : M;
    p.n64 = (p.n + 63) / 64 * 64;
    p.k64 = (p.k + 63) / 64 * 64;
    p.x_size = (int64_t)p.n64 * p.k64;
    p.s_size = (int64_t)p.n64 * p.n64;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    p.parts = take((int64_t)batch * norm_parts(M, N) * 8);
    for (int i = 0; i < 2; ++i) {
        p.x[i] = take(batch * p.x_size * 2);
        p.xt[i] = take(batch * p.x_size * 2);
        p.lo[i] = take(batch * p.x_size * 2);
    }
    p.gram = take(batch * p.s_size * 2);
    p.poly = take(batch * p.s_size * 2);
    p.diag = take((int64_t)batch * p.n64 * 4);
    p.bytes = at;
    return p;
}

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
    // each one a tile (two side by side where one does not go round), no part below 512 deep.
    // 8192 x 1024 (36 tiles): 344 us for the whole call in 7 parts, 350 in 14, 466
    // in one; 1024 x 8192 348, 365, 605; 2048 x 8192 (136 tiles) 796 in 3, 854 in 7, 936 in one.
    p.splits = 1;
    p.kc = p.k;
    const int64_t tiles = lower_tiles(p.n, kGramTile) * batch;
    const int64_t want = (tiles <= 128 ? 256 : 512) / tiles, most = p.k / 512;
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
    p.parts = take((int64_t)batch * norm_parts(M, N) * 8);
    for (int i = 0; i < 2; ++i) {
        p.hi[i] = take(batch * p.x_size * 2);
        p.lo[i] = take(batch * p.x_size * 2);
    }
    p.gram = take(batch * p.s_size * 2);
    p.poly = take(batch * p.s_size * 2);
    p.diag = take((int64_t)batch * p.n * 4);
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

inline int64_t workspace_bytes(int M, int N, int batch) {
    return is_small(M, N, batch) ? make_small_plan(M, N, batch).bytes : make_plan(M, N, batch).bytes;
}

hipError_t launch(const Plan& p, const Call& c, hipStream_t s);
hipError_t launch_small(const SmallPlan& p, const Call& c, hipStream_t s);
// The partial sums of squares of a batch (k_orth.hip).
hipError_t launch_norm(const Call& c, int M, int N, int batch, double* parts, hipStream_t s);

// FP16's range: S is held times 2^12, the step polynomial times 2^10, X times
// 2^scale_exp near the square root of its larger dimension.
constexpr float kGramScale = 4096.0f;
constexpr float kPolyScale = 1024.0f;
inline int scale_exp(int k) { return (int)std::lround(0.5 * std::log2((double)k)); }

}  // namespace orth
}  // namespace dgt
