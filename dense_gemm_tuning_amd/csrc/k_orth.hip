// k_orth.hip -- orthogonalisation by Newton-Schulz steps.
//
//     X <- G / (|G|_F + eps);   steps times:  S = X X^T,  X <- a X + (b S + c S S) X
//
// (M <= N; for M > N the same from the right: S = X^T X, X <- a X + X (b S + c S S),
// so no matrix is transposed in memory).  The three products of a step are the
// library's FP16 tile product (mfma16_tile.hpp) with epilogues of their own:
//   S   its tiles on and below the diagonal (half the work), each stored and mirrored;
//   B = b S + c S S   likewise, S's rows serving as its columns;
//   X   a X added from the two halves below, the next two halves or the bf16 result
//       stored.
// A Gram matrix with too few tiles for the chip is summed over k in parts.
//
// Rounding.  The products' operands are FP16.  Each step multiplies what
// rounding X adds in the weak singular directions by up to a (3.4 with the
// usual coefficients, 484 over five steps), so X rounded to 16 bits costs a matrix
// of rank one 0.15, and 3.3e-3 if only the last two steps' X is, against 1.7e-3 that the
// result's own bf16 rounding costs.  X is therefore kept as two halves hi + lo
// (22 bits) in every step; the products read hi, the term a X both.  What hi's
// rounding E adds through the products reaches the weak directions only as (b S + c S S) E,
// small where S is.  B is largest on its diagonal; what its rounding takes there is kept in
// fp32 and added in the update, times hi like the rest of B's row (one row 5000 long:
// 3.3e-3 without, 2.3e-3 with it; 48 x 2600 3.1e-3, 2.2e-3).  The result is normwise 1.7e-3 off for
// exact low rank and 1/i^2 spectra, 1.7 to 1.8e-3 for 1/i, 1.7 to 2.5e-3 for normal
// values or a floor of them, where the roundings of S and B count too (1 to 4096 rows, five steps).
//
// FP16's range: |X| <= |X|_2, about 1, but its elements are near
// 1/sqrt(max(M, N)) and the Gram matrix's smaller still, so X is held times
// 2^x_exp near that root, S times 2^12 and the polynomial times 2^10 (both at most
// about 13 * 2^10 for singular values up to 1.3); powers of two, so only the
// range moves.
#include "mfma16_tile.hpp"
#include "orth.hpp"

namespace dgt {
namespace orth {

namespace {

using namespace mfma16;

// Eight elements of a row, widened; `vec`: the row starts and pitch are on 16
// bytes.
template <In T>
__device__ __forceinline__ void load8(const typename InFmt<T>::S* row, int col, int N, bool vec,
                                      float (&v)[8]) {
    using E = typename InFmt<T>::S;
    if (vec && col + 8 <= N) {
        constexpr int W = 16 / sizeof(E);  // elements per 16 bytes
#pragma unroll
        for (int h = 0; h < 8 / W; ++h) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(row + col + W * h);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                if constexpr (T == In::F32) v[W * h + e] = __uint_as_float(x[e]);
                else v[e] = InFmt<T>::widen((uint16_t)(x[e / 2] >> (16 * (e % 2))));
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = col + e < N ? load_in<T>(row + col + e) : 0.0f;
    }
}

// Partial sums of squares per matrix, in 64 bits (an fp32 input's squares
// leave fp32's range): workgroup x of matrix blockIdx.y takes every
// gridDim.x-th run of 8 * NT elements.  The order is fixed.
template <In T>
__global__ __launch_bounds__(NT) void norm_kernel(const typename InFmt<T>::S* G, int64_t ldg,
                                                  int64_t stride, int M, int N, bool vec,
                                                  double* parts) {
    G += blockIdx.y * stride;
    const int per_row = (N + 7) / 8;
    const int64_t total = (int64_t)M * per_row;
    double sum = 0.0;
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * NT) {
        float v[8];
        load8<T>(G + e / per_row * ldg, (int)(e % per_row) * 8, N, vec, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += (double)v[i] * (double)v[i];
    }
    __shared__ double red[NT];
    red[threadIdx.x] = sum;
    __syncthreads();
    for (int h = NT / 2; h > 0; h /= 2) {
        if ((int)threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
        __syncthreads();
    }
    if (threadIdx.x == 0) parts[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = red[0];
}

// Eight values as two FP16 halves, x = hi + lo to 22 bits.
__device__ __forceinline__ void split8(const float (&x)[8], halfx8& hi, halfx8& lo) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        hi[e] = (_Float16)x[e];
        lo[e] = (_Float16)(x[e] - (float)hi[e]);
    }
}

// X <- G * 2^x_exp / (|G| + eps) as two halves; zeros in the padding columns.
template <In T>
__global__ __launch_bounds__(NT) void init_kernel(const typename InFmt<T>::S* G, int64_t ldg,
                                                  int64_t stride, int M, int N, bool vec,
                                                  const double* parts, int nparts, double eps,
                                                  double scale, _Float16* hi, _Float16* lo, int64_t ldx) {
    const int64_t z = blockIdx.y;
    G += z * stride;
    hi += z * M * ldx;
    lo += z * M * ldx;
    __shared__ double red[NT];
    double sum = 0.0;
    for (int i = threadIdx.x; i < nparts; i += NT) sum += parts[z * nparts + i];
    red[threadIdx.x] = sum;
    __syncthreads();
    for (int h = NT / 2; h > 0; h /= 2) {
        if ((int)threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
        __syncthreads();
    }
    const double inv = scale / (sqrt(red[0]) + eps);
    const int per_row = (int)(ldx / 8);
    const int64_t total = (int64_t)M * per_row;
    for (int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x; e < total;
         e += (int64_t)gridDim.x * NT) {
        const int64_t row = e / per_row;
        const int col = (int)(e % per_row) * 8;
        float v[8];
        load8<T>(G + row * ldg, col, N, vec, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = col + i < N ? (float)((double)v[i] * inv) : 0.0f;
        halfx8 h, l;
        split8(v, h, l);
        *reinterpret_cast<halfx8*>(hi + row * ldx + col) = h;
        *reinterpret_cast<halfx8*>(lo + row * ldx + col) = l;
    }
}

// ------------------------------------------------------------- epilogues
//
// Accumulators reach memory through the wavefront's LDS region, one row of
// MFMA tiles (32 x R/2 fp32) at a time, so that a lane handles 8 neighbouring
// columns (or, mirrored, 8 neighbouring rows) with 16-byte accesses.  Column c of
// row r sits at c ^ 32*(r/4 & 1): the two half-waves of an accumulator write rows 4
// apart, which then differ in banks.

template <int R>
struct Chunk {
    static constexpr int W = R / 2;           // columns
    static constexpr int GROUPS = W / 8;      // column groups of 8
    float* mem;
    __device__ static int at(int r, int c) { return r * W + (c ^ (32 * ((r >> 2) & 1))); }
    // Lanes read what other lanes of the wavefront wrote: LDS keeps their
    // order, the compiler has to as well.
    __device__ static void fence() {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    // MFMA tiles of tile row ti.
    __device__ void put(const floatx16 (&acc)[Geo<R>::TM], int lane) const {
        const int h = lane >> 5;
        fence();
#pragma unroll
        for (int tj = 0; tj < Geo<R>::TM; ++tj)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                mem[at(8 * (r >> 2) + 4 * h + (r & 3), tj * 32 + (lane & 31))] = acc[tj][r];
        fence();
    }
    __device__ void row8(int r, int c, float (&v)[8]) const {
        const floatx4 a = *reinterpret_cast<const floatx4*>(mem + at(r, c));
        const floatx4 b = *reinterpret_cast<const floatx4*>(mem + at(r, c + 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    }
    __device__ void col8(int r, int c, float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = mem[at(r + e, c)];
    }
    void __device__ set_row8(int r, int c, const float (&v)[8]) const {
        *reinterpret_cast<floatx4*>(mem + at(r, c)) = floatx4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<floatx4*>(mem + at(r, c + 4)) = floatx4{v[4], v[5], v[6], v[7]};
    }
    // The lane's pieces of a chunk: piece i is 8 columns of a row, or
    // (mirrored) 8 rows of a column.
    static constexpr int PIECES = 32 * W / 8 / 64;
    __device__ static int row(int i, int lane) { return (64 * i + lane) / GROUPS; }
    __device__ static int col(int i, int lane) { return (64 * i + lane) % GROUPS * 8; }
    __device__ static int mirror_col(int i, int lane) { return (64 * i + lane) % W; }
    __device__ static int mirror_row(int i, int lane) { return (64 * i + lane) / W * 8; }
};

// Tiles on and below the diagonal, numbered row by row; XCD x takes a
// contiguous range of the launch's tiles.
__device__ __forceinline__ TileIdx lower_tile(int64_t per_problem) {
    const int64_t total = per_problem * gridDim.y;
    const int64_t lin = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    const int64_t x = lin % kXcds, q = lin / kXcds, per = total / kXcds, rem = total % kXcds;
    const int64_t g = x < rem ? x * (per + 1) + q : rem * (per + 1) + (x - rem) * per + q;
    const int64_t idx = g % per_problem;
    int bm = (int)((sqrt(8.0 * (double)idx + 1.0) - 1.0) * 0.5);
    while ((int64_t)bm * (bm + 1) / 2 > idx) --bm;  // the root may be off by its rounding
    while ((int64_t)(bm + 1) * (bm + 2) / 2 <= idx) ++bm;
    return TileIdx{(int)(g / per_problem), bm, (int)(idx - (int64_t)bm * (bm + 1) / 2)};
}

// A symmetric n x n product's tile: OUT <- f1 * sums (+ f2 * D), and mirrored
// off the diagonal; D is OUT's layout.  With D, diag <- what rounding took from
// OUT's diagonal.
template <int R, bool TA, bool TB, bool kEdge, bool kTail, bool kAdd>
__global__ __launch_bounds__(NT, R == 256 ? 1 : 2) void symmetric_kernel(
    GemmParams p, int64_t tiles, _Float16* out, const _Float16* add, float* diag, int64_t ld,
    int64_t size, float f1, float f2) {
    const TileIdx tile = lower_tile(tiles);
    select_problem(p, tile.z);
    out += tile.z * size;
    if constexpr (kAdd) {
        add += tile.z * size;
        diag += (int64_t)tile.z * p.M;
    }
    const int m0 = tile.bm * R, n0 = tile.bn * R;
    dma_tile<In::F16, R, TA, TB, kEdge, kTail>(
        p, m0, n0, nullptr, [&](const auto& acc, int wm, int wn, int lane, uint8_t* mem) {
            using Ch = Chunk<R>;
            const Ch chunk{reinterpret_cast<float*>(mem)};
            static_assert(32 * Ch::W * 4 <= (TA ? Geo<R>::MN_STAGE : Geo<R>::KC_STAGE / 2), "");
            const int row0 = m0 + wm * (R / 2), col0 = n0 + wn * (R / 2);
            // D one chunk ahead of its use
            halfx8 d[2][kAdd ? Ch::PIECES : 1];
            auto fetch = [&](int ti) {
                if constexpr (kAdd) {
#pragma unroll
                    for (int i = 0; i < Ch::PIECES; ++i) {
                        const int row = row0 + 32 * ti + Ch::row(i, lane), col = col0 + Ch::col(i, lane);
                        if (!kEdge || (row < p.M && col < p.N))
                            d[ti & 1][i] = *reinterpret_cast<const halfx8*>(add + row * ld + col);
                    }
                }
            };
            fetch(0);
#pragma unroll
            for (int ti = 0; ti < Geo<R>::TM; ++ti) {
                if (ti + 1 < Geo<R>::TM) fetch(ti + 1);
                chunk.put(acc[ti], lane);
#pragma unroll
                for (int i = 0; i < Ch::PIECES; ++i) {
                    const int r = Ch::row(i, lane), c = Ch::col(i, lane);
                    const int row = row0 + 32 * ti + r, col = col0 + c;
                    float v[8];
                    chunk.row8(r, c, v);
                    halfx8 o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] = kAdd ? fmaf(f2, (float)d[ti & 1][i][e], f1 * v[e]) : f1 * v[e];
                        o[e] = (_Float16)v[e];
                    }
                    if (kAdd && m0 != n0) chunk.set_row8(r, c, v);  // for the mirrored pieces
                    if (!kEdge || (row < p.M && col < p.N))
                        *reinterpret_cast<halfx8*>(out + row * ld + col) = o;
                }
                if (m0 == n0) {
                    if constexpr (kAdd) {  // one lane an element, the same operations as above
                        const int row = row0 + 32 * ti + lane;
                        if (wm == wn && lane < 32 && (!kEdge || row < p.M)) {
                            const float v = fmaf(f2, (float)add[row * ld + row],
                                                 f1 * chunk.mem[Ch::at(lane, 32 * ti + lane)]);
                            diag[row] = v - (float)(_Float16)v;
                        }
                    }
                    continue;
                }
                if constexpr (kAdd) Ch::fence();
#pragma unroll
                for (int i = 0; i < Ch::PIECES; ++i) {
                    const int c = Ch::mirror_col(i, lane), r = Ch::mirror_row(i, lane);
                    const int row = col0 + c, col = row0 + 32 * ti + r;
                    float v[8];
                    chunk.col8(r, c, v);
                    halfx8 o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = (_Float16)(kAdd ? v[e] : f1 * v[e]);
                    if (!kEdge || (row < p.N && col < p.M))
                        *reinterpret_cast<halfx8*>(out + row * ld + col) = o;
                }
            }
        });
}

// X' = a (hi + lo) + f * (sums + diag hi): two halves, or (kLast) the result in
// bf16; diag holds the rest of B's diagonal, of the rows of X (of its columns for a tall
// X, whose B stands on the right).
struct Update {
    const _Float16 *hi, *lo;
    _Float16 *hi2, *lo2;
    const float* diag;
    int64_t ldx, x_size;
    float a, f;
    uint16_t* O;
    int64_t ldo, stride_o;
    float out_scale;
    bool o_vec;  // O's rows on 16 bytes
};
template <int R, bool TB, bool kEdge, bool kTail, bool kLast>
__global__ __launch_bounds__(NT, R == 256 ? 1 : 2) void update_kernel(GemmParams p, int tiles_m,
                                                                    int tiles_n, Update u) {
    const TileIdx tile = xcd_tile(tiles_m, tiles_n, true);
    select_problem(p, tile.z);
    const int m0 = tile.bm * R, n0 = tile.bn * R;
    const int64_t xz = tile.z * u.x_size;
    uint16_t* O = u.O + tile.z * u.stride_o;
    dma_tile<In::F16, R, false, TB, kEdge, kTail>(
        p, m0, n0, nullptr, [&](const auto& acc, int wm, int wn, int lane, uint8_t* mem) {
            using Ch = Chunk<R>;
            const Ch chunk{reinterpret_cast<float*>(mem)};
            const int row0 = m0 + wm * (R / 2), col0 = n0 + wn * (R / 2);
            // X one chunk ahead of its use
            halfx8 h[2][Ch::PIECES], l[2][Ch::PIECES];
            auto fetch = [&](int ti) {
#pragma unroll
                for (int i = 0; i < Ch::PIECES; ++i) {
                    const int row = row0 + 32 * ti + Ch::row(i, lane), col = col0 + Ch::col(i, lane);
                    const int64_t at = xz + (int64_t)row * u.ldx + col;
                    if (!kEdge || (row < p.M && col < p.N)) {
                        h[ti & 1][i] = *reinterpret_cast<const halfx8*>(u.hi + at);
                        l[ti & 1][i] = *reinterpret_cast<const halfx8*>(u.lo + at);
                    }
                }
            };
            fetch(0);
            // The diagonal's rest.  Of the rows: one per lane, taken from the lane
            // that has it; of the columns: a lane's eight are the same in every piece.
            constexpr int ND = TB ? 8 : R / 128;
            static_assert(64 % Ch::GROUPS == 0, "a lane's columns");
            const float* diag = u.diag + (int64_t)tile.z * (TB ? p.N : p.M);
            float d[ND];
#pragma unroll
            for (int j = 0; j < ND; ++j) {
                const int at = TB ? col0 + Ch::col(0, lane) + j : row0 + 64 * j + lane;
                d[j] = at < (TB ? p.N : p.M) ? diag[at] : 0.0f;
            }
#pragma unroll
            for (int ti = 0; ti < Geo<R>::TM; ++ti) {
                if (ti + 1 < Geo<R>::TM) fetch(ti + 1);
                chunk.put(acc[ti], lane);
#pragma unroll
                for (int i = 0; i < Ch::PIECES; ++i) {
                    const int r = Ch::row(i, lane), c = Ch::col(i, lane);
                    const int row = row0 + 32 * ti + r, col = col0 + c;
                    float x[8];
                    chunk.row8(r, c, x);
                    const float dr = TB ? 0.0f : __shfl(d[TB ? 0 : ti / 2], 32 * (ti & 1) + r);
                    if (kEdge && (row >= p.M || col >= p.N)) continue;
                    const int64_t at = xz + (int64_t)row * u.ldx + col;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float hi = (float)h[ti & 1][i][e];
                        x[e] = u.a * (hi + (float)l[ti & 1][i][e]) +
                               u.f * fmaf(TB ? d[TB ? e : 0] : dr, hi, x[e]);
                    }
                    if constexpr (kLast) {
                        bf16x8 o;
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = (__bf16)(x[e] * u.out_scale);
                        uint16_t* out = O + (int64_t)row * u.ldo + col;
                        if (u.o_vec && col + 8 <= p.N) {
                            *reinterpret_cast<bf16x8*>(out) = o;
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const __bf16 b = o[e];
                                if (col + e < p.N) out[e] = __builtin_bit_cast(uint16_t, b);
                            }
                        }
                    } else {
                        halfx8 nh, nl;
                        split8(x, nh, nl);
                        *reinterpret_cast<halfx8*>(u.hi2 + at) = nh;
                        *reinterpret_cast<halfx8*>(u.lo2 + at) = nl;
                    }
                }
            }
        });
}

// Row and column of lower-triangle tile idx.
__device__ __forceinline__ void lower_pair(int idx, int& bm, int& bn) {
    bm = 0;
    while ((bm + 1) * (bm + 2) / 2 <= idx) ++bm;
    bn = idx - bm * (bm + 1) / 2;
}

// One part of the Gram matrix's sums: tile idx, part, of problem z, kGramTile^2
// floats to its place in `partial`.  XCD x takes a contiguous range of the
// (tiles * splits * batch) workgroups, tiles fastest: it reads one or two parts
// of X, each many times, where workgroups in launch order read all of X through every
// L2 (a whole call on 8192 x 1024 329 us against 348, on 1024 x 8192 328 against 353).
template <bool TA, bool TB, bool kTail>
__global__ __launch_bounds__(NT, 2) void gram_part_kernel(GemmParams p, int kc, int splits,
                                                          int tiles, float* partial) {
    constexpr int R = kGramTile;
    const int x = blockIdx.x % kXcds, q = blockIdx.x / kXcds;
    const int per = gridDim.x / kXcds, rem = gridDim.x % kXcds;
    const int g = x * per + min(x, rem) + q;
    const int idx = g % tiles, part = g / tiles % splits, z = g / tiles / splits;
    int bm, bn;
    lower_pair(idx, bm, bn);
    select_problem(p, z);
    const int k0 = part * kc;
    const int64_t skip = TA ? (int64_t)k0 * p.lda : k0;
    p.A = static_cast<const uint16_t*>(p.A) + skip;
    p.B = static_cast<const uint16_t*>(p.B) + skip;
    p.K = min(kc, p.K - k0);
    float* raw = partial + (((int64_t)z * tiles + idx) * splits + part) * R * R;
    dma_tile<In::F16, R, TA, TB, true, kTail>(p, bm * R, bn * R, raw);
}

// S <- f * the parts' sums, in part order, stored and mirrored.  Each lane
// takes 8 neighbouring elements of a tile's row; a workgroup 16 rows.
__global__ __launch_bounds__(NT) void gram_join_kernel(const float* partial, int splits, int n,
                                                       _Float16* S, int64_t ld, int64_t size,
                                                       float f) {
    constexpr int R = kGramTile;
    __shared__ _Float16 turn[16][R + 2];
    const int idx = blockIdx.x, strip = blockIdx.y;
    int bm, bn;
    lower_pair(idx, bm, bn);
    S += blockIdx.z * size;
    partial += ((int64_t)blockIdx.z * gridDim.x + idx) * splits * R * R;
    const int r = threadIdx.x / 16, c = threadIdx.x % 16 * 8;
    const float* src = partial + (16 * strip + r) * R + c;
    floatx4 s0 = *reinterpret_cast<const floatx4*>(src);
    floatx4 s1 = *reinterpret_cast<const floatx4*>(src + 4);
    for (int i = 1; i < splits; ++i) {
        s0 += *reinterpret_cast<const floatx4*>(src + (int64_t)i * R * R);
        s1 += *reinterpret_cast<const floatx4*>(src + (int64_t)i * R * R + 4);
    }
    halfx8 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o[e] = (_Float16)(f * s0[e]);
        o[4 + e] = (_Float16)(f * s1[e]);
    }
    const int row0 = bm * R + 16 * strip, col0 = bn * R;
    if (row0 + r < n && col0 + c < n)
        *reinterpret_cast<halfx8*>(S + (row0 + r) * ld + col0 + c) = o;
    if (bm == bn) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) turn[r][c + e] = o[e];
    __syncthreads();
    const int col = threadIdx.x / 2, half = threadIdx.x % 2 * 8;  // column of the tile, 8 rows
    halfx8 t;
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = turn[half + e][col];
    if (col0 + col < n && row0 + half < n)
        *reinterpret_cast<halfx8*>(S + (col0 + col) * ld + row0 + half) = t;
}

unsigned grid_for(int64_t items) {
    const int64_t g = (items + NT - 1) / NT;
    return (unsigned)(g < 2048 ? g : 2048);  // grid-stride loops cover the rest
}

GemmParams operands(const Plan& p, int M, int N, int K, const _Float16* A, int64_t lda, int64_t sa,
                    const _Float16* B, int64_t ldb, int64_t sb) {
    GemmParams g = {};
    g.M = M; g.N = N; g.K = K;
    g.A = A; g.lda = lda; g.stride_a = sa * 2;
    g.B = B; g.ldb = ldb; g.stride_b = sb * 2;
    g.batch = p.batch;
    return g;
}

// The tile size with less time by the wave model of the 16-bit kernel (t256,
// t128: tiles of the launch).  Whole calls, us (all 128 / all 256 / as chosen): 1024^2 218 /
// 373 / 219, 2600^2 617 / 862 / 613, 2048 x 8192 816 / 902 / 797, 4096^2 1832 / 1563 / 1561,
// 16 x 1024^2 666 / 640 / 640, 16 x 2048^2 3903 / 3497 / 3494.
bool use128(int64_t t256, int64_t t128) {
    const double time256 = (double)((t256 + kCUs - 1) / kCUs) * 4.0;
    const double time128 = (double)((t128 + 2 * kCUs - 1) / (2 * kCUs)) * 2.0 * 1.22;
    return time128 < time256;
}

template <bool TA, bool TB, bool kAdd>
hipError_t symmetric(const GemmParams& g, _Float16* out, const _Float16* add, float* diag,
                     int64_t ld, int64_t size, float f1, float f2, hipStream_t s) {
    auto go = [&](auto rc) {
        constexpr int R = decltype(rc)::value;
        const int64_t tiles = lower_tiles(g.M, R);
        if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
        auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)tiles, g.batch), dim3(NT), 0, s, g, tiles,
                               out, add, diag, ld, size, f1, f2);
            return hipGetLastError();
        };
        if (g.K % (BK * NSTAGE) != 0) return launch(symmetric_kernel<R, TA, TB, true, true, kAdd>);
        if (g.M % R != 0) return launch(symmetric_kernel<R, TA, TB, true, false, kAdd>);
        return launch(symmetric_kernel<R, TA, TB, false, false, kAdd>);
    };
    return use128(lower_tiles(g.M, 256) * g.batch, lower_tiles(g.M, 128) * g.batch)
               ? go(std::integral_constant<int, 128>{})
               : go(std::integral_constant<int, 256>{});
}

template <bool TB>
hipError_t update(const GemmParams& g, const Update& u, bool last, hipStream_t s) {
    auto go = [&](auto rc, auto lc) {
        constexpr int R = decltype(rc)::value;
        constexpr bool kLast = decltype(lc)::value;
        const int tm = (g.M + R - 1) / R, tn = (g.N + R - 1) / R;
        const int64_t tiles = (int64_t)tm * tn;
        if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
        auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)tiles, g.batch), dim3(NT), 0, s, g, tm, tn, u);
            return hipGetLastError();
        };
        if (g.K % (BK * NSTAGE) != 0) return launch(update_kernel<R, TB, true, true, kLast>);
        if (g.M % R != 0 || g.N % R != 0) return launch(update_kernel<R, TB, true, false, kLast>);
        return launch(update_kernel<R, TB, false, false, kLast>);
    };
    auto tiles = [&](int R) { return (int64_t)((g.M + R - 1) / R) * ((g.N + R - 1) / R) * g.batch; };
    auto size = [&](auto rc) { return last ? go(rc, std::true_type{}) : go(rc, std::false_type{}); };
    return use128(tiles(256), tiles(128)) ? size(std::integral_constant<int, 128>{})
                                          : size(std::integral_constant<int, 256>{});
}

template <bool TA, bool TB>
hipError_t gram(const Plan& p, const GemmParams& g, _Float16* S, float f, uint8_t* ws,
                hipStream_t s) {
    if (p.splits == 1) return symmetric<TA, TB, false>(g, S, nullptr, nullptr, p.lds, p.s_size, f, 0.0f, s);
    float* partial = reinterpret_cast<float*>(ws + p.partial);
    const unsigned tiles = (unsigned)lower_tiles(p.n, kGramTile);
    const dim3 grid(tiles * p.splits * p.batch);  // a few hundred at most (make_plan)
    if (g.K % (BK * NSTAGE) != 0)
        hipLaunchKernelGGL((gram_part_kernel<TA, TB, true>), grid, dim3(NT), 0, s, g, p.kc,
                           p.splits, (int)tiles, partial);
    else
        hipLaunchKernelGGL((gram_part_kernel<TA, TB, false>), grid, dim3(NT), 0, s, g, p.kc,
                           p.splits, (int)tiles, partial);
    hipLaunchKernelGGL(gram_join_kernel, dim3(tiles, kGramTile / 16, p.batch), dim3(NT), 0, s,
                       partial, p.splits, p.n, S, p.lds, p.s_size, f);
    return hipGetLastError();
}

template <In T>
hipError_t norm(const Call& c, int M, int N, int batch, double* parts, hipStream_t s) {
    using E = typename InFmt<T>::S;
    const E* G = static_cast<const E*>(c.G);
    const bool vec = rows_16b_aligned(G, c.ldg, sizeof(E)) && c.stride_g * sizeof(E) % 16 == 0;
    hipLaunchKernelGGL(norm_kernel<T>, dim3(norm_parts(M, N), batch), dim3(NT), 0, s, G, c.ldg,
                       c.stride_g, M, N, vec, parts);
    return hipGetLastError();
}

template <In T>
hipError_t init(const Plan& p, const Call& c, _Float16* hi, _Float16* lo, hipStream_t s) {
    using E = typename InFmt<T>::S;
    const E* G = static_cast<const E*>(c.G);
    double* parts = reinterpret_cast<double*>(c.ws + p.parts);
    const bool vec = rows_16b_aligned(G, c.ldg, sizeof(E)) && c.stride_g * sizeof(E) % 16 == 0;
    const hipError_t e = launch_norm(c, p.M, p.N, p.batch, parts, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(init_kernel<T>, dim3(grid_for(p.x_size / 8), p.batch), dim3(NT), 0, s, G,
                       c.ldg, c.stride_g, p.M, p.N, vec, parts, norm_parts(p.M, p.N), (double)c.eps,
                       std::ldexp(1.0, scale_exp(p.k)), hi, lo, p.ldx);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const Call& c, int M, int N, int batch, double* parts, hipStream_t s) {
    return c.t == In::F32    ? norm<In::F32>(c, M, N, batch, parts, s)
           : c.t == In::BF16 ? norm<In::BF16>(c, M, N, batch, parts, s)
                             : norm<In::F16>(c, M, N, batch, parts, s);
}

hipError_t launch(const Plan& p, const Call& c, hipStream_t s) {
    auto half = [&](int64_t at) { return reinterpret_cast<_Float16*>(c.ws + at); };
    _Float16* hi[2] = {half(p.hi[0]), half(p.hi[1])};
    _Float16* lo[2] = {half(p.lo[0]), half(p.lo[1])};
    _Float16 *S = half(p.gram), *B = half(p.poly);
    float* diag = reinterpret_cast<float*>(c.ws + p.diag);
    hipError_t e = c.t == In::F32    ? init<In::F32>(p, c, hi[0], lo[0], s)
                   : c.t == In::BF16 ? init<In::BF16>(p, c, hi[0], lo[0], s)
                                     : init<In::F16>(p, c, hi[0], lo[0], s);
    const bool tall = p.M > p.N;
    const float xs = std::ldexp(1.0f, scale_exp(p.k));
    Update u = {};
    u.diag = diag;
    u.ldx = p.ldx; u.x_size = p.x_size;
    u.a = c.a; u.f = 1.0f / kPolyScale;
    u.O = c.O; u.ldo = c.ldo; u.stride_o = c.stride_o;
    u.out_scale = 1.0f / xs;
    u.o_vec = rows_16b_aligned(c.O, c.ldo, 2) && c.stride_o % 8 == 0;
    for (int i = 0; i < c.steps && e == hipSuccess; ++i) {
        const int r = i & 1, w = 1 - r;
        // S: rows of X against rows (wide), columns against columns (tall)
        GemmParams g = operands(p, p.n, p.n, p.k, hi[r], p.ldx, p.x_size, hi[r], p.ldx, p.x_size);
        const float fs = kGramScale / (xs * xs);
        e = tall ? gram<true, false>(p, g, S, fs, c.ws, s) : gram<false, true>(p, g, S, fs, c.ws, s);
        if (e != hipSuccess) return e;
        g = operands(p, p.n, p.n, p.n, S, p.lds, p.s_size, S, p.lds, p.s_size);
        e = symmetric<false, true, true>(g, B, S, diag, p.lds, p.s_size,
                                         c.c * (kPolyScale / (kGramScale * kGramScale)),
                                         c.b * (kPolyScale / kGramScale), s);
        if (e != hipSuccess) return e;
        u.hi = hi[r]; u.lo = lo[r];
        u.hi2 = hi[w]; u.lo2 = lo[w];
        const bool last = i + 1 == c.steps;
        if (tall) {
            g = operands(p, p.M, p.N, p.n, hi[r], p.ldx, p.x_size, B, p.lds, p.s_size);
            g.tb = 1;
            e = update<true>(g, u, last, s);
        } else {
            g = operands(p, p.M, p.N, p.n, B, p.lds, p.s_size, hi[r], p.ldx, p.x_size);
            e = update<false>(g, u, last, s);
        }
    }
    return e;
}

}  // namespace orth
}  // namespace dgt
