// k_orth_small.hip -- Newton-Schulz steps of matrices too small for the tile
// kernels (k_orth.hip): 15 products of a few microseconds each, where what
// counts is the latency of one.
//
// A workgroup computes one 32 x 32 tile, its four waves a quarter of k each:
// operands go from memory (L2) straight into the matrix cores' layout, 16
// bytes (8 k) per lane, no LDS and no barrier before the one that joins the
// four partial sums.  The code is short: a tile kernel's long straight epilogue
// costs a launch of this size as much in instruction fetches as its work does.
// That wants every operand stored with k contiguous, so X is kept both ways round
// (x, and transposed xt), a tall G is taken transposed, and symmetric
// products are simply computed whole.  Every matrix is padded with zeros to
// multiples of 64; products of zero rows are zero, so the padding stays zero by
// itself and nothing is masked.
//
// Precision as in k_orth.hip: X = hi + lo, products read hi, a X both; what
// rounding takes from B's diagonal is added to the update in fp32.
#include "orth.hpp"

namespace dgt {
namespace orth {

namespace {

constexpr int T = 32, NW = 4;
constexpr int NTI = 256;

typedef _Float16 halfx4 __attribute__((ext_vector_type(4)));

// x, xt, lo (xt's layout) <- G * scale / (|G| + eps), zeros in the padding; kTall: X = G^T.
// One lane per element of x.
template <In E, bool kTall>
__global__ __launch_bounds__(NTI) void small_init_kernel(const typename InFmt<E>::S* G, int64_t ldg,
                                                         int64_t stride, SmallPlan p,
                                                         const double* parts, int nparts, double eps,
                                                         double scale, _Float16* x, _Float16* xt,
                                                         _Float16* lo) {
    const int64_t z = blockIdx.y;
    G += z * stride;
    x += z * p.x_size;
    xt += z * p.x_size;
    lo += z * p.x_size;
    __shared__ double red[NTI];
    double sum = 0.0;
    for (int i = threadIdx.x; i < nparts; i += NTI) sum += parts[z * nparts + i];
    red[threadIdx.x] = sum;
    __syncthreads();
    for (int h = NTI / 2; h > 0; h /= 2) {
        if ((int)threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
        __syncthreads();
    }
    const double inv = scale / (sqrt(red[0]) + eps);
    for (int64_t e = (int64_t)blockIdx.x * NTI + threadIdx.x; e < p.x_size;
         e += (int64_t)gridDim.x * NTI) {
        const int i = (int)(e / p.k64), j = (int)(e % p.k64);
        float v = 0.0f;
        if (i < p.n && j < p.k)
            v = (float)((double)load_in<E>(G + (kTall ? (int64_t)j * ldg + i : (int64_t)i * ldg + j)) * inv);
        const _Float16 h = (_Float16)v;
        x[e] = h;
        xt[(int64_t)j * p.n64 + i] = h;
        lo[(int64_t)j * p.n64 + i] = (_Float16)(v - (float)h);
    }
}

// What becomes of a tile's sums.  Lane l of the joining wave holds column
// l % 32 and rows 8q + 4(l/32) .. +3 (q = 0 .. 3) of the 32 x 32 tile.
enum class Kind { Gram, Poly, Update, Last };
struct Out {
    _Float16* a;        // Gram: S; Poly: B; Update: x (row-major)
    _Float16 *at, *lo;  // Update: xt and lo
    const _Float16 *prev, *prev_lo;  // Poly: S; Update, Last: xt and lo of X
    float* diag;        // what rounding took from B's diagonal (n64 floats)
    uint16_t* O;        // Last
    int64_t ldo, stride_o;
    int M, N;
    float f, g;         // Gram: f * sums; Poly: g * S + f * sums; Update: g * X + f * (sums + diag x)
    float out_scale;
};

// sums = A B^T over k: A rows of `rows` (lda), B rows of `cols`; both row
// pitches are k's padded length.
template <Kind K, bool kTall>
__global__ __launch_bounds__(64 * NW) void small_product_kernel(const _Float16* A, const _Float16* B,
                                                                int64_t size_a, int64_t size_b,
                                                                int64_t size_out, int kpad,
                                                                int tiles_n, int rows, int cols,
                                                                Out o) {
    __shared__ floatx4 part[NW][4][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t z = blockIdx.y;
    const int m0 = (int)(blockIdx.x / tiles_n) * T, n0 = (int)(blockIdx.x % tiles_n) * T;
    // lane l: row l % 32 of the tile, 8 k from 8 * (l / 32) on
    const int64_t off = 8 * (lane >> 5);
    const _Float16* a = A + z * size_a + (int64_t)(m0 + (lane & 31)) * kpad + off;
    const _Float16* b = B + z * size_b + (int64_t)(n0 + (lane & 31)) * kpad + off;
    floatx16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
    // The wave's 16-deep steps: wave, wave + 4, .. (kpad is a multiple of 64);
    // up to U of them are loaded before the first is used.
    constexpr int U = 4;
    const int steps = kpad / (16 * NW);
    for (int i0 = 0; i0 < steps; i0 += U) {
        u32x4 fa[U], fb[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + i < steps) {
                const int k = 16 * (NW * (i0 + i) + wave);
                fa[i] = *reinterpret_cast<const u32x4*>(a + k);
                fb[i] = *reinterpret_cast<const u32x4*>(b + k);
            }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + i < steps) acc = mfma32x32x16<In::F16>(fa[i], fb[i], acc);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
        part[wave][q][lane] = floatx4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    __syncthreads();
    const int q = wave;  // wave q joins the four rows of quarter q
    floatx4 sum = part[0][q][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += part[w][q][lane];
    const int m = m0 + 8 * q + 4 * (lane >> 5), n = n0 + (lane & 31);
    const int64_t t = z * size_out + (int64_t)n * rows + m;  // 4 neighbours of the transposed layout
    float* diag = o.diag + z * rows;
    if constexpr (K == Kind::Gram || K == Kind::Poly) {  // symmetric: stored transposed
        halfx4 v;
        if constexpr (K == Kind::Poly) {
            const halfx4 s = *reinterpret_cast<const halfx4*>(o.prev + t);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float b = o.g * (float)s[r] + o.f * sum[r];
                v[r] = (_Float16)b;
                if (m + r == n) diag[n] = b - (float)v[r];
            }
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = (_Float16)(o.f * sum[r]);
        }
        *reinterpret_cast<halfx4*>(o.a + t) = v;
    } else {
        const halfx4 h = *reinterpret_cast<const halfx4*>(o.prev + t);
        const halfx4 l = *reinterpret_cast<const halfx4*>(o.prev_lo + t);
        const floatx4 d = *reinterpret_cast<const floatx4*>(diag + m);
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r] = o.g * ((float)h[r] + (float)l[r]) + o.f * fmaf(d[r], (float)h[r], sum[r]);
        if constexpr (K == Kind::Update) {
            halfx4 nh, nl;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                nh[r] = (_Float16)x[r];
                nl[r] = (_Float16)(x[r] - (float)nh[r]);
                o.a[z * size_out + (int64_t)(m + r) * cols + n] = nh[r];
            }
            *reinterpret_cast<halfx4*>(o.at + t) = nh;
            *reinterpret_cast<halfx4*>(o.lo + t) = nl;
        } else {
            uint16_t* O = o.O + z * o.stride_o;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const __bf16 v = (__bf16)(x[r] * o.out_scale);
                const int i = kTall ? n : m + r, j = kTall ? m + r : n;
                if (i < o.M && j < o.N) O[(int64_t)i * o.ldo + j] = __builtin_bit_cast(uint16_t, v);
            }
        }
    }
}

template <Kind K>
hipError_t product(const SmallPlan& p, bool tall, const _Float16* A, const _Float16* B,
                   int64_t size_a, int64_t size_b, int64_t size_out, int rows, int cols, int kpad,
                   const Out& o, hipStream_t s) {
    const dim3 grid((unsigned)(rows / T * (cols / T)), p.batch);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(64 * NW), 0, s, A, B, size_a, size_b, size_out, kpad,
                           cols / T, rows, cols, o);
        return hipGetLastError();
    };
    return K == Kind::Last && tall ? go(small_product_kernel<K, K == Kind::Last>)
                                   : go(small_product_kernel<K, false>);
}

template <In E>
hipError_t init(const SmallPlan& p, const Call& c, const double* parts, _Float16* x, _Float16* xt,
                _Float16* lo, hipStream_t s) {
    const int64_t wgs = (p.x_size + NTI - 1) / NTI;
    const dim3 grid((unsigned)(wgs < 1024 ? wgs : 1024), p.batch);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(NTI), 0, s,
                           static_cast<const typename InFmt<E>::S*>(c.G), c.ldg, c.stride_g, p, parts,
                           norm_parts(p.M, p.N), (double)c.eps, std::ldexp(1.0, scale_exp(p.k)), x, xt, lo);
        return hipGetLastError();
    };
    return p.M > p.N ? go(small_init_kernel<E, true>) : go(small_init_kernel<E, false>);
}

}  // namespace

hipError_t launch_small(const SmallPlan& p, const Call& c, hipStream_t s) {
    auto half = [&](int64_t at) { return reinterpret_cast<_Float16*>(c.ws + at); };
    _Float16 *S = half(p.gram), *B = half(p.poly);
    double* parts = reinterpret_cast<double*>(c.ws + p.parts);
    hipError_t e = launch_norm(c, p.M, p.N, p.batch, parts, s);
    if (e != hipSuccess) return e;
    e = c.t == In::F32    ? init<In::F32>(p, c, parts, half(p.x[0]), half(p.xt[0]), half(p.lo[0]), s)
        : c.t == In::BF16 ? init<In::BF16>(p, c, parts, half(p.x[0]), half(p.xt[0]), half(p.lo[0]), s)
                          : init<In::F16>(p, c, parts, half(p.x[0]), half(p.xt[0]), half(p.lo[0]), s);
    const float xs = std::ldexp(1.0f, scale_exp(p.k));
    const bool tall = p.M > p.N;
    for (int i = 0; i < c.steps && e == hipSuccess; ++i) {
        const int r = i & 1, w = 1 - r;
        const _Float16 *x = half(p.x[r]), *xt = half(p.xt[r]);
        Out o = {};
        o.diag = reinterpret_cast<float*>(c.ws + p.diag);
        o.a = S;
        o.f = kGramScale / (xs * xs);
        e = product<Kind::Gram>(p, tall, x, x, p.x_size, p.x_size, p.s_size, p.n64, p.n64, p.k64, o, s);
        if (e != hipSuccess) return e;
        o.a = B;
        o.prev = S;
        o.f = c.c * (kPolyScale / (kGramScale * kGramScale));
        o.g = c.b * (kPolyScale / kGramScale);
        e = product<Kind::Poly>(p, tall, S, S, p.s_size, p.s_size, p.s_size, p.n64, p.n64, p.n64, o, s);
        if (e != hipSuccess) return e;
        // X' = a X + B X: rows of B against rows of xt
        o.a = half(p.x[w]);
        o.at = half(p.xt[w]);
        o.lo = half(p.lo[w]);
        o.prev = xt;
        o.prev_lo = half(p.lo[r]);
        o.f = 1.0f / kPolyScale;
        o.g = c.a;
        if (i + 1 < c.steps) {
            e = product<Kind::Update>(p, tall, B, xt, p.s_size, p.x_size, p.x_size, p.n64, p.k64,
                                      p.n64, o, s);
        } else {
            o.O = c.O; o.ldo = c.ldo; o.stride_o = c.stride_o;
            o.M = p.M; o.N = p.N;
            o.out_scale = 1.0f / xs;
            e = product<Kind::Last>(p, tall, B, xt, p.s_size, p.x_size, p.x_size, p.n64, p.k64,
                                    p.n64, o, s);
        }
    }
    return e;
}

}  // namespace orth
}  // namespace dgt
