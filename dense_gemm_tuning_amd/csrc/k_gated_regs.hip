// k_gated_regs.hip -- the gated projections and their gradient for operands of
// any alignment, staged through registers.
//
// Tile BM rows by BB products, 2 x 2 wavefronts of BM/2 x BB/2 (v_mfma_f32_32x32x16).
// Forward: a wavefront's 64 products are 32 of the gate and
// the same 32 columns of the other projection, so that both pre-activations of
// an element end up in one lane.  Gradient: BB columns of dh.
//
// K advances in slices of 64, the next one loaded into registers while the
// current one is multiplied from LDS (two buffers, one barrier a slice), 16 bytes at a time
// from wherever a row starts (the GPU runs with unaligned access enabled), rows past the
// end re-reading the last one (their products are not stored).
// Chunk q (8 k) of row r sits at q ^ ((r ^ r>>3) & 7).
#include "dma_common.hpp"
#include "gated.hpp"

namespace dgt {
namespace gated {

namespace {

constexpr int BK = 64, NT = 256, CPR = BK / 8;

__device__ __forceinline__ int swz(int r) { return (r ^ (r >> 3)) & 7; }

// In the loads below a whole 16 bytes lies inside the row: those of a piece that crosses its end
// or lies behind it are the row's last ones, put right where they are stored to LDS (a load's
// value used before the products would be waited for there).  Rows of fewer than 8 are gathered.
__device__ __forceinline__ int past_end(int at, int limit) {
    return limit >= 8 ? min(max(at - (limit - 8), 0), 8) : 0;
}

// An operand stored with k contiguous, R rows of it: lane chunk i is staged row tid/8 + 32*i,
// chunk tid%8.
template <int R>
struct Rows {
    static constexpr int C = R / 32;
    const uint16_t* row[C];
    u32x4 v[C];
    int at, K;
    template <bool kFirst>
    __device__ void load(std::bool_constant<kFirst>, int k0, int K_, int q) {
        at = k0 + 8 * q;
        K = K_;
        if (kFirst && K < 8) {  // uniform; then there is one slice
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = gather8(row[i], at, K);
            return;
        }
        const int from = min(at, K - 8);
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = load16(row[i] + from);
    }
    __device__ void store(u32x4* dst, int tid) const {
        const bool cut = at - 8 * (tid & 7) + BK > K;  // uniform
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int r = (tid >> 3) + 32 * i;
            dst[r * CPR + ((tid & 7) ^ swz(r))] = cut ? shift_out(v[i], past_end(at, K)) : v[i];
        }
    }
};

// An operand stored K x N, BB columns of it: the lane takes KR k-rows from KR*(tid/G) on,
// columns 8*(tid%G) .. +7 of the tile, and writes them as eight columns of KR k.  kNarrow: N < 8.
template <int BB, bool kNarrow>
struct Columns {
    static constexpr int G = BB / 8, KR = BK * G / NT;
    static_assert(KR == 2 || KR == 4, "whole dwords, inside a chunk");
    u32x4 v[KR];
    int col, N, k, K;
    bool cut;  // the slice or the tile crosses an end (uniform)
    __device__ void load(const uint16_t* W, int64_t ld, int n0, int N_, int k0, int K_, int tid) {
        N = N_;
        K = K_;
        col = n0 + 8 * (tid % G);
        k = k0 + KR * (tid / G);
        cut = k0 + BK > K || n0 + BB > N;
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const uint16_t* row = W + (int64_t)min(k + i, K - 1) * ld;
            if (kNarrow) v[i] = gather8(row, col, N);
            else v[i] = load16(row + min(col, N - 8));
        }
    }
    __device__ void store(u32x4* dst, int tid) {
        const int kk = KR * (tid / G);
        if (cut) {
            const int past = past_end(col, N);
#pragma unroll
            for (int i = 0; i < KR; ++i) v[i] = shift_out(v[i], k + i < K ? past : 8);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int n = 8 * (tid % G) + j;
            uint32_t c[KR / 2];
#pragma unroll
            for (int e = 0; e < KR / 2; ++e) {
                const uint32_t a = v[2 * e][j / 2], b = v[2 * e + 1][j / 2];
                c[e] = j % 2 ? (a >> 16) | (b & 0xffff0000u) : (a & 0xffffu) | (b << 16);
            }
            uint32_t* to =
                reinterpret_cast<uint32_t*>(dst + n * CPR + ((kk / 8) ^ swz(n))) + kk % 8 / 2;
            __builtin_memcpy(__builtin_assume_aligned(to, 2 * KR), c, 2 * KR);
        }
    }
};

struct Place {
    int lane, wm, wn, h, c;  // h: half of the wavefront, c: its column
};

// The sums of one tile; load and store move slice k0 of both operands.
template <In T, int BM, int BB, typename Load, typename Store>
__device__ __forceinline__ void products(int K, const u32x4 (*As)[BM * CPR],
                                         const u32x4 (*Bs)[BB * CPR], const Place& at, Load&& load,
                                         Store&& store, floatx16 (&acc)[BM / 64][BB / 64]) {
#pragma unroll
    for (int i = 0; i < BM / 64; ++i)
#pragma unroll
        for (int j = 0; j < BB / 64; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    const int nk = K / BK + (K % BK != 0);
    if (nk == 0) return;
    load(std::true_type{}, 0);
    store(0);
    __syncthreads();
    for (int t = 0; t < nk; ++t) {
        const int buf = t & 1;
        if (t + 1 < nk) load(std::false_type{}, (t + 1) * BK);
#pragma unroll
        for (int s = 0; s < BK / 16; ++s) {
            const int q = 2 * s + at.h;
            u32x4 a[BM / 64], b[BB / 64];
#pragma unroll
            for (int i = 0; i < BM / 64; ++i) {
                const int r = at.wm * (BM / 2) + i * 32 + at.c;
                a[i] = As[buf][r * CPR + (q ^ swz(r))];
            }
#pragma unroll
            for (int j = 0; j < BB / 64; ++j) {
                const int r = at.wn * (BB / 2) + j * 32 + at.c;
                b[j] = Bs[buf][r * CPR + (q ^ swz(r))];
            }
#pragma unroll
            for (int i = 0; i < BM / 64; ++i)
#pragma unroll
                for (int j = 0; j < BB / 64; ++j) acc[i][j] = mfma32x32x16<T>(a[i], b[j], acc[i][j]);
        }
        if (t + 1 < nk) store(buf ^ 1);
        __syncthreads();
    }
}

__device__ __forceinline__ Place place() {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    return Place{lane, wave >> 1, wave & 1, lane >> 5, lane & 31};
}

// Row of register r of an MFMA tile (32x32 accumulator layout).
__device__ __forceinline__ int acc_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

template <In T, int BM>
__global__ __launch_bounds__(NT, 2) void forward_regs_kernel(Forward p, int tiles_n) {
    constexpr int BB = 128;
    __shared__ u32x4 As[2][BM * CPR], Bs[2][BB * CPR];
    const int tid = threadIdx.x;
    const Place at = place();
    const int m0 = (int)(blockIdx.x / (unsigned)tiles_n) * BM;
    const int n0 = (int)(blockIdx.x % (unsigned)tiles_n) * (BB / 2);
    Rows<BM> ra;
    Rows<BB> rb;
#pragma unroll
    for (int i = 0; i < BM / 32; ++i)
        ra.row[i] = p.X + (int64_t)min(m0 + (tid >> 3) + 32 * i, p.M - 1) * p.ldx;
#pragma unroll
    for (int i = 0; i < BB / 32; ++i) {
        const int r = (tid >> 3) + 32 * i;
        const int64_t n = min(n0 + 32 * (r / 64) + r % 32, p.N - 1);
        rb.row[i] = (r / 32) % 2 ? p.Wu + n * p.ldwu : p.Wg + n * p.ldwg;
    }
    floatx16 acc[BM / 64][BB / 64];
    products<T, BM, BB>(
        p.K, As, Bs, at,
        [&](auto first, int k0) {
            ra.load(first, k0, p.K, tid & 7);
            rb.load(first, k0, p.K, tid & 7);
        },
        [&](int buf) {
            ra.store(As[buf], tid);
            rb.store(Bs[buf], tid);
        },
        acc);
    const int col = n0 + 32 * at.wn + at.c;
    if (col >= p.N) return;
    const float bg = p.bg ? p.bg[col] : 0.0f, bu = p.bu ? p.bu[col] : 0.0f;
#pragma unroll
    for (int i = 0; i < BM / 64; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int64_t row = m0 + BM / 2 * at.wm + 32 * i + acc_row(r, at.h);
            if (row >= p.M) continue;
            const float g = acc[i][0][r] + bg, u = acc[i][1][r] + bu;
            p.H[row * p.ldh + col] = to_bits<T>(act_of(p.act, g) * u);
            if (p.G) p.G[row * p.ldg + col] = to_bits<T>(g);
            if (p.U) p.U[row * p.ldu + col] = to_bits<T>(u);
        }
}

template <In T, int BM, int BB, bool kNarrow>
__global__ __launch_bounds__(NT, 2) void grad_regs_kernel(Grad p, int tiles_n) {
    __shared__ u32x4 As[2][BM * CPR], Bs[2][BB * CPR];
    const int tid = threadIdx.x;
    const Place at = place();
    const int bm = (int)(blockIdx.x / (unsigned)tiles_n);
    const int m0 = bm * BM, n0 = (int)(blockIdx.x % (unsigned)tiles_n) * BB;
    Rows<BM> ra;
    Columns<BB, kNarrow> rb;
#pragma unroll
    for (int i = 0; i < BM / 32; ++i)
        ra.row[i] = p.dY + (int64_t)min(m0 + (tid >> 3) + 32 * i, p.M - 1) * p.lddy;
    floatx16 acc[BM / 64][BB / 64];
    products<T, BM, BB>(
        p.K, As, Bs, at,
        [&](auto first, int k0) {
            ra.load(first, k0, p.K, tid & 7);
            rb.load(p.Wd, p.ldw, n0, p.N, k0, p.K, tid);
        },
        [&](int buf) {
            ra.store(As[buf], tid);
            rb.store(Bs[buf], tid);
        },
        acc);
#pragma unroll
    for (int j = 0; j < BB / 64; ++j) {
        const int col = n0 + BB / 2 * at.wn + 32 * j + at.c;
        const int64_t from = min(col, p.N - 1);
        float sg = 0.0f, su = 0.0f;
#pragma unroll
        for (int i = 0; i < BM / 64; ++i) {
            // R rows' loads first, those past the edges from the last row or column: behind a
            // branch each would wait for one another
            constexpr int R = 8;
#pragma unroll
            for (int r0 = 0; r0 < 16; r0 += R) {
                // opaque: the addresses of all rows made ahead would not fit the registers
                int row0 = m0 + BM / 2 * at.wm + 32 * i;
                asm volatile("" : "+v"(row0));
                uint16_t g[R], u[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int64_t row = min(row0 + acc_row(r0 + r, at.h), p.M - 1);
                    g[r] = p.G[row * p.ldg + from];
                    u[r] = p.U[row * p.ldu + from];
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int64_t row = row0 + acc_row(r0 + r, at.h);
                    const GradOut o = grad_at(p.act, acc[i][j][r0 + r], InFmt<T>::widen(g[r]),
                                              InFmt<T>::widen(u[r]));
                    if (row >= p.M || col >= p.N) continue;
                    p.dG[row * p.lddg + col] = to_bits<T>(o.dg);
                    p.dU[row * p.lddu + col] = to_bits<T>(o.du);
                    if (p.H) p.H[row * p.ldh + col] = to_bits<T>(o.h);
                    sg += o.dg;
                    su += o.du;
                }
            }
        }
        if (!p.parts) continue;  // uniform
        // a part is kPartRows rows: a wavefront's, or two wavefronts' joined in LDS
        sg += __shfl_xor(sg, 32);
        su += __shfl_xor(su, 32);
        constexpr bool kJoin = BM / 2 < kPartRows;
        float* half = reinterpret_cast<float*>(As[0]) + 2 * (BB / 2 * at.wn + 32 * j + at.c);
        if (kJoin) {
            if (at.wm == 1 && at.h == 0) half[0] = sg, half[1] = su;
            __syncthreads();
            if (at.wm == 0) sg += half[0], su += half[1];
        }
        const int64_t at_part = kJoin ? bm : 2 * (int64_t)bm + at.wm;
        if (at.h == 0 && col < p.N && (!kJoin || at.wm == 0)) {
            float* part = p.parts + 2 * at_part * p.N;
            part[col] = sg;
            part[p.N + col] = su;
        }
    }
}

// Sums over the parts: 64 columns a workgroup, four lanes a column, each every
// fourth part, joined in order.  Columns run over dG's and then dU's.
__global__ __launch_bounds__(NT) void join_kernel(const float* parts, int64_t n_parts, int N,
                                                  float* dbg, float* dbu) {
    __shared__ float part[4][64];
    const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + c;
    float sum = 0.0f;
    if (col < 2 * (int64_t)N)
        for (int64_t i = q; i < n_parts; i += 4) sum += parts[2 * i * N + col];
    part[q][c] = sum;
    __syncthreads();
    if (q != 0 || col >= 2 * (int64_t)N) return;
    sum = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
    if (col < N) {
        if (dbg) dbg[col] = sum;
    } else if (dbu) {
        dbu[col - N] = sum;
    }
}

bool launchable(int64_t wgs) { return wgs < (int64_t(1) << 32) / NT; }

}  // namespace

// Tiles of 64 rows (gradient: 64 x 64) where those of 128 would leave CUs without one (us, 64
// against 128, forward and gradient at K = 1001: 16 x 1000 17.7/23.1 and 16.3/35.4, 1000 x 1000
// 21.6/29.9 and 20.0/40.9, 1500 x 1000 25.9/30.3 and 21.6/41.6).  What bounds them is the
// loads of rows that start off 16-byte boundaries: 2048 x 8192 x 1001 forward takes 141 us here and
// 87 on the DMA tiles when its rows are 1008 apart.
template <In T, int BM>
hipError_t launch_forward_rows(const Forward& p, hipStream_t s) {
    const int64_t tiles_n = ((int64_t)p.N + 63) / 64;
    const int64_t wgs = tiles_n * (((int64_t)p.M + BM - 1) / BM);
    if (BM == 128 && wgs < dma::kCUs) return launch_forward_rows<T, 64>(p, s);
    if (!launchable(wgs)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((forward_regs_kernel<T, BM>), dim3((unsigned)wgs), dim3(NT), 0, s, p,
                       (int)tiles_n);
    return hipGetLastError();
}

template <In T, int B>
hipError_t launch_grad_rows(const Grad& p, int64_t* parts, hipStream_t s) {
    const int64_t tiles_n = ((int64_t)p.N + B - 1) / B, tiles_m = ((int64_t)p.M + B - 1) / B;
    const int64_t wgs = tiles_n * tiles_m;
    if (B == 128 && wgs < dma::kCUs) return launch_grad_rows<T, 64>(p, parts, s);
    if (!launchable(wgs)) return hipErrorInvalidConfiguration;
    *parts = B / kPartRows * tiles_m;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)wgs), dim3(NT), 0, s, p, (int)tiles_n);
        return hipGetLastError();
    };
    return p.N < 8 ? go(grad_regs_kernel<T, B, B, true>) : go(grad_regs_kernel<T, B, B, false>);
}

template <In T>
hipError_t launch_forward_regs(const Forward& p, hipStream_t s) {
    return launch_forward_rows<T, 128>(p, s);
}

template <In T>
hipError_t launch_grad_regs(const Grad& p, int64_t* parts, hipStream_t s) {
    return launch_grad_rows<T, 128>(p, parts, s);
}

hipError_t launch_join(const float* parts, int64_t n_parts, int N, float* dbg, float* dbu,
                       hipStream_t s) {
    const int64_t wgs = (2 * (int64_t)N + 63) / 64;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)wgs), dim3(NT), 0, s, parts, n_parts, N, dbg,
                       dbu);
    return hipGetLastError();
}

template hipError_t launch_forward_regs<In::BF16>(const Forward&, hipStream_t);
template hipError_t launch_forward_regs<In::F16>(const Forward&, hipStream_t);
template hipError_t launch_grad_regs<In::BF16>(const Grad&, int64_t*, hipStream_t);
template hipError_t launch_grad_regs<In::F16>(const Grad&, int64_t*, hipStream_t);

}  // namespace gated
}  // namespace dgt
