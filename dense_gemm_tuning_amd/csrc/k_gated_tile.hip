// k_gated_tile.hip -- the gated projections and their gradient on the 16-bit
// DMA tiles (mfma16_tile.hpp), for operands whose rows are 16-byte aligned.
//
// Forward: of a wavefront's 128 (or 64) products a row, half are the gate's and
// half the other projection's at the same columns; the tile's copies of the
// weights choose between the two matrices, and the K loop is the plain
// product's with both operands k-contiguous.  Gradient: the plain product dY*Wd,
// with Wd as stored.
//
// Epilogues go through the wavefront's LDS region, 32 rows at a time, so that a lane
// has 8 neighbouring columns of a row, of both projections, and loads and
// stores 16 bytes.  Their outer loops are not unrolled: a tile runs its epilogue
// once, and straight code would be fetched from memory as it runs.
#include "gated.hpp"
#include "mfma16_tile.hpp"

namespace dgt {
namespace gated {

namespace {

using namespace mfma16;

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Eight 16-bit values at columns col .. col+7 of a row of N, at any alignment.
template <In T, bool kEdge>
__device__ __forceinline__ void store8(uint16_t* row, int col, int N, const float (&x)[8]) {
    uint16_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = to_bits<T>(x[e]);
    if (!kEdge || col + 8 <= N) {
        u32x4_any v;
#pragma unroll
        for (int d = 0; d < 4; ++d) v[d] = b[2 * d] | ((uint32_t)b[2 * d + 1] << 16);
        // the tiles' stores arrive as bursts, which drain sooner non-temporal (4096 x 14336
        // x 4096 forward 848 -> 777 us, 8192 x 4096 x 1024 gradient 125 -> 112)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(row + col));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < N) row[col + e] = b[e];
    }
}
template <In T>
__device__ __forceinline__ float widen(const u32x4& v, int e) {
    return InFmt<T>::widen((uint16_t)(v[e / 2] >> (16 * (e % 2))));
}

// f(std::integral_constant<Act, act>): one branch for many elements.
template <typename F>
__device__ __forceinline__ void with_act(Act act, F&& f) {
    switch (act) {
        case Act::Silu: f(std::integral_constant<Act, Act::Silu>{}); break;
        case Act::Gelu: f(std::integral_constant<Act, Act::Gelu>{}); break;
        case Act::GeluTanh: f(std::integral_constant<Act, Act::GeluTanh>{}); break;
        case Act::Relu: f(std::integral_constant<Act, Act::Relu>{}); break;
        case Act::Sigmoid: f(std::integral_constant<Act, Act::Sigmoid>{}); break;
        default: f(std::integral_constant<Act, Act::Identity>{}); break;
    }
}

// Tile row ti's accumulators into the wavefront's region; ti is not known at
// compile time, the registers are.
template <int R>
__device__ __forceinline__ void put_row(const Chunk<R>& chunk, const floatx16 (&acc)[Geo<R>::TM][Geo<R>::TM],
                                        int ti, int lane) {
#pragma unroll
    for (int i = 0; i < Geo<R>::TM; ++i)
        if (ti == i) chunk.put(acc[i], lane);
}

template <In T, int R, bool kEdge, bool kTail>
__global__ __launch_bounds__(NT, R == 256 ? 1 : 2) void forward_tile_kernel(GemmParams g, Forward p,
                                                                          int tiles_m, int tiles_n) {
    // XCD-grouped tiles, unlike the plain product with both operands k-contiguous:
    // 8192^3 1683 us against 1976 in row order (with the stores below 1647)
    const TileIdx tile = xcd_tile(tiles_m, tiles_n, true);
    const int m0 = tile.bm * R, n0 = tile.bn * (R / 2);
    dma_tile<T, R, false, true, kEdge, kTail>(
        g, m0, n0, nullptr,
        [&](const auto& acc, int wm, int wn, int lane, uint8_t* mem) DGT_INLINE {
            using Ch = Chunk<R>;
            const Ch chunk{reinterpret_cast<float*>(mem)};
            constexpr int W = R / 4, GROUPS = W / 8;  // columns of either projection, and lanes a row
            const int row0 = m0 + wm * (R / 2), c = lane % GROUPS * 8, col = n0 + wn * W + c;
            float bg[8], bu[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = !kEdge || col + e < p.N;
                bg[e] = p.bg && in ? p.bg[col + e] : 0.0f;
                bu[e] = p.bu && in ? p.bu[col + e] : 0.0f;
            }
#pragma unroll 1
            for (int ti = 0; ti < Geo<R>::TM; ++ti) {
                put_row<R>(chunk, acc, ti, lane);
#pragma unroll
                for (int r = lane / GROUPS; r < 32; r += 64 / GROUPS) {
                    const int64_t row = row0 + 32 * ti + r;
                    if (kEdge && (row >= p.M || col >= p.N)) continue;
                    float x[8], u[8], h[8];
                    chunk.row8(r, c, x);
                    chunk.row8(r, W + c, u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] += bg[e], u[e] += bu[e];
                    with_act(p.act, [&](auto a) DGT_INLINE {
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = act_of(decltype(a)::value, x[e]) * u[e];
                    });
                    store8<T, kEdge>(p.H + row * p.ldh, col, p.N, h);
                    if (p.G) store8<T, kEdge>(p.G + row * p.ldg, col, p.N, x);
                    if (p.U) store8<T, kEdge>(p.U + row * p.ldu, col, p.N, u);
                }
            }
        },
        TwoB{p.Wu, p.ldwu});
}

// The gradient's epilogue of one wavefront, its rows from row0 and columns from
// colw on.  kEdge: rows or columns may lie past the end.  Pieces (8 columns of a row) are
// loaded B ahead: 8 KB in flight a wavefront at 256 x 256, 4 at 128 x 128, where there are twice
// the wavefronts (at an edge 4 at either: more goes to scratch memory).
template <In T, int R, bool kEdge>
__device__ __forceinline__ void grad_epilogue(const Grad& p, const floatx16 (&acc)[Geo<R>::TM][Geo<R>::TM],
                                              int row0, int colw, int part, int lane, uint8_t* mem) {
    using Ch = Chunk<R>;
    const Ch chunk{reinterpret_cast<float*>(mem)};
    constexpr int B = kEdge ? 2 : R / 64, BATCHES = Ch::PIECES / B, ALL = Geo<R>::TM * BATCHES;
    static_assert(Ch::PIECES % B == 0 && 64 % Ch::GROUPS == 0, "a lane's columns are one group's");
    const int c = Ch::col(0, lane), col = colw + c;
    const int past = kEdge && p.N >= 8 ? min(max(col - (p.N - 8), 0), 8) : 0;
    u32x4 vg[B], vu[B];
    float sg[8], su[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sg[e] = su[e] = 0.0f;
    auto row_of = [&](int b, int i) DGT_INLINE {  // piece i of batch b, in the wavefront's rows
        return 32 * (b / BATCHES) + Ch::row(B * (b % BATCHES) + i, lane);
    };
    auto fetch = [&](int b) DGT_INLINE {
#pragma unroll
        for (int i = 0; i < B; ++i) {
            // rows past the end re-read the last one
            const int64_t row = kEdge ? min(row0 + row_of(b, i), p.M - 1) : row0 + row_of(b, i);
            const uint16_t *g = p.G + row * p.ldg, *u = p.U + row * p.ldu;
            if (kEdge && p.N < 8) {  // uniform
                vg[i] = gather8(g, col, p.N);
                vu[i] = gather8(u, col, p.N);
            } else {  // what crosses a row's end is shifted where it is used
                const int from = kEdge ? min(col, p.N - 8) : col;
                vg[i] = load16(g + from);
                vu[i] = load16(u + from);
            }
        }
    };
    with_act(p.act, [&](auto a) DGT_INLINE {
        fetch(0);
#pragma unroll 1
        for (int b = 0; b < ALL; ++b) {
            u32x4 cg[B], cu[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                cg[i] = kEdge ? shift_out(vg[i], past) : vg[i];
                cu[i] = kEdge ? shift_out(vu[i], past) : vu[i];
            }
            if (b + 1 < ALL) fetch(b + 1);
            if (b % BATCHES == 0) put_row<R>(chunk, acc, b / BATCHES, lane);
#pragma unroll
            for (int i = 0; i < B; ++i) {
                __builtin_amdgcn_sched_barrier(0);  // one piece's values at a time
                const int r = row_of(b, i);
                const int64_t row = row0 + r;
                const bool in = !kEdge || (row < p.M && col < p.N);
                float dg[8], du[8], h[8], dh[8];
                chunk.row8(r % 32, c, dh);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const GradOut o =
                        grad_at(decltype(a)::value, dh[e], widen<T>(cg[i], e), widen<T>(cu[i], e));
                    dg[e] = o.dg;
                    du[e] = o.du;
                    h[e] = o.h;
                    sg[e] += in ? o.dg : 0.0f;
                    su[e] += in ? o.du : 0.0f;
                }
                if (in) {
                    store8<T, kEdge>(p.dG + row * p.lddg, col, p.N, dg);
                    store8<T, kEdge>(p.dU + row * p.lddu, col, p.N, du);
                    if (p.H) store8<T, kEdge>(p.H + row * p.ldh, col, p.N, h);
                }
            }
        }
    });
    if (!p.parts) return;
    // the lanes of one column group are GROUPS apart
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int d = Ch::GROUPS; d < 64; d *= 2) {
            sg[e] += __shfl_xor(sg[e], d);
            su[e] += __shfl_xor(su[e], d);
        }
    if (lane >= Ch::GROUPS) return;
    float* out = p.parts + 2 * (int64_t)part * p.N;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (!kEdge || col + e < p.N) {
            out[col + e] = sg[e];
            out[p.N + col + e] = su[e];
        }
}

template <In T, int R, bool kEdge, bool kTail>
__global__ __launch_bounds__(NT, R == 256 ? 1 : 2) void grad_tile_kernel(GemmParams g, Grad p,
                                                                       int tiles_m, int tiles_n) {
    const TileIdx tile = xcd_tile(tiles_m, tiles_n, true);
    const int m0 = tile.bm * R, n0 = tile.bn * R;
    dma_tile<T, R, false, false, kEdge, kTail>(
        g, m0, n0, nullptr,
        [&](const auto& acc, int wm, int wn, int lane, uint8_t* mem) DGT_INLINE {
            const int row0 = m0 + wm * (R / 2), col0 = n0 + wn * (R / 2), part = 2 * tile.bm + wm;
            if (kEdge && (m0 + R > p.M || n0 + R > p.N))
                grad_epilogue<T, R, true>(p, acc, row0, col0, part, lane, mem);
            else
                grad_epilogue<T, R, false>(p, acc, row0, col0, part, lane, mem);
        });
}

bool rows_ok(const void* p, int64_t ld) { return rows_16b_aligned(p, ld, 2) && ld < kMaxBufferPitch; }

// The tile by the 16-bit kernel's wave model: rounds of the CUs, a round of 128-tiles
// (two a CU) taking 2 * 1.22 quarters of a round of 256-tiles.
bool take_128(int64_t M, int64_t N) {
    const int64_t t256 = (M + 255) / 256 * ((N + 255) / 256), t128 = (M + 127) / 128 * ((N + 127) / 128);
    const double time256 = (double)((t256 + kCUs - 1) / kCUs) * 4.0;
    const double time128 = (double)((t128 + 2 * kCUs - 1) / (2 * kCUs)) * 2.0 * 1.22;
    return time128 < time256;
}

template <In T, int R>
hipError_t forward_tiles(const Forward& p, hipStream_t s) {
    const int64_t tiles_m = ((int64_t)p.M + R - 1) / R, tiles_n = ((int64_t)p.N + R / 2 - 1) / (R / 2);
    const int64_t wgs = tiles_m * tiles_n;
    if (wgs >= (int64_t(1) << 32) / NT) return hipErrorInvalidConfiguration;
    GemmParams g = {};
    g.M = p.M; g.N = p.N; g.K = p.K;
    g.A = p.X; g.lda = p.ldx;
    g.B = p.Wg; g.ldb = p.ldwg;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)wgs), dim3(NT), 0, s, g, p, (int)tiles_m,
                           (int)tiles_n);
        return hipGetLastError();
    };
    if (p.K % (BK * NSTAGE) != 0) return go(forward_tile_kernel<T, R, true, true>);
    if (p.M % R != 0 || p.N % (R / 2) != 0) return go(forward_tile_kernel<T, R, true, false>);
    return go(forward_tile_kernel<T, R, false, false>);
}

template <In T, int R>
hipError_t grad_tiles(const Grad& p, int64_t* parts, hipStream_t s) {
    const int64_t tiles_m = ((int64_t)p.M + R - 1) / R, tiles_n = ((int64_t)p.N + R - 1) / R;
    const int64_t wgs = tiles_m * tiles_n;
    if (wgs >= (int64_t(1) << 32) / NT) return hipErrorInvalidConfiguration;
    *parts = parts_for(p.M, R);
    GemmParams g = {};
    g.M = p.M; g.N = p.N; g.K = p.K;
    g.A = p.dY; g.lda = p.lddy;
    g.B = p.Wd; g.ldb = p.ldw;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)wgs), dim3(NT), 0, s, g, p, (int)tiles_m,
                           (int)tiles_n);
        return hipGetLastError();
    };
    if (p.K % (BK * NSTAGE) != 0) return go(grad_tile_kernel<T, R, true, true>);
    if (p.M % R != 0 || p.N % R != 0) return go(grad_tile_kernel<T, R, true, false>);
    return go(grad_tile_kernel<T, R, false, false>);
}

}  // namespace

template <In T>
hipError_t launch_forward(const Forward& p, hipStream_t s) {
    if (strip_eligible(p)) return launch_forward_strip<T>(p, s);
    if (p.K == 0 || !rows_ok(p.X, p.ldx) || !rows_ok(p.Wg, p.ldwg) || !rows_ok(p.Wu, p.ldwu))
        return launch_forward_regs<T>(p, s);
    return take_128(p.M, 2 * (int64_t)p.N) ? forward_tiles<T, 128>(p, s) : forward_tiles<T, 256>(p, s);
}

template <In T>
hipError_t launch_grad(const Grad& p, int64_t* parts, hipStream_t s) {
    if (p.K == 0 || !rows_ok(p.dY, p.lddy) || !rows_ok(p.Wd, p.ldw))
        return launch_grad_regs<T>(p, parts, s);
    return take_128(p.M, p.N) ? grad_tiles<T, 128>(p, parts, s) : grad_tiles<T, 256>(p, parts, s);
}

template hipError_t launch_forward<In::BF16>(const Forward&, hipStream_t);
template hipError_t launch_forward<In::F16>(const Forward&, hipStream_t);
template hipError_t launch_grad<In::BF16>(const Grad&, int64_t*, hipStream_t);
template hipError_t launch_grad<In::F16>(const Grad&, int64_t*, hipStream_t);

}  // namespace gated
}  // namespace dgt
