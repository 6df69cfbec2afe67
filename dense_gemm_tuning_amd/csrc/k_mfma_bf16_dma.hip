// k_mfma_bf16_dma.hip -- 16-bit-input (BF16 or FP16) / FP32-accumulate GEMM:
// global -> LDS by DMA up to three K slices ahead, operands stored with m / n
// contiguous transposed by the LDS read.
//
// Tiling as in the register-staged kernel (256 x 256 workgroup tile, 2 x 2
// wavefronts of 128 x 128, v_mfma_f32_32x32x16: dilfish.github.io 5.3-5.5,
// qwbw.cn Level 2), or, for launches with few such tiles, 128 x 128 (two
// workgroups per CU, wavefronts of 64 x 64), with a deeper software
// pipeline than the pages' double buffer (dilfish.github.io 5.4; qwbw.cn's
// double-buffering row).  The notes below give the 256 x 256 sizes; at 128
// a stage holds half the rows or columns and each wave half the copies:
//
//  * K advances in slices of 32.  Copies use buffer_load_dwordx4 ... lds:
//    lane l's 16 bytes land at LDS base + 16*l, so one instruction fills
//    1 KiB and no operand byte passes through a VGPR; a swizzle is applied by
//    the choice of which global chunk each lane fetches.  Each wave addresses
//    its rows through a buffer descriptor (wave-uniform base, 32-bit lane
//    offsets, range-checked by the hardware); against the same copies as
//    global_load_lds the L2 requests return sooner and the kernel is ~2%
//    faster.
//  * An operand is staged by how it is stored, not by whether it is A or B.
//    K-contiguous (A as M x K, B transposed as N x K): two LDS stages of two
//    slices each, 256 rows of 128 B (chunk q of row r at q ^ ((r ^ r>>3) & 7)),
//    so each copy request covers a 128-byte row segment; a lane reads its 8
//    consecutive k with one 16-byte LDS read.  MN-contiguous (B as K x N, A
//    transposed as K x M): four stages of one slice, 32 k-rows of 512 B
//    (chunk c of row k at c ^ (4*(k & 3))); ds_read_b64_tr_b16 transposes
//    on the read: within each 16-lane group, source lane 4r+q names row r,
//    columns 4q..4q+3, and destination lane j receives column j, rows 0..3;
//    two reads give a lane its 8 consecutive k (the pages warn that an
//    operand in the wrong major order still "looks right": dilfish.github.io
//    5.5).  Either way 64 KiB per operand, 128 KiB of the 160 KiB LDS.
//  * Copies start as soon as a stage is retired, 1.25 to 2.5 slices (1200 to
//    2500 MFMA cycles) before the data is needed, which covers L2-miss
//    latency to the memory side.  Each wave's copies are spread one per two
//    MFMAs; issued in bursts they queue at the address unit and in L1 and
//    hold back the wave's MFMA issue.  Copies past the last slice re-read the last
//    slice (never consumed) so every step waits on the same count.
//  * Per slice each wavefront issues 32 MFMAs in two 16-deep steps; the LDS
//    reads of the next step are interleaved with them.  The workgroup
//    barrier sits between the two steps: it publishes slice t+1 (every wave
//    has waited for its own copies) and retires slice t's stage, so the
//    first operands of slice t+1 are read while step 2 of slice t computes.
//
// Used for any M, N and K with 16-byte aligned rows and row pitches below
// 2^24 elements (so that a wave's rows of lane offsets fit 32 bits).  On edge
// tiles the copy descriptors' ranges stop at the operands' last elements and
// the epilogue stores only the valid part.  When K is not a multiple of 128
// the K loop runs in groups of four 32-deep slices and the last group (1 to
// 4 slices) after it as ordinary slices (each keeps its copies, waits and
// barrier, so every wait count holds); in a partial last slice the
// k-contiguous fragments are masked past K, and m/n-contiguous rows past K
// read as zeros through the descriptor range.  The register-staged kernel
// handles unaligned operands.
#include "mfma16_tile.hpp"
#include "streamk.hpp"

namespace dgt {

namespace {

using namespace mfma16;

constexpr double kCost128 = 1.22;           // a 128-tile's time, in quarters of a 256-tile's

template <In T, int R, bool TA, bool TB, bool kEdge, bool kTail>
__global__ __launch_bounds__(NT, R == 256 ? 1 : 2) void mfma16_dma_kernel(GemmParams p,
                                                                        int tiles_m,
                                                                        int tiles_n,
                                                                        int grouped) {
    const TileIdx tile = xcd_tile(tiles_m, tiles_n, grouped != 0);
    select_problem(p, tile.z);
    dma_tile<T, R, TA, TB, kEdge, kTail>(p, tile.bm * R, tile.bn * R, nullptr);
}


// ------------------------------------------------------------- stream-K
// (the schedule and the fix-up kernel: streamk.hpp)

constexpr int kSkIterK = streamk::kIterK16;
static_assert(kSkIterK == BK * NSTAGE, "a stream-K iteration is one group of four slices");

template <In T, bool TA, bool TB, bool kRagged>
__global__ __launch_bounds__(NT, 1) void mfma16_streamk_kernel(GemmParams p, streamk::StreamK sk,
                                                               float* ws) {
    streamk::walk<TA, TB, 2>(p, sk, ws, [&](const GemmParams& q, int m0, int n0, float* raw) {
        dma_tile<T, streamk::R, TA, TB, kRagged, kRagged>(q, m0, n0, raw);
    });
}

}  // namespace

int64_t streamk_workspace_bytes(const GemmParams& p, bool f32) {
    return streamk::workspace_bytes(p, f32 ? streamk::kIterKF32 : streamk::kIterK16);
}

template <In T>
hipError_t launch_mfma16_streamk(const GemmParams& p, float* ws, hipStream_t s) {
    if (p.batch != 1 || p.k_last > 0 || !mfma16_dma_eligible(p)) return hipErrorInvalidConfiguration;
    const streamk::StreamK sk = streamk::plan(p, kSkIterK);
    if (sk.T > 0x7fffffff) return hipErrorInvalidConfiguration;
    const bool ragged = p.M % 256 != 0 || p.N % 256 != 0 || p.K % kSkIterK != 0;
    hipError_t e = with_layout(p, [&](auto ta, auto tb) {
        constexpr bool TA = decltype(ta)::value, TB = decltype(tb)::value;
        if (ragged)
            hipLaunchKernelGGL((mfma16_streamk_kernel<T, TA, TB, true>), dim3(sk.G), dim3(NT), 0,
                               s, p, sk, ws);
        else
            hipLaunchKernelGGL((mfma16_streamk_kernel<T, TA, TB, false>), dim3(sk.G), dim3(NT), 0,
                               s, p, sk, ws);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    return streamk::launch_fixup(p, sk, ws, s);
}
template hipError_t launch_mfma16_streamk<In::BF16>(const GemmParams&, float*, hipStream_t);
template hipError_t launch_mfma16_streamk<In::F16>(const GemmParams&, float*, hipStream_t);

// Any M, N and K (edge tiles and a K tail are clipped or masked), 16-byte
// aligned rows, and pitches within the 32-bit buffer offsets.
bool mfma16_dma_eligible(const GemmParams& p) {
    return operands_16b_aligned(p, 2) && p.M > 0 && p.N > 0 && p.K > 0 &&
           p.lda < kMaxBufferPitch && p.ldb < kMaxBufferPitch;
}

namespace {

template <In T, int R>
hipError_t launch_tiles(const GemmParams& p, hipStream_t s) {
    const int tiles_m = (p.M + R - 1) / R, tiles_n = (p.N + R - 1) / R;
    const int64_t blocks = (int64_t)tiles_m * tiles_n;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    const bool edge = p.M % R != 0 || p.N % R != 0;
    const bool tail = !k_multiple(p, BK * NSTAGE);
    return with_layout(p, [&](auto ta, auto tb) {
        constexpr bool TA = decltype(ta)::value, TB = decltype(tb)::value;
        // linear order only for one problem with both operands k-contiguous
        const int grouped = !(p.batch == 1 && !TA && TB);
        const dim3 grid((unsigned)blocks, p.batch);
        auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, dim3(NT), 0, s, p, tiles_m, tiles_n, grouped);
        };
        // a K tail takes the edge-tile instance whatever M and N (its guards
        // then always pass); built without edges it spills registers
        if (tail) go(mfma16_dma_kernel<T, R, TA, TB, true, true>);
        else if (edge) go(mfma16_dma_kernel<T, R, TA, TB, true, false>);
        else go(mfma16_dma_kernel<T, R, TA, TB, false, false>);
        return hipGetLastError();
    });
}

}  // namespace

template <In T>
hipError_t launch_mfma16_dma_tile(const GemmParams& p, hipStream_t s, int tile) {
    return tile == 128 ? launch_tiles<T, 128>(p, s) : launch_tiles<T, 256>(p, s);
}

// Tile size by the waves of tiles the CUs work through.  A CU runs one
// 256-tile, or two 128-tiles side by side (alone, a 128-tile leaves the CU
// about as slow as a pair does), and a 128-tile costs kCost128 quarters of a
// 256-tile's time (measured at 8192^3: 0.932 against 0.766 ms).  In units
// of a quarter 256-tile: 4 per wave of 256 tiles against 2 * kCost128 per
// wave of 512.  Ties keep the larger tile.
template <In T>
hipError_t launch_mfma16_dma(const GemmParams& p, hipStream_t s) {
    const int64_t t256 = (int64_t)((p.M + 255) / 256) * ((p.N + 255) / 256) * p.batch;
    const int64_t t128 = (int64_t)((p.M + 127) / 128) * ((p.N + 127) / 128) * p.batch;
    const double time256 = (double)((t256 + kCUs - 1) / kCUs) * 4.0;
    const double time128 = (double)((t128 + 2 * kCUs - 1) / (2 * kCUs)) * 2.0 * kCost128;
    return time128 < time256 ? launch_tiles<T, 128>(p, s) : launch_tiles<T, 256>(p, s);
}
template hipError_t launch_mfma16_dma<In::BF16>(const GemmParams&, hipStream_t);
template hipError_t launch_mfma16_dma<In::F16>(const GemmParams&, hipStream_t);
template hipError_t launch_mfma16_dma_tile<In::BF16>(const GemmParams&, hipStream_t, int);
template hipError_t launch_mfma16_dma_tile<In::F16>(const GemmParams&, hipStream_t, int);

}  // namespace dgt
