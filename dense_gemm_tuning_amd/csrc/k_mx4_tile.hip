// k_mx4_tile.hip -- products of two microscaled 4-bit operands on the matrix
// cores: C <- alpha*A*B^T + beta*C + bias, both operands stored with k
// contiguous.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 with 4-bit operands takes, per lane, one
// 16-byte chunk of codes (32 consecutive k of one row: a whole block) and one
// scale byte, and multiplies blocks by 2^(sa + sb - 254) inside the sum.  A
// chunk is as many bytes as the eight 16-bit elements of a lane of the
// 32x32x16 product, and the instruction takes as long, so the kernel is the
// k-contiguous form of the 16-bit tile kernel (mfma16_tile.hpp: operands
// copied by DMA in pairs of 64-byte slices, 2 x 2 wavefronts, waits counted
// in copies) with a chunk for eight elements: four times the k per byte, and
// per second.  Its operand class is used as it is, on rows of 8*ceil(K/32)
// "elements".
//
// Scales: a group of four slices is 16 blocks, 16 scale bytes per row of
// each operand.  One copy instruction brings 64 rows of them into LDS, two
// per wave and group (one at 128 x 128), issued after the barrier of the
// group's first slice and needed at the barrier of its last; at the start of a
// group every lane reads the 16 bytes of its rows once (TM reads per
// operand) and keeps them in registers, so one LDS buffer serves.
// Step s of slice J multiplies chunks 2s + h (h the half of the wave): its
// byte is 2s + h of dword J, which a shift by 8h brings to byte 2s for every
// lane, selected by the instruction.
#include "mfma16_tile.hpp"
#include "mx4.hpp"

namespace dgt {
namespace mx4 {

namespace {

using namespace mfma16;

typedef int intx8 __attribute__((ext_vector_type(8)));

// 4-bit operands occupy the first four of the eight operand registers.
__device__ __forceinline__ intx8 widen(u32x4 x) {
    return intx8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
}

constexpr int kFp4 = 4;  // operand format code of E2M1

// One wave's copies of a group's scales: 64 rows of an operand per copy.
struct ScaleCopy {
    const uint8_t* base;
    uint32_t range, voff, at;  // at: byte offset in the LDS buffer

    // rows row0 .. row0+63 of an operand of `rows` rows; `groups` 16-byte
    // pieces per row; `lds_row`: first row's place in the buffer.
    __device__ void init(const uint8_t* S, int64_t lds, int row0, int rows, int groups, int lds_row,
                         int lane) {
        const int n = min(64, rows - row0);
        base = S + (int64_t)row0 * lds;
        range = n <= 0 ? 0u : (uint32_t)((int64_t)(n - 1) * lds + 16 * (int64_t)groups);
        voff = (uint32_t)(lane * lds);
        at = 16 * lds_row;
    }
    __device__ void copy(uint8_t* buf, int g) const {
        dma16(base, range, buf + at, voff + 16u * (uint32_t)g, 0);
    }
};

template <int R, bool kEdge, bool kTail>
__global__ __launch_bounds__(NT, R == 256 ? 1 : 2) void mx4_tile_kernel(Params p, int tiles_n,
                                                                      int nb) {
    constexpr int TM = Geo<R>::TM;
    using Op = KcOperand<R>;
    constexpr int CKC = Op::kHalfCopies;
    constexpr int SC = R == 256 ? 2 : 1;  // scale copies per wave and group
    __shared__ __attribute__((aligned(1024))) uint8_t sA0[Op::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t sA1[Op::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t sB0[Op::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t sB1[Op::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t sS[2 * R * 16];  // rows of A, then of B

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1, h = lane >> 5;
    // tile rows in order: as for the 16-bit kernel with both operands
    // k-contiguous, XCD-grouped tiles measured 3% slower (8192^3)
    const unsigned bm = blockIdx.x / (unsigned)tiles_n;
    const int m0 = (int)bm * R, n0 = (int)(blockIdx.x - bm * (unsigned)tiles_n) * R;
    const int ku = 8 * nb;                  // row length in 16-bit units
    const int nk = (ku + BK - 1) / BK;      // slices of four blocks
    const int groups = (nb + 15) / 16;

    Op opa, opb;
    opa.template init<kEdge>(static_cast<const uint16_t*>(p.A), p.lda / 2, m0, wm, wave, lane, nk,
                             p.M, ku);
    opb.template init<kEdge>(reinterpret_cast<const uint16_t*>(p.B), p.ldb / 2, n0, wn, wave, lane,
                             nk, p.N, ku);
    ScaleCopy sc[SC];
    if constexpr (R == 256) {
        sc[0].init(p.SA, p.ldsa, m0 + 64 * wave, p.M, groups, 64 * wave, lane);
        sc[1].init(p.SB, p.ldsb, n0 + 64 * wave, p.N, groups, R + 64 * wave, lane);
    } else {
        const int half = 64 * (wave & 1);
        if (wave < 2) sc[0].init(p.SA, p.ldsa, m0 + half, p.M, groups, half, lane);
        else sc[0].init(p.SB, p.ldsb, n0 + half, p.N, groups, R + half, lane);
    }

    floatx16 acc[TM][TM];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    auto frags = [&](auto Jc, int s, u32x4 (&a)[TM], u32x4 (&b)[TM]) DGT_INLINE {
        constexpr int J = decltype(Jc)::value;
        opa.frags(pick<J / 2>(sA0, sA1, sA0, sA0), J % 2, s, a);
        opb.frags(pick<J / 2>(sB0, sB1, sB0, sB0), J % 2, s, b);
    };
    // Half `half` of pair pr of an operand's slices.  When the last group is
    // cut by the row's end (kTail), the chunks at or past nb read as zeros,
    // so a row is whole groups for the loop.
    int chunk[Geo<R>::KC_INSTR];  // of the lane, in a pair's row
#pragma unroll
    for (int i = 0; i < Geo<R>::KC_INSTR; ++i)
        chunk[i] = (lane & 7) ^ swz_kc(8 * (Geo<R>::KC_INSTR * wave + i) + (lane >> 3));
    auto copy = [&](const Op& op, uint8_t* st, int pr, int half) DGT_INLINE {
        if constexpr (!kTail) {
            op.template copy<kEdge, false>(st, pr, half, wave);
        } else {
            constexpr int HALF = Geo<R>::KC_INSTR / 2;
            const int left = nb - 8 * pr;
#pragma unroll
            for (int i = HALF * half; i < HALF * half + HALF; ++i)
                dma16(op.base, op.bytes, st + (Geo<R>::KC_INSTR * wave + i) * 1024,
                      chunk[i] < left ? op.voff[i] : 0xfffffff0u, (uint32_t)pr * 128u);
        }
    };
    auto copy_scales = [&](int g) DGT_INLINE {
        g = g < groups ? g : groups - 1;  // past the end: the last group, never used
#pragma unroll
        for (int i = 0; i < SC; ++i) sc[i].copy(sS, g);
    };
    // The scales of group g for this lane's rows.  Blocks at or past nb (in
    // the last group) get the scale 1: what is stored there may be the NaN scale, and
    // their codes are zero.
    u32x4 sa[TM], sb[TM];
    const int srow_a = 16 * (wm * (R / 2) + (lane & 31));
    const int srow_b = 16 * (R + wn * (R / 2) + (lane & 31));
    auto read_scales = [&](int g) DGT_INLINE {
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            sa[t] = *reinterpret_cast<const u32x4*>(sS + srow_a + 512 * t);
            sb[t] = *reinterpret_cast<const u32x4*>(sS + srow_b + 512 * t);
        }
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                sa[t][d] >>= 8 * h;
                sb[t][d] >>= 8 * h;
            }
        if constexpr (kTail) {  // every group: a branch here costs the loop its registers
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int left = nb - (16 * g + 4 * d + h);  // blocks from byte 0 on
                const uint32_t keep = left <= 0 ? 0u : left <= 2 ? 0xffffu : 0xffffffffu;
#pragma unroll
                for (int t = 0; t < TM; ++t) {
                    sa[t][d] = (sa[t][d] & keep) | (0x7f7f7f7fu & ~keep);
                    sb[t][d] = (sb[t][d] & keep) | (0x7f7f7f7fu & ~keep);
                }
            }
        }
    };

    // The products of step kS of slice kJ on (a, b); LDS reads and copies
    // are spread between them as in the 16-bit kernel, kReads of 16 bytes per
    // four products.
    auto mfma_step = [&](auto Jc, auto Sc, auto Rc, const u32x4 (&a)[TM], const u32x4 (&b)[TM]) DGT_INLINE {
        constexpr int J = decltype(Jc)::value, kS = decltype(Sc)::value, kReads = decltype(Rc)::value;
#pragma unroll
        for (int ti = 0; ti < TM; ++ti)
#pragma unroll
            for (int tj = 0; tj < TM; ++tj)
                acc[ti][tj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    widen(a[ti]), widen(b[tj]), acc[ti][tj], kFp4, kFp4, 2 * kS, (int)sa[ti][J],
                    2 * kS, (int)sb[tj][J]);
        if constexpr (TM == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                     // MFMA
                    if (m < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // LDS read
                    if (m & 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);          // copy
                }
            }
        } else {
#pragma unroll
            for (int m = 0; m < TM * TM; ++m) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS reads
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // copy
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    u32x4 a0[TM], b0[TM], a1[TM], b1[TM];
    // Slice kt at position J of its group: the copies, waits and barrier of the
    // 16-bit kernel with both operands k-contiguous (even slices copy the second half of
    // the next pair before the barrier, odd ones the first half of the pair
    // after it behind the barrier), plus the next group's scales after the
    // barrier of slice 0: newer than what slice 1's barrier publishes, so its
    // wait lets them through; slice 2's wait covers them.
    auto slice = [&](auto Jc, int kt) DGT_INLINE {
        constexpr int J = decltype(Jc)::value;
        constexpr bool kEven = J % 2 == 0;
        using Two = std::integral_constant<int, 2>;
        frags(Jc, 1, a1, b1);
        if constexpr (kEven) {
            copy(opa, pick<(J / 2 + 1) % 2>(sA0, sA1, sA0, sA0), kt / 2 + 1, 1);
            copy(opb, pick<(J / 2 + 1) % 2>(sB0, sB1, sB0, sB0), kt / 2 + 1, 1);
        }
        mfma_step(Jc, std::integral_constant<int, 0>{}, Two{}, a0, b0);
        DMA_WAIT_VMCNT_LGKM0((copies_after<true, true, kEven>(CKC, 0) + (J == 1 ? SC : 0)));
        barrier();
        frags(std::integral_constant<int, (J + 1) % 4>{}, 0, a0, b0);
        if constexpr (J == 0) copy_scales(kt / 4 + 1);
        if constexpr (!kEven) {
            copy(opa, pick<((J + 3) / 2) % 2>(sA0, sA1, sA0, sA0), (kt + 3) / 2, 0);
            copy(opb, pick<((J + 3) / 2) % 2>(sB0, sB1, sB0, sB0), (kt + 3) / 2, 0);
        }
        mfma_step(Jc, std::integral_constant<int, 1>{}, Two{}, a1, b1);
        if constexpr (J == 3) read_scales(kt / 4 + 1);
    };

    copy_scales(0);
    copy(opa, sA0, 0, 0);
    copy(opa, sA0, 0, 1);
    copy(opb, sB0, 0, 0);
    copy(opb, sB0, 0, 1);
    copy(opa, sA1, 1, 0);
    copy(opb, sB1, 1, 0);
    DMA_WAIT_VMCNT((prologue_after<true, true>(CKC, 0)));  // slice 0 and its scales landed
    barrier();
    frags(std::integral_constant<int, 0>{}, 0, a0, b0);
    read_scales(0);
    for (int kt = 0; kt < NSTAGE * groups; kt += NSTAGE) {
        slice(std::integral_constant<int, 0>{}, kt);
        slice(std::integral_constant<int, 1>{}, kt + 1);
        slice(std::integral_constant<int, 2>{}, kt + 2);
        slice(std::integral_constant<int, 3>{}, kt + 3);
    }
    DMA_WAIT_VMCNT(0);  // no copy may still target LDS when the workgroup ends

    // Accumulator layout: register r of lane l is row 8*(r/4) + 4*(l/32) +
    // r%4, column l%32 of the MFMA tile.
    const float alpha = p.alpha, beta = p.beta;
    if constexpr (kEdge) {
        // A wave's rows of MFMA tiles through LDS, then whole rows in batches of
        // a short loop, where straight code would guard each of a lane's 64 or
        // 256 stores: 1000 x 1000 x 1000 7.0 us against 11.8, 3000^3 32 against 36,
        // 8000^3 290 against 304 (1024^3, without edges, 5.1).  Column c of row r
        // sits at c ^ 32*(r/4 & 1).
        constexpr int W = R / 2;
        dma::barrier();  // no wave still reads the stages
        float* mem = reinterpret_cast<float*>((wave < 2 ? sA0 : sA1) + (wave & 1) * (Op::kStage / 2));
        static_assert(32 * W * 4 <= Op::kStage / 2, "a wave's region holds 32 rows");
        const int row0 = m0 + wm * W, col0 = n0 + wn * W + lane;
        float bias[W / 64];
#pragma unroll
        for (int c = 0; c < W / 64; ++c)
            bias[c] = p.bias && col0 + 64 * c < p.N ? p.bias[col0 + 64 * c] : -0.0f;
#pragma unroll
        for (int ti = 0; ti < TM; ++ti) {
            asm volatile("" ::: "memory");  // LDS keeps the wave's order, so must the compiler
#pragma unroll
            for (int tj = 0; tj < TM; ++tj)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    mem[(8 * (r >> 2) + 4 * h + (r & 3)) * W + ((tj * 32 + (lane & 31)) ^ (32 * h))] =
                        acc[ti][tj][r];
            asm volatile("" ::: "memory");
            const int rows = min(32, p.M - (row0 + 32 * ti));
            float* crow = p.C + (int64_t)(row0 + 32 * ti) * p.ldc + col0;
            // Whole batches of rows without a guard but the column's; C is read
            // (beta != 0) a batch ahead of its stores: vector memory operations
            // complete in order, so a read waits for the stores before it.
            constexpr int B = 8;
            auto store_rows = [&](auto bc) DGT_INLINE {
                constexpr bool kBeta = decltype(bc)::value;
                auto put = [&](int r0, auto nc) DGT_INLINE {
                    constexpr int n = decltype(nc)::value;
#pragma unroll
                    for (int c = 0; c < W / 64; ++c) {
                        if (col0 + 64 * c >= p.N) continue;
                        float* at = crow + (int64_t)r0 * p.ldc + 64 * c;
                        float x[n], o[n];
#pragma unroll
                        for (int r = 0; r < n; ++r) {
                            const int row = r0 + r;
                            x[r] = alpha * mem[row * W + ((lane + 64 * c) ^ (32 * ((row >> 2) & 1)))];
                            o[r] = kBeta ? beta * at[(int64_t)r * p.ldc] : 0.0f;
                        }
#pragma unroll
                        for (int r = 0; r < n; ++r)
                            __builtin_nontemporal_store((kBeta ? x[r] + o[r] : x[r]) + bias[c],
                                                        &at[(int64_t)r * p.ldc]);
                    }
                };
                int r0 = 0;
                for (; r0 + B <= rows; r0 += B) put(r0, std::integral_constant<int, B>{});
                for (; r0 < rows; ++r0) put(r0, std::integral_constant<int, 1>{});
            };
            if (beta == 0.0f) store_rows(std::false_type{});
            else store_rows(std::true_type{});
        }
    } else {
        // Stores are non-temporal, and with beta != 0 C is read one MFMA tile
        // ahead of its stores, as in the 16-bit kernel.
        const int col0 = n0 + wn * (R / 2) + (lane & 31);
        float* cbase = p.C + (int64_t)(m0 + wm * (R / 2) + 4 * h) * p.ldc + col0;
        float bias[TM];
#pragma unroll
        for (int tj = 0; tj < TM; ++tj) bias[tj] = p.bias ? p.bias[col0 + tj * 32] : -0.0f;
        auto at = [&](int ti, int tj, int r) -> float* {
            return &cbase[(int64_t)(ti * 32 + 8 * (r >> 2) + (r & 3)) * p.ldc + tj * 32];
        };
        if (beta == 0.0f) {
#pragma unroll
            for (int ti = 0; ti < TM; ++ti)
#pragma unroll
                for (int tj = 0; tj < TM; ++tj)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        __builtin_nontemporal_store(alpha * acc[ti][tj][r] + bias[tj], at(ti, tj, r));
        } else {
#pragma unroll
            for (int ti = 0; ti < TM; ++ti)
#pragma unroll
                for (int tj = 0; tj < TM; ++tj) {
                    float cv[16];
#pragma unroll
                    for (int r = 0; r < 16; ++r) cv[r] = *at(ti, tj, r);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        __builtin_nontemporal_store(
                            (alpha * acc[ti][tj][r] + beta * cv[r]) + bias[tj], at(ti, tj, r));
                }
        }
    }
}

template <int R>
hipError_t launch_tiles(const Params& p, hipStream_t s) {
    const int64_t tiles_m = ((int64_t)p.M + R - 1) / R, tiles_n = ((int64_t)p.N + R - 1) / R;
    const int64_t wgs = tiles_m * tiles_n;
    const int nb = blocks(p.K);
    if (!launchable(wgs, NT)) return hipErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)wgs), dim3(NT), 0, s, p, (int)tiles_n, nb);
        return hipGetLastError();
    };
    if (nb % 16 != 0) return go(mx4_tile_kernel<R, true, true>);
    if (p.M % R != 0 || p.N % R != 0) return go(mx4_tile_kernel<R, true, false>);
    return go(mx4_tile_kernel<R, false, false>);
}

}  // namespace

// Tile size by the wave model of the 16-bit kernel.  On MX4 operands, us (128 /
// 256, the choice last): 1024^3 8.3 / 11.0 128, 2048^3 11.9 / 16.4 128, 3000^3 36.3 / 32.6 256,
// 4096^3 47.4 / 43.8 256, 6144^3 143.8 / 139.7 256, 8192^3 324 / 261 256, 1024 x 28672 x 8192
// 165 / 123 256.  With a short K the 256-tile's longer prologue and epilogue outweigh its
// loop and the model, which does not look at K, is wrong by up to a quarter: 4096 x 4096 x 512
// 15.7 / 20.5 256, 8192 x 8192 x 1024 63.3 / 77.4 256, 3000 x 3100 x 544 20.9 / 22.7 256.
hipError_t launch_product_tile(const Params& p, hipStream_t s) {
    const int64_t M = p.M, N = p.N;
    const int64_t t256 = (M + 255) / 256 * ((N + 255) / 256);
    const int64_t t128 = (M + 127) / 128 * ((N + 127) / 128);
    const double time256 = (double)((t256 + kCUs - 1) / kCUs) * 4.0;
    const double time128 = (double)((t128 + 2 * kCUs - 1) / (2 * kCUs)) * 2.0 * 1.22;
    return time128 < time256 ? launch_tiles<128>(p, s) : launch_tiles<256>(p, s);
}

}  // namespace mx4
}  // namespace dgt
