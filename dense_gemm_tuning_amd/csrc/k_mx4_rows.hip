// k_mx4_rows.hip -- decode batches against a microscaled 4-bit weight stored
// N x K, for weights with enough columns to give every compute unit a strip.
//
// Streaming B once (17 bytes per 32 weights) is the floor.  A workgroup shares
// both operands of a strip of up to COLS stored rows of B and up to 16*RBT rows
// of A: a step of K (ROWB bytes of codes per row) of both, with the scales, is copied into one
// of NS LDS stages, NS - 1 steps ahead, and one barrier per step both
// publishes the step and retires the stage before it.  Every operand byte is
// read from memory once per workgroup, by copies that write LDS.
//
// The 8 waves split the step's K KS ways and the strip's columns 8/KS ways,
// each wave all rows of A: the LDS bytes a step reads are then A times 8/KS
// plus B once, where waves side by side in the output would read A (16-bit:
// twice B's bytes at 64 rows) once for every column part and convert B for every row
// part.  The KS partial tiles are summed in LDS in a fixed order at the end.
//
// Chunk c of a row sits at c ^ swz(row) in LDS (16 rows reading one chunk
// touch 16 distinct 16-byte bank groups); the copies choose which chunk each
// lane fetches.  Lane (i, g) = (lane % 16, lane / 16) of a 16-column block:
//  * MX4 A: one 16x16x128 scaled product per 4 blocks; group g holds block g.
//  * 16-bit A: one 16x16x32 product per block, 8 k (a dword of codes) per
//    group.  BF16: the codes are converted to BF16 with their scale (exact:
//    4 bits times a power of two).  FP16: converted unscaled, and the product is
//    scaled as it is added.
//
// Workgroups start at different steps and wrap around: all at one k, they
// would ask for the same columns of rows whose pitch is often a power of two,
// and so for the same memory channels (28672 x 8192 weights, MX4, M = 8: 28.5 us
// without, 23.8 with; with B's copies non-temporal 22.0, 5.7 TB/s).
//
// 16-bit A needs 16-byte aligned rows and a pitch below 2^24 elements; other
// A takes the wave-private kernel (k_mx4_skinny.hip).
#include "dma_common.hpp"
#include "mx4_device.hpp"

namespace dgt {
namespace mx4 {

namespace {

constexpr int NWAVE = 8;

template <Kind KA, int RBT, int COLS_, int KS, int ROWB>
struct Tile {
    static constexpr int COLS = COLS_;
    static constexpr int STEPB = ROWB / 16;               // blocks per step
    static constexpr int BPW = STEPB / KS;                // ... of them a wave's
    static constexpr int CBW = COLS * KS / NWAVE / 16;    // 16-column blocks per wave
    static constexpr int PA = KA == Kind::MX4 ? 1 : 4;    // 16-byte pieces of A per block
    static constexpr int AROW = ROWB * PA;                // bytes of a row of A per step
    static constexpr int B_BYTES = COLS * ROWB;           // a stage: codes of B,
    static constexpr int A_BYTES = 16 * RBT * AROW;       // A,
    static constexpr int SROWS = COLS + (KA == Kind::MX4 ? 64 : 0);
    static constexpr int S_BYTES = SROWS * STEPB;         // and scales, B's rows then A's
    static constexpr int STAGE = B_BYTES + A_BYTES + S_BYTES;
    // Copies per step: IB of B per wave; NA of A and NSC of scales dealt out
    // over the waves.
    static constexpr int SLANE = KA == Kind::MX4 ? 16 : 4;   // bytes per lane of a scale copy
    static constexpr int IB = B_BYTES / 1024 / NWAVE, NA = A_BYTES / 1024;
    static constexpr int NSC = S_BYTES / (64 * SLANE), NX = NA + NSC;
    static constexpr int IX = (NX + NWAVE - 1) / NWAVE;      // most of a wave
    static constexpr int XREST = NX % NWAVE == 0 ? NWAVE : NX % NWAVE;  // waves with IX of them
    static_assert(B_BYTES % (1024 * NWAVE) == 0 && A_BYTES % 1024 == 0 && COLS * STEPB % (64 * SLANE) == 0 &&
                      S_BYTES % (64 * SLANE) == 0,
                  "whole copies, each of one operand");
    static_assert(KA != Kind::MX4 || BPW == 4, "a wave's blocks are one scaled product");
    __device__ static int swz_b(int r) { return ROWB == 256 ? (r & 15) : ((r >> 1) & 7); }
    __device__ static int swz_a(int r) { return AROW >= 256 ? (r & 15) : ((r >> 1) & 7); }
};

// One piece of kBytes per lane into LDS (lane l's bytes at lds + kBytes*l).
template <int kBytes, int kPolicy>
__device__ __forceinline__ void copy_piece(const void* base, uint32_t range, uint8_t* lds,
                                           uint32_t voff) {
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, range, kBufferRsrcW3);
    if constexpr (kBytes == 16)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (dma::lds_void*)lds, 16, voff, 0, 0, kPolicy);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (dma::lds_void*)lds, 4, voff, 0, 0, kPolicy);
}

template <Kind KA, int RBT, int COLS, int KS, int ROWB, int NS>
__global__ __launch_bounds__(NWAVE * 64, 1) void mx4_rows_kernel(Params p, int cols, int nb,
                                                                 int mchunks) {
    using G = Tile<KA, RBT, COLS, KS, ROWB>;
    constexpr int PA = G::PA, CBW = G::CBW, BPW = G::BPW;
    static_assert(NS == 3 || NS == 4, "ring sizes");
    // One object per stage, so that the compiler's wait-count pass can tell a
    // copy into one from reads of another.
    __shared__ __attribute__((aligned(1024))) uint8_t st0[G::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[G::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t st2[G::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t st3[NS > 3 ? G::STAGE : 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, i = lane & 15;
    const int wk = wave % KS, wc = wave / KS;
    // the row chunks of one strip on one XCD, as in k_mx4_skinny.hip
    const int q8 = blockIdx.x / (8 * mchunks), r8 = blockIdx.x % (8 * mchunks);
    const int n0 = (8 * q8 + r8 % 8) * cols;
    const int mbase = (r8 / 8) * 16 * RBT;
    if (n0 >= p.N) return;
    const int nlim = min(n0 + cols, p.N);
    const int rowsA = min(16 * RBT, p.M - mbase);
    const int nsteps = (nb + G::STEPB - 1) / G::STEPB;
    const int first = (int)((unsigned)q8 % (unsigned)nsteps);
    auto at = [&](int s) DGT_INLINE { return s + first < nsteps ? s + first : s + first - nsteps; };

    // One descriptor per operand, ending with the last valid row (rows past
    // it read as zeros).  A's 16-bit rows end on a whole 16-byte piece.
    const int64_t rowbytes = (int64_t)kChunk * nb;
    const int64_t pitch_a = KA == Kind::MX4 ? p.lda : 2 * p.lda;
    const int pieces_a = KA == Kind::MX4 ? nb : (p.K + 7) / 8;  // 16-byte pieces of a row of A
    const uint8_t* base_b = p.B + (int64_t)n0 * p.ldb;
    const uint32_t range_b = (uint32_t)((int64_t)(nlim - 1 - n0) * p.ldb + rowbytes);
    const uint8_t* base_a = static_cast<const uint8_t*>(p.A) + (int64_t)mbase * pitch_a;
    const uint32_t range_a = (uint32_t)((int64_t)(rowsA - 1) * pitch_a + 16 * (int64_t)pieces_a);
    // This wave's copies: IB of B, then every eighth of A's and the scales'
    // (a copy costs the CU about the same whatever it fetches, so none is
    // repeated to even out the waves).  All are one piece per lane at
    // base + voff + step, if the piece lies inside the row.
    uint32_t voff_b[G::IB], voff_x[G::IX];
    int cb[G::IB], cx[G::IX];  // the lane's piece within the step
    const uint8_t* base_x[G::IX];
    uint32_t range_x[G::IX];
#pragma unroll
    for (int j = 0; j < G::IB; ++j) {
        constexpr int L = ROWB / 16;  // lanes per row
        const int row = (64 / L) * (G::IB * wave + j) + lane / L;
        cb[j] = (lane % L) ^ G::swz_b(row);
        voff_b[j] = (uint32_t)(row * p.ldb + 16 * cb[j]);
    }
    const uint32_t sprow = (uint32_t)(16 * ((nb + 15) / 16));
    // whether the wave's j-th of these is A's (known at compile time but for
    // a j that has some of each)
    auto is_a = [&](auto jc) DGT_INLINE {
        constexpr int x0 = NWAVE * decltype(jc)::value;
        if constexpr (x0 + NWAVE <= G::NA) return true;
        else if constexpr (x0 >= G::NA) return false;
        else return x0 + wave < G::NA;
    };
    static_for<G::IX>([&](auto jc) DGT_INLINE {
        constexpr int j = decltype(jc)::value;
        const int x = NWAVE * j + wave;
        if (is_a(jc)) {
            constexpr int L = G::AROW / 16;
            const int row = (64 / L) * x + lane / L;
            cx[j] = (lane % L) ^ G::swz_a(row);
            voff_x[j] = (uint32_t)(row * pitch_a + 16 * cx[j]);
            base_x[j] = base_a;
            range_x[j] = range_a;
        } else {  // 64 * SLANE / STEPB rows of scales: of B, from COLS on of A
            constexpr int L = G::STEPB / G::SLANE;
            const int srow = (64 / L) * (x - G::NA);
            const bool of_a = KA == Kind::MX4 && srow >= COLS;
            const int64_t pitch = of_a ? p.ldsa : p.ldsb;
            cx[j] = 0;
            voff_x[j] = (uint32_t)((srow - (of_a ? COLS : 0) + lane / L) * pitch + G::SLANE * (lane % L));
            base_x[j] = of_a ? p.SA + (int64_t)mbase * p.ldsa : p.SB + (int64_t)n0 * p.ldsb;
            range_x[j] = (uint32_t)((int64_t)((of_a ? rowsA : nlim - n0) - 1) * pitch + sprow);
        }
    });

    floatx4 acc[RBT][CBW];
#pragma unroll
    for (int rb = 0; rb < RBT; ++rb)
#pragma unroll
        for (int c = 0; c < CBW; ++c) acc[rb][c] = floatx4{0.f, 0.f, 0.f, 0.f};

    auto copy_step = [&](auto qc, int t) DGT_INLINE {
        uint8_t* st = dma::pick<decltype(qc)::value>(st0, st1, st2, st3);
        const int s = at(min(t, nsteps - 1));
        const int lim_b = t < nsteps ? nb - G::STEPB * s : 0;  // pieces left in a row
        const int lim_a = t < nsteps ? pieces_a - G::STEPB * PA * s : 0;
#pragma unroll
        for (int j = 0; j < G::IB; ++j)
            copy_piece<16, 2>(base_b, range_b, st + 1024 * (G::IB * wave + j),
                              cb[j] < lim_b ? voff_b[j] + (uint32_t)(ROWB * s) : 0xfffffff0u);
        static_for<G::IX>([&](auto jc) DGT_INLINE {
            constexpr int j = decltype(jc)::value;
            const int x = NWAVE * j + wave;
            if (is_a(jc))
                copy_piece<16, 1>(base_x[j], range_x[j], st + G::B_BYTES + 1024 * x,
                                  cx[j] < lim_a ? voff_x[j] + (uint32_t)(G::AROW * s) : 0xfffffff0u);
            else if (x < G::NX)
                copy_piece<G::SLANE, 1>(base_x[j], range_x[j],
                                        st + G::B_BYTES + G::A_BYTES + 64 * G::SLANE * (x - G::NA),
                                        voff_x[j] + (uint32_t)(G::STEPB * s));
        });
    };

    // The wave's part of step s, in stage st; kCut: the row ends inside the step.
    auto compute = [&](const uint8_t* st, auto cutc, int s) DGT_INLINE {
        constexpr bool kCut = decltype(cutc)::value;
        const uint8_t* sa_ = st + G::B_BYTES;
        const uint8_t* scales = sa_ + G::A_BYTES;
        const int b0 = G::STEPB * s + BPW * wk;  // the wave's first block
        if constexpr (KA == Kind::MX4) {
            const int chunk = 4 * wk + g;
            const bool past = kCut && b0 + g >= nb;  // its codes are zero
            u32x4 a[RBT], w[CBW];
            uint32_t sa[RBT], sb[CBW];
#pragma unroll
            for (int rb = 0; rb < RBT; ++rb) {
                const int row = 16 * rb + i;
                a[rb] = *reinterpret_cast<const u32x4*>(sa_ + row * G::AROW +
                                                        ((chunk ^ G::swz_a(row)) << 4));
                sa[rb] = past ? 127u : scales[(COLS + row) * G::STEPB + chunk];
            }
#pragma unroll
            for (int c = 0; c < CBW; ++c) {
                const int row = 16 * (CBW * wc + c) + i;
                w[c] = *reinterpret_cast<const u32x4*>(st + row * ROWB +
                                                       ((chunk ^ G::swz_b(row)) << 4));
                sb[c] = past ? 127u : scales[row * G::STEPB + chunk];
            }
#pragma unroll
            for (int c = 0; c < CBW; ++c)
#pragma unroll
                for (int rb = 0; rb < RBT; ++rb)
                    acc[rb][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        widen(a[rb]), widen(w[c]), acc[rb][c], 4, 4, 0, (int)sa[rb], 0, (int)sb[c]);
        } else {
#pragma unroll
            for (int e = 0; e < BPW; ++e) {
                const int blk = BPW * wk + e;
                u32x4 a[RBT];
#pragma unroll
                for (int rb = 0; rb < RBT; ++rb) {
                    const int row = 16 * rb + i;
                    a[rb] = *reinterpret_cast<const u32x4*>(
                        sa_ + row * G::AROW + (((4 * blk + g) ^ G::swz_a(row)) << 4));
                }
                if constexpr (kCut) {  // what follows k = K - 1 in A's rows may be anything
                    const int left = p.K - (kBlock * (b0 + e) + 8 * g);
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const uint32_t keep = (2 * d < left ? 0x0000ffffu : 0u) |
                                              (2 * d + 1 < left ? 0xffff0000u : 0u);
#pragma unroll
                        for (int rb = 0; rb < RBT; ++rb) a[rb][d] &= keep;
                    }
                }
#pragma unroll
                for (int c = 0; c < CBW; ++c) {
                    const int row = 16 * (CBW * wc + c) + i;
                    const uint32_t q = *reinterpret_cast<const uint32_t*>(
                        st + row * ROWB + ((blk ^ G::swz_b(row)) << 4) + 4 * g);
                    const uint32_t sb = kCut && b0 + e >= nb ? 127u : scales[row * G::STEPB + blk];
                    if constexpr (KA == Kind::F16) {
                        const u32x4 v = decode8_f16(q);
                        const float f = scale_number(sb, 0);
#pragma unroll
                        for (int rb = 0; rb < RBT; ++rb)
                            acc[rb][c] = scaled_product_f16(a[rb], v, f, acc[rb][c]);
                    } else {
                        const u32x4 v = decode8(q, scale_bits(sb));
#pragma unroll
                        for (int rb = 0; rb < RBT; ++rb)
                            acc[rb][c] = mfma16x16x32<In::BF16>(a[rb], v, acc[rb][c]);
                    }
                }
            }
        }
    };
    auto fence = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // Step s in stage Q.  At the wait the wave's copies of steps s+1 .. s+NS-2
    // are newer than this step's.
    constexpr int kMost = G::IB + G::IX;
    auto step = [&](auto qc, int s) DGT_INLINE {
        constexpr int Q = decltype(qc)::value;
        const int k = at(s);
        if (wave < G::XREST) {
            DMA_WAIT_VMCNT_LGKM0(((NS - 2) * kMost));
        } else {
            DMA_WAIT_VMCNT_LGKM0(((NS - 2) * (kMost - 1)));
        }
        dma::barrier();  // step s is in LDS for every wave; step s-1's stage is free
        copy_step(std::integral_constant<int, (Q + NS - 1) % NS>{}, s + NS - 1);
        fence();
        // one branch for the whole step
        const uint8_t* st = dma::pick<Q>(st0, st1, st2, st3);
        if (kBlock * G::STEPB * (k + 1) > p.K) compute(st, std::true_type{}, k);
        else compute(st, std::false_type{}, k);
    };
    static_for<NS - 1>([&](auto qc) DGT_INLINE { copy_step(qc, decltype(qc)::value); });
    fence();
    for (int s = 0; s < nsteps; s += NS) {  // stages are compile-time
        static_for<NS>([&](auto jc) DGT_INLINE {
            constexpr int j = decltype(jc)::value;
            if (s + j < nsteps) step(jc, s + j);
        });
    }
    DMA_WAIT_VMCNT_LGKM0(0);  // no copy may still target LDS: the stages are reused

    // The KS partial tiles, summed RR rows at a time in stages 0 and 1 in
    // turn (one barrier per pass: a buffer is written again two passes later).
    // 16x16 accumulator layout: register r of lane (i, g) is row 4g + r,
    // column i.
    constexpr int kFit = G::STAGE / (KS * COLS * 4);
    constexpr int RR = kFit >= 16 ? 16 : kFit >= 8 ? 8 : 4;
    static_assert(RR * KS * COLS * 4 <= G::STAGE, "a pass fits a stage");
    dma::barrier();
    static_for<RBT * 16 / RR>([&](auto pc) DGT_INLINE {
        constexpr int pass = decltype(pc)::value, rb = pass * RR / 16, r0 = pass * RR % 16;
        float* red = reinterpret_cast<float*>(dma::pick<pass % 2>(st0, st1, st0, st0));
        if (4 * g >= r0 && 4 * g < r0 + RR) {
#pragma unroll
            for (int c = 0; c < CBW; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    red[(RR * wk + 4 * g + r - r0) * COLS + ((16 * (CBW * wc + c) + i) ^ (16 * g))] =
                        acc[rb][c][r];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < RR * COLS; e += NWAVE * 64) {
            const int row = r0 + e / COLS, col = e % COLS;
            const int m = 16 * rb + row, n = n0 + col;
            if (m >= rowsA || n >= nlim) continue;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < KS; ++w)
                sum += red[(RR * w + row - r0) * COLS + (col ^ (16 * (row >> 2)))];
            float* cptr = p.C + (int64_t)(mbase + m) * p.ldc + n;
            *cptr = epilogue(sum, p, cptr, n);
        }
    });
}

template <Kind KA, int RBT, int COLS, int KS, int ROWB, int NS>
hipError_t launch_strips(const Params& p, int cols, hipStream_t s) {
    const int mchunks = (int)(((int64_t)p.M + 16 * RBT - 1) / (16 * RBT));
    const int64_t strips = ((int64_t)p.N + cols - 1) / cols;
    const int64_t wgs = (strips + 7) / 8 * 8 * mchunks;
    if (!launchable(wgs, NWAVE * 64)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((mx4_rows_kernel<KA, RBT, COLS, KS, ROWB, NS>), dim3((unsigned)wgs),
                       dim3(NWAVE * 64), 0, s, p, cols, blocks(p.K), mchunks);
    return hipGetLastError();
}

// Strips of up to 64 columns while those take one round of the CUs, else of
// up to 128, as narrow as their number of rounds allows (28672 x 8192, MX4,
// M = 8: 21.4 us in 256 strips of 112, 26.9 in 448 of 64; 14336 x 8192: 14.3 in 224 of 64).
template <Kind KA, int RBT, int NS64, int NS128>
hipError_t launch_width(const Params& p, hipStream_t s) {
    constexpr int KS = 4, ROWB = KA == Kind::MX4 ? 256 : 128;
    const int64_t chunks = ((int64_t)p.M + 16 * RBT - 1) / (16 * RBT);
    auto strips = [&](int c) { return ((int64_t)p.N + c - 1) / c * chunks; };
    // (FP16 at 64 rows: 128 columns do not fit the registers)
    if (strips(64) <= dma::kCUs || (KA == Kind::F16 && RBT == 4))
        return launch_strips<KA, RBT, 64, KS, ROWB, NS64>(p, 64, s);
    const int64_t rounds = (strips(128) + dma::kCUs - 1) / dma::kCUs;
    int cols = 128;
    while (cols > 80 && strips(cols - 16) <= rounds * dma::kCUs) cols -= 16;
    return launch_strips<KA, RBT, (KA == Kind::F16 && RBT == 4) ? 64 : 128, KS, ROWB, NS128>(
        p, cols, s);
}

// 16-bit rows that the copies take.
bool rows_copyable(const Params& p) {
    return rows_16b_aligned(p.A, p.lda, 2) && p.lda < kMaxBufferPitch;
}

// Workgroups of a launch in strips of `cols` columns and rb blocks of 16 rows,
// and whether the CUs take them in one round.
bool one_round(const Params& p, int cols, int rb) {
    return ((int64_t)p.N + cols - 1) / cols * (((int64_t)p.M + 16 * rb - 1) / (16 * rb)) <= dma::kCUs;
}

}  // namespace

// Few outputs leave only K to share: the form with the smallest workgroups
// (16 rows x 16, then 32 columns, wave-private) whose launch is one round of
// the CUs has the shortest way through K; then 32 x 32, and one round of this
// kernel, where K is long or M small.  Else tiles above 64 rows.  us (16 x 16 / 16 x 32
// / 32 x 32 wave-private, this kernel, tiles), weights in L2:
//   K = 8192: M = 32   N = 2048   6.8   8.3  11.8        14.7
//                      N = 8192  22.7  17.3  13.3  16.3  21.3
//             M = 128  N = 1024  11.4   8.1  11.5  12.2  14.5
//                      N = 2048  20.5  15.1  11.6  12.4  14.6
//                      N = 4096  40.7  30.6  23.8  12.9  14.7
//                      N = 8192  79.8  60.5  46.7  15.9  21.9
//   K = 1024: M = 128  N = 1024   4.3   4.4   4.3   5.5   4.6
//                      N = 4096  10.1   9.5   7.6   5.6   4.7
// and from memory M = 8, K = 8192: N = 3584 7.3 (16 x 16) / 12.4 (this), 8192 10.9
// (16 x 32) / 12.8, 14336 18.7 / 14.3.
hipError_t launch_product(const Params& p, hipStream_t s) {
    if (one_round(p, 16, 1)) return launch_skinny(p, 1, 16, s);
    if (one_round(p, 32, 1)) return launch_skinny(p, 1, 32, s);
    const bool long_k = p.K >= 4096;
    if (p.M > 16 && (p.M <= 64 || long_k) && one_round(p, 32, 2)) return launch_skinny(p, 2, 32, s);
    if (p.M <= 16) return launch_width<Kind::MX4, 1, 4, 3>(p, s);
    if (p.M <= 32) return launch_width<Kind::MX4, 2, 4, 3>(p, s);
    if (p.M <= 64 || (long_k && one_round(p, 64, 4))) return launch_width<Kind::MX4, 4, 4, 3>(p, s);
    return launch_product_tile(p, s);
}

// The same for 16-bit A, up to 512 rows (a strip's A comes from L2 only while other
// strips read it too).  us at K = 8192, weights in L2 (wave-private / this):
//   BF16  M = 32:  N = 1024 13.6 / 18.7, 4096 16.9 / 19.7
//         M = 64:  14.3 / 26.5, 19.8 / 26.6;  M = 256: N = 1024 20.2 / 29.0
//         M = 1024: N = 256 41.5 / 29.9
//   FP16  M = 32:  12.6 / 23.0, 15.9 / 23.1;  M = 64: 12.8 / 32.6, 24.7 / 33.7
// and from memory, M = 8: BF16 N = 14336 20.0 / 23.0, 28672 37.9 / 30.8; FP16
// 14336 27.0 / 33.2.
hipError_t launch_product16(In t, const Params& p, hipStream_t s) {
    for (int cols = 16; cols <= 64 && p.M <= 512; cols *= 2)
        if (one_round(p, cols, 1)) return launch_skinny16(t, p, 1, cols, s);
    if (!rows_copyable(p)) return launch_skinny16(t, p, t == In::BF16 && p.M > 16 ? 2 : 1, 64, s);
    if (t == In::F16)
        return p.M <= 16   ? launch_width<Kind::F16, 1, 4, 4>(p, s)
               : p.M <= 32 ? launch_width<Kind::F16, 2, 4, 4>(p, s)
                           : launch_width<Kind::F16, 4, 3, 3>(p, s);
    return p.M <= 16   ? launch_width<Kind::BF16, 1, 4, 4>(p, s)
           : p.M <= 32 ? launch_width<Kind::BF16, 2, 4, 4>(p, s)
                       : launch_width<Kind::BF16, 4, 3, 3>(p, s);
}

}  // namespace mx4
}  // namespace dgt
