// k_mx4_skinny.hip -- products of few outputs with a microscaled 4-bit weight
// (decode batches against a share of a layer, short batches against narrow
// weights): A (MX4, BF16 or FP16, k contiguous) against B stored N x K.  The
// time is the latency of one pass through K (and, of a weight that comes from
// memory, of its 17 bytes per 32 elements): narrow strips, few rows, K split over the
// waves.  Wide weights and larger batches take k_mx4_rows.hip, where the choice
// is made, or tiles.
//
// Each wave copies its pieces of B straight into a private LDS ring by
// buffer loads that write LDS (no workgroup barrier in the loop; the scheme of
// k_skinny_dma.hip): a step is ROWB bytes (ROWB/16 blocks) of each stored row
// of the strip, in NG groups of GR rows, copied NS - 1 groups ahead.
// The strip's K range is split over the NW waves and the partial tiles are summed
// in LDS in wave order (deterministic, no atomics, no workspace).
//
// Lane (i, g) = (lane % 16, lane / 16) of a 16-column block takes row i's
// U = ROWB/64 chunks U*g .. U*g + U-1 of the step, so that the U scale
// bytes it needs are adjacent: one load per row block and step, the product
// picks its byte.  A is loaded the same way (any order of k serves as long
// as both operands use it).
//
//  * MX4 A: one 16x16x128 scaled product per chunk pair.
//  * BF16 A: the chunk's 32 values are converted to BF16 with their scale (exact:
//    4 bits times a power of two) and meet four 16-byte pieces of A in four
//    16x16x32 products.
//  * FP16 A: the scales' range does not fit FP16, so the codes are converted
//    unscaled and each block's product is scaled as it is added. For that the four
//    lane groups take the same block, 8 k each (a dword of its codes), and a
//    row's scale bytes of the whole step are loaded.
#include "dma_common.hpp"
#include "mx4_device.hpp"
#include "skinny_common.hpp"

namespace dgt {
namespace mx4 {

namespace {

using skinny::u32x4_any;

constexpr int NW = 8;       // waves per workgroup
constexpr int kBPolicy = 2; // cache policy of the B copies: nt (streamed once)

// One 16-byte piece per lane into LDS (lane l's bytes at lds + 16*l).
__device__ __forceinline__ void copy_b(const void* base, uint32_t range, uint8_t* lds,
                                       uint32_t voff) {
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, range, kBufferRsrcW3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (dma::lds_void*)lds, 16, voff, 0, 0, kBPolicy);
}

// RB: blocks of 16 rows of A.  NG groups of GR stored rows per step.
template <Kind KA, int RB, int ROWB, int NS, int NG, int GR>
struct Cfg {
    static constexpr int U = ROWB / 64;            // chunks per lane and step
    static constexpr int STEPB = ROWB / 16;        // blocks per step
    static constexpr int COLS = NG * GR;           // columns per workgroup
    static constexpr int CB = COLS / 16;           // 16-column blocks
    static constexpr int NBK = GR / 16;            // ... per group
    static constexpr int STAGE = GR * ROWB;        // bytes of one group
    static constexpr int INSTR = STAGE / 1024;     // copies per group
    static constexpr int RPI = 1024 / ROWB;        // rows per copy
    static constexpr int LPR = ROWB / 16;          // lanes per row
    static constexpr int D = NS - 1;               // groups copied ahead
    static constexpr int PA = KA == Kind::MX4 ? 1 : 4;  // 16-byte pieces of A per chunk
    static constexpr int SW = KA == Kind::F16 ? STEPB / 4 : 1;  // scale dwords per row and step
    static constexpr int LA = RB * U * PA + (KA == Kind::MX4 ? RB : 0) + CB;  // loads per step
    static constexpr int RED_ROWS = STAGE / (COLS * 4) < 16 ? STAGE / (COLS * 4) : 16;
    __device__ static int swz(int r) { return ROWB == 256 ? (r & 15) : ((r >> 1) & 7); }
};

template <Kind KA, int RB, int ROWB, int NS, int NG, int GR>
__global__ __launch_bounds__(NW * 64, 1) void mx4_skinny_kernel(Params p, int cols, int nb,
                                                                int mchunks) {
    using G = Cfg<KA, RB, ROWB, NS, NG, GR>;
    constexpr int U = G::U, D = G::D, STAGE = G::STAGE, PA = G::PA, CB = G::CB;
    static_assert(ROWB == 256 || ROWB == 128, "a row piece is 256 or 128 bytes");
    static_assert(NS == 2 || NS == 4, "ring sizes");
    __shared__ __attribute__((aligned(16))) uint8_t st0[NW * STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t st1[NW * STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t st2[NS > 2 ? NW * STAGE : 16];
    __shared__ __attribute__((aligned(16))) uint8_t st3[NS > 2 ? NW * STAGE : 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, i = lane & 15;
    // Workgroups go to the 8 XCDs round-robin: the row chunks of one strip
    // are 8 apart, so that they run on one XCD and share B in its L2.
    const int q8 = blockIdx.x / (8 * mchunks), r8 = blockIdx.x % (8 * mchunks);
    const int strip = 8 * q8 + r8 % 8;
    const int mbase = (r8 / 8) * 16 * RB;
    const int n0 = strip * cols;
    if (n0 >= p.N) return;
    const int nlim = min(n0 + cols, p.N);
    const int rowsA = min(16 * RB, p.M - mbase);

    const int64_t rowbytes = (int64_t)kChunk * nb;
    const uint8_t* gbase[NG];
    uint32_t grange[NG];
#pragma unroll
    for (int cp = 0; cp < NG; ++cp) {
        const int row0 = n0 + GR * cp;
        const int rows = min(GR, nlim - row0);
        gbase[cp] = p.B + (int64_t)row0 * p.ldb;
        grange[cp] = rows <= 0 ? 0u : (uint32_t)((int64_t)(rows - 1) * p.ldb + rowbytes);
    }
    uint32_t vrow[G::INSTR];
    int cb[G::INSTR];  // the lane's chunk within the step
#pragma unroll
    for (int j = 0; j < G::INSTR; ++j) {
        const int lr = G::RPI * j + lane / G::LPR;
        cb[j] = (lane % G::LPR) ^ G::swz(lr);
        vrow[j] = (uint32_t)(lr * p.ldb + 16 * cb[j]);
    }
    const int nsteps = (nb + G::STEPB - 1) / G::STEPB;
    int s0, s1;
    skinny::wave_steps(nsteps, NW, wave, s0, s1);

    // scales of B: rows of the strip; past them the range ends (scale 0,
    // codes 0)
    const uint32_t sprow = (uint32_t)(16 * ((nb + 15) / 16));
    const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(p.SB + (int64_t)n0 * p.ldsb), 0,
        (uint32_t)((int64_t)(nlim - 1 - n0) * p.ldsb + sprow), kBufferRsrcW3);
    // A: MX4 codes and scales through descriptors; 16-bit rows by address
    // (rows past M re-read the last one; their sums are not stored)
    const __amdgpu_buffer_rsrc_t rsa = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(static_cast<const uint8_t*>(p.A) +
                             (KA == Kind::MX4 ? (int64_t)mbase * p.lda : 0)),
        0, KA == Kind::MX4 ? (uint32_t)((int64_t)(rowsA - 1) * p.lda + rowbytes) : 0u, kBufferRsrcW3);
    const __amdgpu_buffer_rsrc_t rssa = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(KA == Kind::MX4 ? p.SA + (int64_t)mbase * p.ldsa : p.SB), 0,
        KA == Kind::MX4 ? (uint32_t)((int64_t)(rowsA - 1) * p.ldsa + sprow) : 0u, kBufferRsrcW3);
    const uint16_t* arow[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
        arow[rb] = static_cast<const uint16_t*>(p.A) +
                   (int64_t)(mbase + min(16 * rb + i, rowsA - 1)) * (KA == Kind::MX4 ? 0 : p.lda);

    floatx4 acc[RB][CB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int c = 0; c < CB; ++c) acc[rb][c] = floatx4{0.f, 0.f, 0.f, 0.f};

    struct Ops {
        u32x4 a[RB][U * PA];
        uint32_t sa[RB], sb[CB][G::SW];  // U scale bytes each (FP16: the step's)
    };

    // Copy group cp of step s into ring stage Q (chunks past the row's end,
    // and steps past the wave's range, read as zeros without memory traffic).
    auto issue = [&](auto qc, auto cpc, int s) DGT_INLINE {
        constexpr int cp = decltype(cpc)::value, Q = decltype(qc)::value;
        uint8_t* dst = dma::pick<Q>(st0, st1, st2, st3) + STAGE * wave;
        const int lim = s < s1 ? nb - G::STEPB * s : 0;
#pragma unroll
        for (int j = 0; j < G::INSTR; ++j) {
            const uint32_t voff = cb[j] < lim ? vrow[j] + (uint32_t)(ROWB * s) : grange[cp];
            copy_b(gbase[cp], grange[cp], dst + 1024 * j, voff);
        }
    };
    auto load_scale = [&](const __amdgpu_buffer_rsrc_t& rs, uint32_t off) DGT_INLINE -> uint32_t {
        if constexpr (U == 4) return __builtin_amdgcn_raw_buffer_load_b32(rs, (int)off, 0, 0);
        else return (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, (int)off, 0, 0);
    };
    // A and the scales of step s (past the last step: the last one's).
    // Always LA vector loads, which the waits below count on; a cut-off step
    // of 16-bit A may issue fewer and waits for everything instead.
    auto load_ops = [&](int s, Ops& o) DGT_INLINE {
        s = min(s, nsteps - 1);
        const int b0 = G::STEPB * s + U * g;  // the lane's first block
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            if constexpr (KA == Kind::F16) {
                static_assert(G::SW == 2, "a step's scales are one 8-byte load");
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(
                    rsb, (int)((16 * c + i) * p.ldsb + G::STEPB * s), 0, 0);
                o.sb[c][0] = v[0];
                o.sb[c][1] = v[1];
            } else {
                o.sb[c][0] = load_scale(rsb, (uint32_t)((16 * c + i) * p.ldsb + b0));
            }
        }
        if constexpr (KA == Kind::MX4) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const bool row_ok = 16 * rb + i < rowsA;
                o.sa[rb] = load_scale(rssa, row_ok ? (uint32_t)((16 * rb + i) * p.ldsa + b0) : 0xfffffff0u);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint32_t off = row_ok && b0 + u < nb
                                             ? (uint32_t)((16 * rb + i) * p.lda + 16 * (b0 + u))
                                             : 0xfffffff0u;
                    o.a[rb][u] = __builtin_bit_cast(
                        u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsa, (int)off, 0, 0));
                }
            }
        } else {
            const bool cut = kBlock * G::STEPB * (s + 1) > p.K;  // uniform
            // piece e of the lane: 8 k from here
            auto at = [&](int e) DGT_INLINE {
                return KA == Kind::F16 ? kBlock * (G::STEPB * s + e) + 8 * g : kBlock * b0 + 8 * e;
            };
            if (!cut) {
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                    for (int e = 0; e < U * PA; ++e) {
                        const u32x4_any v = *reinterpret_cast<const u32x4_any*>(
                            arow[rb] + at(e));
                        o.a[rb][e] = u32x4{v[0], v[1], v[2], v[3]};
                    }
            } else {
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                    for (int e = 0; e < U * PA; ++e)
                        o.a[rb][e] = skinny::load16_cached<uint16_t, true, true>(
                            arow[rb], at(e), p.K, true);
                DMA_WAIT_VMCNT(0);
            }
        }
    };
    // Scale bytes past the last block (in the row's last step) become 2^0.
    auto mask_scales = [&](int s, Ops& o) DGT_INLINE {
        if (G::STEPB * (s + 1) <= nb) return;
        const int left = nb - (G::STEPB * s + U * g);
        const uint32_t keep = left <= 0 ? 0u : left >= 4 ? 0xffffffffu : (1u << (8 * left)) - 1u;
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            if constexpr (KA == Kind::F16) {
#pragma unroll
                for (int d = 0; d < G::SW; ++d) {
                    const int n = nb - (G::STEPB * s + 4 * d);
                    const uint32_t k = n <= 0 ? 0u : n >= 4 ? 0xffffffffu : (1u << (8 * n)) - 1u;
                    o.sb[c][d] = (o.sb[c][d] & k) | (0x7f7f7f7fu & ~k);
                }
            } else {
                o.sb[c][0] = (o.sb[c][0] & keep) | (0x7f7f7f7fu & ~keep);
            }
        }
        if constexpr (KA == Kind::MX4) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) o.sa[rb] = (o.sa[rb] & keep) | (0x7f7f7f7fu & ~keep);
        }
    };
    auto compute = [&](auto qc, auto cpc, const Ops& o) DGT_INLINE {
        constexpr int cp = decltype(cpc)::value, Q = decltype(qc)::value;
        const uint8_t* st = dma::pick<Q>(st0, st1, st2, st3) + STAGE * wave;
        if constexpr (KA == Kind::F16) {
            uint32_t w[G::NBK][G::STEPB];
#pragma unroll
            for (int b = 0; b < G::NBK; ++b)
#pragma unroll
                for (int e = 0; e < G::STEPB; ++e)
                    w[b][e] = *reinterpret_cast<const uint32_t*>(
                        st + (16 * b + i) * ROWB + ((e ^ G::swz(16 * b + i)) << 4) + 4 * g);
            __builtin_amdgcn_sched_barrier(0);  // keep the reads ahead of the products
#pragma unroll
            for (int b = 0; b < G::NBK; ++b)
#pragma unroll
                for (int e = 0; e < G::STEPB; ++e) {
                    const u32x4 v = decode8_f16(w[b][e]);
                    const float sc = scale_number(o.sb[G::NBK * cp + b][e / 4], e % 4);
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb)
                        acc[rb][G::NBK * cp + b] =
                            scaled_product_f16(o.a[rb][e], v, sc, acc[rb][G::NBK * cp + b]);
                    // four products at a time: all at once do not fit the registers
                    if (e % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
            return;
        }
        u32x4 bop[G::NBK][U];
#pragma unroll
        for (int b = 0; b < G::NBK; ++b)
#pragma unroll
            for (int u = 0; u < U; ++u)
                bop[b][u] = *reinterpret_cast<const u32x4*>(
                    st + (16 * b + i) * ROWB + (((U * g + u) ^ G::swz(16 * b + i)) << 4));
        __builtin_amdgcn_sched_barrier(0);  // keep them ahead of the products
        static_for<G::NBK>([&](auto bc) DGT_INLINE {
            constexpr int b = decltype(bc)::value, c = G::NBK * cp + b;
            static_for<U>([&](auto uc) DGT_INLINE {
                constexpr int u = decltype(uc)::value;
                if constexpr (KA == Kind::MX4) {
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb)
                        acc[rb][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            widen(o.a[rb][u]), widen(bop[b][u]), acc[rb][c], 4, 4, u, (int)o.sa[rb],
                            u, (int)o.sb[c][0]);
                } else {
                    const float sc = scale_bits((o.sb[c][0] >> (8 * u)) & 255u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u32x4 w = decode8(bop[b][u][j], sc);
#pragma unroll
                        for (int rb = 0; rb < RB; ++rb) {
                            acc[rb][c] = mfma16x16x32<In::BF16>(o.a[rb][4 * u + j], w, acc[rb][c]);
                        }
                    }
                }
            });
        });
    };
    auto fence = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // Group cp of step s, in ring stage Q.  The wave first copies the group D
    // places ahead (in phase 0 it then loads the next step's operands), then waits until its
    // own copy of this group has landed: newer are the D groups' copies after
    // it, and this step's load of operands when that group's copy was issued in this
    // step's phase 0 or before (cp <= D).  Loads of earlier steps may be newer
    // too; not counting them only waits for more.  A load that waited for
    // everything (a cut-off step) leaves no older copy in flight, so the
    // counts hold after it as well.
    auto phase = [&](auto qc, auto cpc, int s, Ops& o, Ops& next) DGT_INLINE {
        constexpr int cp = decltype(cpc)::value, Q = decltype(qc)::value;
        constexpr int ahead = cp + D;
        DMA_WAIT_VMCNT_LGKM0(63);  // this wave's reads of the stage have returned
        issue(std::integral_constant<int, (Q + D) % NS>{}, std::integral_constant<int, ahead % NG>{},
              s + ahead / NG);
        fence();
        if constexpr (cp == 0) {
            load_ops(s + 1, next);
            fence();
        }
        constexpr int after = G::INSTR * D + (cp <= D ? G::LA : 0);
        DMA_WAIT_VMCNT((after < 63 ? after : 63));
        fence();
        if constexpr (cp == 0) mask_scales(s, o);
        compute(qc, cpc, o);
        fence();
    };
    // Steps whose groups start at ring stage Q0.
    auto step = [&](auto q0c, int s, Ops& o, Ops& next) DGT_INLINE {
        constexpr int Q0 = decltype(q0c)::value;
        static_for<NG>([&](auto cpc) DGT_INLINE {
            phase(std::integral_constant<int, (Q0 + decltype(cpc)::value) % NS>{}, cpc, s, o, next);
        });
    };

    if (s0 < s1) {
        Ops o0, o1;
        auto copies = [&]() DGT_INLINE {
            static_for<D>([&](auto dc) DGT_INLINE {
                constexpr int d = decltype(dc)::value;
                issue(dc, std::integral_constant<int, d % NG>{}, s0 + d / NG);
            });
            fence();
        };
        load_ops(s0, o0);
        fence();
        copies();
        // Unrolled so that ring stages and operand buffers are compile-time.
        constexpr int kRing = NS > NG ? NS / NG : 1;
        constexpr int kUnroll = kRing > 2 ? kRing : 2;
        for (int s = s0; s < s1; s += kUnroll) {
            static_for<kUnroll>([&](auto jc) DGT_INLINE {
                constexpr int j = decltype(jc)::value;
                if (s + j >= s1) return;
                using Q0 = std::integral_constant<int, (j * NG) % NS>;
                if constexpr (j % 2 == 0) step(Q0{}, s + j, o0, o1);
                else step(Q0{}, s + j, o1, o0);
            });
        }
    }
    DMA_WAIT_VMCNT_LGKM0(0);  // every copy has landed: the stages can be reused

    // Partial tiles summed in wave order, RR rows at a time, in stage 0.
    constexpr int RR = G::RED_ROWS, COLS = G::COLS;
    constexpr int kSwz = COLS >= 64 ? 16 : 0;  // spreads a write's four row quarters over banks
    __syncthreads();
    float* red = reinterpret_cast<float*>(st0);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int hh = 0; hh < 16 / RR; ++hh) {
            if (rb + hh) __syncthreads();  // the previous pass's sums have been read
            if ((4 * g) / RR == hh) {
#pragma unroll
                for (int c = 0; c < CB; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        red[(RR * wave + 4 * g + r - RR * hh) * COLS + ((16 * c + i) ^ (kSwz * g))] =
                            acc[rb][c][r];
            }
            __syncthreads();
            for (int o = threadIdx.x; o < RR * COLS; o += NW * 64) {
                const int row = o / COLS, cl = o % COLS, grow = RR * hh + row;
                const int m = 16 * rb + grow, n = n0 + cl;
                if (m >= rowsA || n >= nlim) continue;
                const int at = row * COLS + (cl ^ (kSwz * ((grow >> 2) & 3)));
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < NW; ++w) sum += red[RR * COLS * w + at];
                float* cptr = p.C + (int64_t)(mbase + m) * p.ldc + n;
                *cptr = epilogue(sum, p, cptr, n);
            }
        }
}

template <Kind KA, int RB, int ROWB, int NS, int NG, int GR>
hipError_t launch_cfg(const Params& p, hipStream_t s) {
    constexpr int cols = NG * GR;
    const int mchunks = (int)(((int64_t)p.M + 16 * RB - 1) / (16 * RB));
    const int64_t strips = ((int64_t)p.N + cols - 1) / cols;
    const int64_t wgs = (strips + 7) / 8 * 8 * mchunks;
    if (!launchable(wgs, NW * 64)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((mx4_skinny_kernel<KA, RB, ROWB, NS, NG, GR>), dim3((unsigned)wgs),
                       dim3(NW * 64), 0, s, p, cols, blocks(p.K), mchunks);
    return hipGetLastError();
}

}  // namespace

// The forms that the choice in k_mx4_rows.hip reaches: rb blocks of 16 rows,
// strips of `cols` columns.
hipError_t launch_skinny(const Params& p, int rb, int cols, hipStream_t s) {
    if (rb == 1 && cols == 16) return launch_cfg<Kind::MX4, 1, 256, 2, 1, 16>(p, s);
    if (rb == 1 && cols == 32) return launch_cfg<Kind::MX4, 1, 256, 2, 1, 32>(p, s);
    if (rb == 2 && cols == 32) return launch_cfg<Kind::MX4, 2, 256, 2, 1, 32>(p, s);
    return hipErrorInvalidConfiguration;
}

hipError_t launch_skinny16(In t, const Params& p, int rb, int cols, hipStream_t s) {
    if (t == In::F16 && rb == 1)
        return cols == 16   ? launch_cfg<Kind::F16, 1, 128, 4, 1, 16>(p, s)
               : cols == 32 ? launch_cfg<Kind::F16, 1, 128, 4, 1, 32>(p, s)
                            : launch_cfg<Kind::F16, 1, 128, 4, 2, 32>(p, s);
    if (t == In::BF16 && rb == 1)
        return cols == 16   ? launch_cfg<Kind::BF16, 1, 256, 2, 1, 16>(p, s)
               : cols == 32 ? launch_cfg<Kind::BF16, 1, 256, 2, 1, 32>(p, s)
                            : launch_cfg<Kind::BF16, 1, 256, 2, 2, 32>(p, s);
    if (t == In::BF16 && rb == 2) return launch_cfg<Kind::BF16, 2, 128, 4, 2, 32>(p, s);
    return hipErrorInvalidConfiguration;
}

}  // namespace mx4
}  // namespace dgt
