// strip.hpp -- products of few rows with weights stored N x K (16-bit, or 4-bit
// with group scales), plain or gated: the kernel of k_gated_strip.hip and
// k_w4_strip.hip.  The time is the time to stream the weights once: gated 8 x 28672 x 8192,
// 140 us for 940 MB of 16-bit weights (6.7 TB/s) and 55 for 241 MB of 4-bit ones (4.4 TB/s); plain
// 1 x 28672 x 8192 in 4 bits 26 us (4.7 TB/s).  Small weights are bound by the launch and
// the latency of a wave's steps one after the other (4-bit 1 x 3584 x 8192: 8.7 us for 15 MB).
//
// A workgroup owns a strip of outputs over the whole of K, each of its 8
// waves one range of it; the partial tiles are summed in LDS in wave order
// (deterministic, no atomics, no workspace).  A wave copies its pieces of the
// weights straight into a private LDS ring by buffer loads that write LDS, so
// the loop has no workgroup barrier: a step is ROWB bytes of every stored row of the
// strip, in NG groups of GR rows, copied D = NS - 1 groups ahead.  Of a gated
// strip's groups the even ones are the gate's rows and the odd ones the other
// projection's rows for the same outputs.
//
// Lane (i, g) = (lane % 16, lane / 16) of a 16-row block takes 8 of every 32 k of row
// i: 16 bytes of a 16-bit weight (k 8g .. 8g+7), a dword of codes.  Of a scale
// group of GB blocks of 32 k it takes k 8*GB*g .. 8*GB*(g+1)-1, GB neighbouring dwords, as GB
// products.  The activations are loaded the same way into registers a step ahead.
// Chunk c (16 bytes) of row r sits at c ^ swz(r) in LDS: 16 rows reading one
// chunk touch 16 distinct 16-byte bank groups.
//
// 4-bit weights: a code in a byte, read as an E4M3 number, is the code times
// 2^-9 (they are that format's subnormal numbers and its first binade), so the scaled
// conversion gives the codes themselves, exactly, two per instruction; no
// weight is rounded.  The even codes of a dword come from its low halves of bytes and the
// odd ones from the high halves, so the activations are put into the order 0 2 4 6 1 3
// 5 7 once a step.  Per group acc += s * (sum xq - z * sum x), with sum x a product
// with ones, once for all rows of the strip, or (kKeepSums) with -z inside the
// same sum.
#pragma once

#include "dma_common.hpp"
#include "mx4_device.hpp"
#include "skinny_common.hpp"
#include "w4.hpp"

namespace dgt {
namespace strip {

using mx4::static_for;
using skinny::u32x4_any;

constexpr int NW = 8;        // waves per workgroup
constexpr int kBPolicy = 2;  // cache policy of the weights' copies: nt (streamed once)

struct Params {
    int M, N, K;
    const uint16_t* X;
    int64_t ldx;                   // elements
    const uint8_t* W[2];           // rows of output 0 on (plain: the first only)
    int64_t ldw[2];                // bytes
    int chunks;                    // 16-byte pieces of a row
    const uint16_t* S[2];          // 4-bit weights: scales and zero points
    const uint8_t* Z[2];           // (null: 8)
    int64_t lds, ldz;
    int groups;
    bool s_bf16;
    // gated
    gated::Act act;
    const float *bg, *bu;
    uint16_t *H, *G, *U;
    int64_t ldh, ldg, ldu;
    // plain
    float alpha, beta;
    float* C;
    int64_t ldc;
    const float* bias;
};

// kW4: 4-bit weights, 2^LG blocks of 32 k a scale group.
template <bool kW4_, int LG_, bool kGated_, int RB_, int NG_, int GR_, int ROWB_>
struct Cfg {
    static constexpr bool kW4 = kW4_, kGated = kGated_;
    static constexpr int RB = RB_, NG = NG_, GR = GR_, ROWB = ROWB_;
    static constexpr int NS = 4, D = NS - 1;
    static constexpr int KS = kW4 ? 2 * ROWB : ROWB / 2;  // k per step
    static constexpr int P = KS / 32;                     // 32-k blocks per step
    static constexpr int CPS = ROWB / 16;                 // chunks of a row per step
    static constexpr int NBK = GR / 16;                   // 16-row blocks per group
    static constexpr int CB = NG * NBK;                   // ... per strip
    static constexpr int ROWS = NG * GR;                  // stored rows per strip
    static constexpr int COLS = kGated ? ROWS / 2 : ROWS; // outputs per strip
    static constexpr int STAGE = GR * ROWB;
    static constexpr int INSTR = STAGE / 1024, RPI = 1024 / ROWB, LPR = ROWB / 16;
    static constexpr int GB = 1 << LG_;                   // blocks per scale group
    static constexpr int GPS = kW4 ? P / GB : 1;          // scale groups per step
    // Scales and zero points: a lane loads kRun groups' of one stored row at a time (16
    // and 8 bytes), SPS steps' worth, a step ahead.  (A row's next groups lie in the
    // same cache line, but the streamed weights drive it out of L1 between steps: two
    // groups at a time fetched more bytes of scales than of codes.)
    static constexpr int kRun = 8, SPS = kRun / GPS;
    static_assert(!kW4 || SPS * GPS == kRun, "a run is whole steps");
    static constexpr int NSC = kW4 ? (ROWS + 63) / 64 : 0;
    // Vector loads per step besides the copies (those of scales where every
    // step has them; elsewhere they are not counted, which only waits for more).
    static constexpr int LA = RB * P + (SPS == 1 ? 2 * NSC : 0);
    // Whether the activations' sums per scale group are made once a step and kept, or
    // (their registers are many when the scale groups are) the products with
    // the zero point are added up with those with the codes.
    static constexpr bool kKeepSums = RB * GPS <= 4;
    // rows of a reduction pass in one stage of all waves
    static constexpr int RR = STAGE / (ROWS * 4) < 16 ? STAGE / (ROWS * 4) : 16;
    static_assert(ROWB == 256 || ROWB == 128, "a row piece is 256 or 128 bytes");
    static_assert(NG == 1 || NG == 2 || NG == 4 || NG == 8, "groups map onto the ring");
    static_assert(!kGated || NG % 2 == 0, "a gated strip's groups come in pairs");
    static_assert(!kW4 || P % GB == 0, "a scale group does not cross steps");
    static_assert(RR >= 4, "a pass holds an accumulator's rows");
    __device__ static int swz(int r) {  // 256 / ROWB rows share a line of all banks
        return ROWB == 256 ? (r & 15) : ((r >> 1) & 7);
    }
    // Loads of operands behind the copy of group cp of the wave's step t, D phases
    // before that group's wait: one in each phase 0 behind its copy.  In the first kFirst steps
    // some of those phases are the prologue, which loads before it copies.
    static constexpr int kFirst = NG >= D + 1 ? 0 : (D + NG - 1) / NG;
    static constexpr int loads(int cp, int t) {
        int n = 0;
        for (int x = cp - D; x <= cp; ++x) n += x >= -t * NG && x % NG == 0;
        return n;
    }
};
static_assert(Cfg<true, 2, false, 1, 4, 16, 128>::kFirst == 0 &&
                  Cfg<true, 2, false, 1, 4, 16, 128>::loads(0, 0) == 1 &&
                  Cfg<true, 2, false, 1, 4, 16, 128>::loads(3, 0) == 1 &&
                  Cfg<true, 2, false, 1, 2, 16, 128>::loads(1, 0) == 1 &&
                  Cfg<true, 2, false, 1, 2, 16, 128>::loads(0, 2) == 2 &&
                  Cfg<true, 2, false, 1, 1, 16, 128>::kFirst == 3 &&
                  Cfg<true, 2, false, 1, 1, 16, 128>::loads(0, 3) == 4 &&
                  Cfg<false, 0, true, 1, 8, 16, 256>::loads(4, 0) == 0,
              "loads behind a group's copy");

// 16-bit ones, and the 8 codes of a dword as 16-bit numbers in the order
// 0 2 4 6 1 3 5 7.
template <In T>
__device__ __forceinline__ u32x4 ones() {
    const uint32_t o = T == In::BF16 ? 0x3f803f80u : 0x3c003c00u;
    return u32x4{o, o, o, o};
}
template <In T>
__device__ __forceinline__ u32x4 decode8(uint32_t q) {
    const uint32_t lo = q & 0x0f0f0f0fu, hi = (q >> 4) & 0x0f0f0f0fu;
    if constexpr (T == In::BF16) {
        return u32x4{
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true))};
    } else {
        return u32x4{
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, true)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, true))};
    }
}
// Eight activations in that order.
__device__ __forceinline__ u32x4 even_odd(const u32x4& x) {
    constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;  // halves of two dwords, side by side
    return u32x4{__builtin_amdgcn_perm(x[1], x[0], kLow), __builtin_amdgcn_perm(x[3], x[2], kLow),
                 __builtin_amdgcn_perm(x[1], x[0], kHigh), __builtin_amdgcn_perm(x[3], x[2], kHigh)};
}

// One 16-byte piece per lane into LDS (lane l's bytes at lds + 16*l).
__device__ __forceinline__ void copy_piece(const void* base, uint32_t range, uint8_t* lds,
                                           uint32_t voff) {
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, range, kBufferRsrcW3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (dma::lds_void*)lds, 16, voff, 0, 0, kBPolicy);
}

template <In T, typename G>
__global__ __launch_bounds__(NW * 64, 1) void strip_kernel(Params p, int cols, int mchunks) {
    constexpr bool kW4 = G::kW4, kGated = G::kGated;
    constexpr int RB = G::RB, NG = G::NG, GR = G::GR, ROWB = G::ROWB, NS = G::NS, D = G::D, P = G::P,
                  CB = G::CB, NBK = G::NBK, STAGE = G::STAGE, GPS = G::GPS, GB = G::GB;
    // One object per stage, so that the compiler's wait-count pass can tell a
    // copy into one from reads of another.
    __shared__ __attribute__((aligned(256))) uint8_t st0[NW * STAGE];
    __shared__ __attribute__((aligned(256))) uint8_t st1[NW * STAGE];
    __shared__ __attribute__((aligned(256))) uint8_t st2[NW * STAGE];
    __shared__ __attribute__((aligned(256))) uint8_t st3[NW * STAGE];
    // A run's scales and zero points, [wave][stored row][group]: a scale as fp32, whose last
    // 13 bits or more are zero, with the zero point in its last byte.
    __shared__ __attribute__((aligned(16))) uint32_t factors[kW4 ? NW * G::ROWS * G::kRun : 4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, i = lane & 15;
    // Workgroups go to the 8 XCDs round-robin: the row chunks of one strip
    // are 8 apart, so that they run on one XCD and share the weights in its L2.
    const int q8 = blockIdx.x / (8 * mchunks), r8 = blockIdx.x % (8 * mchunks);
    const int64_t first = (int64_t)(8 * q8 + r8 % 8) * cols;
    if (first >= p.N) return;
    const int n0 = (int)first, nlim = (int)min(first + cols, (int64_t)p.N);
    const int mbase = (r8 / 8) * 16 * RB;
    const int rows_x = min(16 * RB, p.M - mbase);

    // group cp's matrix and first output
    auto matrix = [](int cp) { return kGated ? cp & 1 : 0; };
    auto out0 = [&](int cp) { return n0 + GR * (kGated ? cp >> 1 : cp); };
    const uint8_t* gbase[NG];
    uint32_t grange[NG];
#pragma unroll
    for (int cp = 0; cp < NG; ++cp) {
        const int rows = min(GR, nlim - out0(cp));
        gbase[cp] = p.W[matrix(cp)] + (int64_t)out0(cp) * p.ldw[matrix(cp)];
        grange[cp] = rows <= 0 ? 0u
                               : (uint32_t)((int64_t)(rows - 1) * p.ldw[matrix(cp)] +
                                            16 * (int64_t)p.chunks);
    }
    uint32_t vrow[kGated ? 2 : 1][G::INSTR];
    int cb[G::INSTR];  // the lane's chunk within the step
#pragma unroll
    for (int j = 0; j < G::INSTR; ++j) {
        const int lr = G::RPI * j + lane / G::LPR;
        cb[j] = (lane % G::LPR) ^ G::swz(lr);
#pragma unroll
        for (int m = 0; m < (kGated ? 2 : 1); ++m) vrow[m][j] = (uint32_t)(lr * p.ldw[m] + 16 * cb[j]);
    }
    const int nsteps = (p.chunks + G::CPS - 1) / G::CPS;
    int s0, s1;
    skinny::wave_steps(nsteps, NW, wave, s0, s1);

    // rows past M re-read the last one; their sums are not stored
    auto row_x = [&](int rb) {
        return p.X + (int64_t)(mbase + min(16 * rb + i, rows_x - 1)) * p.ldx;
    };
    // k of the row's last whole piece; where it has none, the weight's first bytes are loaded
    const int whole = p.K & ~7, klast = max(whole - 8, 0);
    const uint16_t* xrow[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
        xrow[rb] = whole > 0 ? row_x(rb) : reinterpret_cast<const uint16_t*>(p.W[0]);

    floatx4 acc[RB][CB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int c = 0; c < CB; ++c) acc[rb][c] = floatx4{0.f, 0.f, 0.f, 0.f};

    struct Ops {
        u32x4 a[RB][P];
    };
    struct Scales {
        uint32_t s[kW4 ? G::NSC : 1][G::kRun / 2], z[kW4 ? G::NSC : 1][G::kRun / 4];
    };

    // Copy group cp of step s into ring stage Q (chunks past the row's end, and
    // steps past the wave's range, read as zeros without memory traffic).
    auto issue = [&](auto qc, auto cpc, int s) DGT_INLINE {
        constexpr int cp = decltype(cpc)::value, Q = decltype(qc)::value;
        uint8_t* dst = dma::pick<Q>(st0, st1, st2, st3) + STAGE * wave;
        const int lim = s < s1 ? p.chunks - G::CPS * s : 0;
#pragma unroll
        for (int j = 0; j < G::INSTR; ++j) {
            const uint32_t voff =
                cb[j] < lim ? vrow[matrix(cp)][j] + (uint32_t)(ROWB * s) : grange[cp];
            copy_piece(gbase[cp], grange[cp], dst + 1024 * j, voff);
        }
    };

    // The lane's rows of scales and zero points: stored row 64j + lane (past the
    // strip its last one, whose sums are not stored).
    const uint16_t* srow[kW4 ? G::NSC : 1];
    const uint8_t* zrow[kW4 ? G::NSC : 1];
    if constexpr (kW4) {
#pragma unroll
        for (int j = 0; j < G::NSC; ++j) {
            const int r = min(64 * j + lane, G::ROWS - 1), cp = r / GR;
            const int64_t out = min(out0(cp) + r % GR, nlim - 1);
            srow[j] = (matrix(cp) ? p.S[1] : p.S[0]) + out * p.lds;
            zrow[j] = p.Z[0] ? (matrix(cp) ? p.Z[1] : p.Z[0]) + out * p.ldz : p.W[0];
        }
    }
    // First k of the lane's product e in a step, from 8*GB*g on.
    auto piece = [](int e) { return 32 * GB * (e / GB) + 8 * (e % GB); };
    const bool few = p.groups < G::kRun;  // then no wave has more than a run
    // First scale group to load for the run that starts with step s: its own, or where the
    // row ends in it the last ones of the row.
    auto group_at = [&](int s) DGT_INLINE { return min(GPS * s, p.groups - G::kRun); };
    // Activations of step s (past the last step: the last one's): RB*P vector
    // loads, which the waits below count on.  Past K the row's last whole piece is loaded, and
    // replaced in `prepare`.  (No branch: where two ways meet, the compiler counts the
    // loads of the shorter one and waits for copies that are still on their way.)
    auto load_ops = [&](int s, Ops& o) DGT_INLINE {
        s = min(s, nsteps - 1);
        const int k0 = G::KS * s + 8 * GB * g;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const u32x4_any v =
                    *reinterpret_cast<const u32x4_any*>(xrow[rb] + min(k0 + piece(e), klast));
                o.a[rb][e] = u32x4{v[0], v[1], v[2], v[3]};
            }
    };
    // The run of scales and zero points from step s on (none of the row's where
    // there are fewer or no zero points: then replaced in `prepare`).
    auto load_scales = [&](int s, Scales& o) DGT_INLINE {
        const int at = group_at(min(s, nsteps - 1));
#pragma unroll
        for (int j = 0; j < G::NSC; ++j) {
            const void* sp = few ? static_cast<const void*>(p.W[0]) : srow[j] + at;
            const void* zp = few || !p.Z[0] ? p.W[0] : zrow[j] + at;
            __builtin_memcpy(o.s[j], sp, 2 * G::kRun);
            __builtin_memcpy(o.z[j], zp, G::kRun);
        }
    };
    auto load_few = [&](Scales& o) DGT_INLINE {
#pragma unroll
        for (int j = 0; j < G::NSC; ++j) {
#pragma unroll
            for (int d = 0; d < G::kRun / 2; ++d) o.s[j][d] = 0u;
#pragma unroll
            for (int d = 0; d < G::kRun / 4; ++d) o.z[j][d] = 0u;
#pragma unroll
            for (int e = 0; e + 1 < G::kRun; ++e) {  // past the last group: it again, not used
                const int at = min(e, p.groups - 1);
                o.s[j][e / 2] |= (uint32_t)srow[j][at] << (16 * (e % 2));
                o.z[j][e / 4] |= (uint32_t)zrow[j][p.Z[0] ? at : 0] << (8 * (e % 4));
            }
        }
    };

    floatx4 xs[RB][kW4 && G::kKeepSums ? GPS : 1];
    // A run of scales into LDS (this wave's part, and LDS keeps its order); past
    // the row's last group scales of 0: its sums are zero, but what is stored there
    // may be anything.
    const uint32_t smask = p.s_bf16 ? 0xffffffffu : 0u;
    uint32_t* const fac = factors + (kW4 ? G::ROWS * G::kRun * wave : 0);
    auto put_scales = [&](int s, Scales& o) DGT_INLINE {
        constexpr int SW = G::kRun / 2, ZW = G::kRun / 4;
        const int skip = GPS * s - (few ? 0 : group_at(s)), left = p.groups - GPS * s;  // uniform
        const uint32_t no_z = p.Z[0] ? 0u : 0xffffffffu;
#pragma unroll
        for (int j = 0; j < G::NSC; ++j) {
#pragma unroll 1
            for (int t = 0; t < skip; ++t) {  // groups before the run
#pragma unroll
                for (int d = 0; d < SW; ++d)
                    o.s[j][d] = (o.s[j][d] >> 16) | (d + 1 < SW ? o.s[j][(d + 1) % SW] << 16 : 0u);
#pragma unroll
                for (int d = 0; d < ZW; ++d)
                    o.z[j][d] = (o.z[j][d] >> 8) | (d + 1 < ZW ? o.z[j][(d + 1) % ZW] << 24 : 0u);
            }
            uint32_t f[G::kRun];
#pragma unroll
            for (int e = 0; e < G::kRun; ++e) {
                // one of the two values by masks: a branch for each would break up the code
                const uint32_t bits = (o.s[j][e / 2] >> (16 * (e % 2))) & 0xffffu;
                const uint32_t half = __float_as_uint(w4::scale_value(bits, false));
                const uint32_t z = (o.z[j][e / 4] >> (8 * (e % 4))) & 255u;
                f[e] = ((bits << 16) & smask) | (half & ~smask) | (z & ~no_z) | (8u & no_z);
                f[e] = e < left ? f[e] : 0u;
            }
            if (64 * (j + 1) <= G::ROWS || lane < G::ROWS - 64 * j)
                __builtin_memcpy(__builtin_assume_aligned(fac + (64 * j + lane) * G::kRun, 16), f,
                                 4 * G::kRun);
        }
        asm volatile("" ::: "memory");
    };
    // Once a step: zeros past K; the activations' order (sums do not mind it),
    // and their sums.
    auto prepare = [&](int s, Ops& o) DGT_INLINE {
        if (G::KS * (s + 1) > p.K) {  // uniform
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                u32x4 tail = {0u, 0u, 0u, 0u};  // the row's last elements, fewer than 8
                if (kW4 && whole < p.K)
                    tail = skinny::load16_cached<uint16_t, true, true>(row_x(rb), whole, p.K, true);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const int k = G::KS * s + 8 * GB * g + piece(e);
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        o.a[rb][e][d] = k < whole ? o.a[rb][e][d] : k == whole ? tail[d] : 0u;
                }
            }
        }
        if constexpr (kW4) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
                for (int e = 0; e < P; ++e) o.a[rb][e] = even_odd(o.a[rb][e]);
                if constexpr (G::kKeepSums) {
#pragma unroll
                    for (int j = 0; j < GPS; ++j) xs[rb][j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < P; ++e)
                        xs[rb][e / GB] = mfma16x16x32<T>(o.a[rb][e], ones<T>(), xs[rb][e / GB]);
                }
            }
        }
    };
    // Byte of the lane's first chunk in a group's stage, row i; chunks further on by
    // a power of two differ in one bit of the swizzled place, and 16 rows further
    // on the swizzle is the same.
    const uint32_t lds_at =
        kW4 ? (uint32_t)(i * ROWB + (((GB * g / 4) ^ G::swz(i)) << 4) + 4 * GB * g % 16)
            : (uint32_t)(i * ROWB + ((g ^ G::swz(i)) << 4));
    static_assert(kW4 || GB == 1, "16-bit weights have no groups");
    auto compute = [&](auto qc, auto cpc, int s, const Ops& o) DGT_INLINE {
        constexpr int cp = decltype(cpc)::value, Q = decltype(qc)::value;
        const uint8_t* st = dma::pick<Q>(st0, st1, st2, st3) + STAGE * wave;
        // not known to the compiler to be the same every time: it would keep
        // every address made from it in a register of its own
        uint32_t at = lds_at;
        asm volatile("" : "+v"(at));
        if constexpr (kW4) {
            uint32_t q[NBK][P];
#pragma unroll
            for (int b = 0; b < NBK; ++b)
#pragma unroll
                for (int u = 0; u < GPS; ++u)
                    __builtin_memcpy(q[b] + GB * u,
                                     __builtin_assume_aligned(
                                         st + (at ^ (16 * GB * u)) + 16 * b * ROWB, 4 * GB),
                                     4 * GB);
            uint32_t f[NBK][GPS];
#pragma unroll
            for (int b = 0; b < NBK; ++b)
                __builtin_memcpy(f[b],
                                 __builtin_assume_aligned(
                                     fac + (GR * cp + 16 * b + i) * G::kRun + GPS * ((s - s0) % G::SPS),
                                     GPS >= 4 ? 16 : 4 * GPS),
                                 4 * GPS);
            __builtin_amdgcn_sched_barrier(0);  // keep the reads ahead of the products
#pragma unroll
            for (int j = 0; j < GPS; ++j) {
#pragma unroll
                for (int b = 0; b < NBK; ++b) {
                    constexpr int c0 = NBK * cp;
                    const float sc = __uint_as_float(f[b][j] & 0xffffff00u);
                    const float z = (float)(f[b][j] & 255u);
                    floatx4 sum[RB];
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) sum[rb] = floatx4{0.f, 0.f, 0.f, 0.f};
                    if constexpr (!G::kKeepSums) {
                        const uint32_t nz = gated::to_bits<T>(-z), pair = nz | (nz << 16);
                        const u32x4 w = {pair, pair, pair, pair};
#pragma unroll
                        for (int e = GB * j; e < GB * (j + 1); ++e)
#pragma unroll
                            for (int rb = 0; rb < RB; ++rb)
                                sum[rb] = mfma16x16x32<T>(o.a[rb][e], w, sum[rb]);
                    }
#pragma unroll
                    for (int e = GB * j; e < GB * (j + 1); ++e) {
                        const u32x4 w = decode8<T>(q[b][e]);
#pragma unroll
                        for (int rb = 0; rb < RB; ++rb) sum[rb] = mfma16x16x32<T>(o.a[rb][e], w, sum[rb]);
                    }
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            float v = sum[rb][r];
                            if constexpr (G::kKeepSums) v = fmaf(-z, xs[rb][j][r], v);
                            acc[rb][c0 + b][r] = fmaf(sc, v, acc[rb][c0 + b][r]);
                        }
                    // here and not later: the compiler would keep the groups' sums instead
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) asm volatile("" : "+v"(acc[rb][c0 + b]));
                }
                // a few products at a time: all at once do not fit the registers
                if (GB * (j + 1) % 2 == 0) __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            u32x4 w[NBK][P];
#pragma unroll
            for (int b = 0; b < NBK; ++b)
#pragma unroll
                for (int e = 0; e < P; ++e)
                    w[b][e] = *reinterpret_cast<const u32x4*>(st + (at ^ (64 * e)) + 16 * b * ROWB);
            __builtin_amdgcn_sched_barrier(0);  // keep the reads ahead of the products
#pragma unroll
            for (int b = 0; b < NBK; ++b)
#pragma unroll
                for (int e = 0; e < P; ++e)
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb)
                        acc[rb][NBK * cp + b] =
                            mfma16x16x32<T>(o.a[rb][e], w[b][e], acc[rb][NBK * cp + b]);
        }
    };
    auto fence = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // Group cp of step s, in ring stage Q.  The wave first copies the group D
    // places ahead (in phase 0 it then loads the next step's operands), then
    // waits until its own copy of this group has landed: newer are the D
    // groups' copies after it, and the loads of operands in the phases since (G::loads).
    auto phase = [&](auto qc, auto cpc, int s, Ops& o, Ops& next, Scales& sc) DGT_INLINE {
        constexpr int cp = decltype(cpc)::value, Q = decltype(qc)::value;
        constexpr int ahead = cp + D;
        DMA_WAIT_VMCNT_LGKM0(63);  // this wave's reads of the stage have returned
        issue(std::integral_constant<int, (Q + D) % NS>{}, std::integral_constant<int, ahead % NG>{},
              s + ahead / NG);
        fence();
        if constexpr (cp == 0) {
            if constexpr (kW4) {
                if ((s - s0) % G::SPS == 0) put_scales(s, sc);
                fence();
            }
            load_ops(s + 1, next);
            if constexpr (kW4) {
                if ((s + 1 - s0) % G::SPS == 0) load_scales(s + 1, sc);
            }
            fence();
        }
        static_for<G::kFirst + 1>([&](auto tc) DGT_INLINE {
            constexpr int t = decltype(tc)::value;
            constexpr int after = G::INSTR * D + G::LA * G::loads(cp, t);
            if (G::kFirst == 0 || (t == G::kFirst ? s - s0 >= t : s - s0 == t)) {  // uniform
                DMA_WAIT_VMCNT((after < 63 ? after : 63));
            }
        });
        fence();
        if constexpr (cp == 0) prepare(s, o);
        compute(qc, cpc, s, o);
        fence();
    };
    // A step whose groups start at ring stage Q0.
    auto step = [&](auto q0c, int s, Ops& o, Ops& next, Scales& sc) DGT_INLINE {
        constexpr int Q0 = decltype(q0c)::value;
        static_for<NG>([&](auto cpc) DGT_INLINE {
            phase(std::integral_constant<int, (Q0 + decltype(cpc)::value) % NS>{}, cpc, s, o, next,
                  sc);
        });
    };

    if (s0 < s1) {
        Scales sc;
        Ops o0, o1;
        load_ops(s0, o0);
        if constexpr (kW4) {
            load_scales(s0, sc);
            if (few) load_few(sc);
        }
        fence();
        static_for<D>([&](auto dc) DGT_INLINE {
            constexpr int d = decltype(dc)::value;
            issue(dc, std::integral_constant<int, d % NG>{}, s0 + d / NG);
        });
        fence();
        // Unrolled so that ring stages and operand buffers are compile-time.
        constexpr int kRing = NS > NG ? NS / NG : 1;
        constexpr int kUnroll = kRing > 2 ? kRing : 2;
        for (int s = s0; s < s1; s += kUnroll) {
            static_for<kUnroll>([&](auto jc) DGT_INLINE {
                constexpr int j = decltype(jc)::value;
                if (s + j >= s1) return;
                using Q0 = std::integral_constant<int, (j * NG) % NS>;
                if constexpr (j % 2 == 0) step(Q0{}, s + j, o0, o1, sc);
                else step(Q0{}, s + j, o1, o0, sc);
            });
        }
    }
    DMA_WAIT_VMCNT_LGKM0(0);  // every copy has landed: the stages can be reused

    // Partial tiles summed in wave order, RR rows at a time, in stage 0: wave
    // w's row at (RR*w + row)*ROWS, stored row 16c + i of the strip at
    // (16c + i) ^ (kSwz * (row/4)), which spreads a write's four row quarters over banks.
    constexpr int RR = G::RR, ROWS = G::ROWS;
    constexpr int kSwz = ROWS >= 64 ? 16 : 0;
    __syncthreads();
    float* red = reinterpret_cast<float*>(st0);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int hh = 0; hh < 16 / RR; ++hh) {
            if (16 * rb + RR * hh >= rows_x) continue;  // uniform
            if (rb + hh) __syncthreads();  // the previous pass's sums have been read
            if ((4 * g) / RR == hh) {
#pragma unroll
                for (int c = 0; c < CB; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        red[(RR * wave + 4 * g + r - RR * hh) * ROWS + ((16 * c + i) ^ (kSwz * g))] =
                            acc[rb][c][r];
            }
            __syncthreads();
            for (int o = threadIdx.x; o < RR * G::COLS; o += NW * 64) {
                const int row = o / G::COLS, cl = o % G::COLS, grow = RR * hh + row;
                const int m = 16 * rb + grow, n = n0 + cl;
                if (m >= rows_x || n >= nlim) continue;
                auto total = [&](int stored) DGT_INLINE {
                    const int at = row * ROWS + (stored ^ (kSwz * ((grow >> 2) & 3)));
                    float sum = 0.0f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) sum += red[RR * ROWS * w + at];
                    return sum;
                };
                const int64_t mm = mbase + m;
                if constexpr (kGated) {
                    const int at = 2 * GR * (cl / GR) + cl % GR;  // its row in an even group
                    float x = total(at), u = total(at + GR);
                    if (p.bg) x += p.bg[n];
                    if (p.bu) u += p.bu[n];
                    p.H[mm * p.ldh + n] = gated::to_bits<T>(gated::act_of(p.act, x) * u);
                    if (p.G) p.G[mm * p.ldg + n] = gated::to_bits<T>(x);
                    if (p.U) p.U[mm * p.ldu + n] = gated::to_bits<T>(u);
                } else {
                    float* c = p.C + mm * p.ldc + n;
                    const float sum = total(cl);
                    const float r = p.beta == 0.0f ? p.alpha * sum : p.alpha * sum + p.beta * *c;
                    *c = p.bias ? r + p.bias[n] : r;
                }
            }
        }
}

// Strips as narrow as the number of rounds of the CUs (a workgroup each) that the widest
// would take allows.  us, so and whole strips, K = 8192: 16-bit gated 1 x 1000 12.1/14.1, 1 x 3584 20.7/20.5, 8 x 9000
// 48/52, 8 x 28672 139/149, 64 x 28672 173/182; 4-bit 1 x 3584 8.8/9.4, 1 x 14336 15.7/15.2, 8 x 28672 27.5/28.6.
template <In T, typename G>
hipError_t launch(const Params& p, hipStream_t s) {
    const int64_t mchunks = ((int64_t)p.M + 16 * G::RB - 1) / (16 * G::RB);
    const int64_t rounds = (((int64_t)p.N + G::COLS - 1) / G::COLS + dma::kCUs - 1) / dma::kCUs;
    const int cols = (int)(((int64_t)p.N + rounds * dma::kCUs - 1) / (rounds * dma::kCUs));
    const int64_t strips = ((int64_t)p.N + cols - 1) / cols;
    const int64_t wgs = (strips + 7) / 8 * 8 * mchunks;
    if (wgs >= (int64_t(1) << 32) / (NW * 64)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((strip_kernel<T, G>), dim3((unsigned)wgs), dim3(NW * 64), 0, s, p, cols,
                       (int)mchunks);
    return hipGetLastError();
}

}  // namespace strip

namespace w4 {
// The kernel with shared activations (k_w4_rows.hip).
hipError_t launch_rows(In t, bool gate, int log_group, const strip::Params& p, hipStream_t s);
}  // namespace w4

}  // namespace dgt
