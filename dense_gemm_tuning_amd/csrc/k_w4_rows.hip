// k_w4_rows.hip -- products of more than a few rows with 4-bit weights, plain and
// gated: what strip.hpp does not reuse, the activations, is shared here.
//
// A workgroup has a strip of 64 or 128 stored rows of the weight (gated: half of them of the gate's and
// the same ones of the other projection's) and 32 or 64 rows of activations.  A step of 256 k
// of both is copied by DMA into one of three LDS stages, two steps ahead, and one
// barrier a step both publishes the step and retires the stage before it.  The 8
// waves split the step's k two ways and the stored rows four ways, each with all
// rows of the activations: those are then read four times from LDS, and every code is
// decoded once (by waves side by side in the rows they would be decoded again for each).
//
// Decoding and the scale groups' sums are strip.hpp's, but that here the codes
// are put into the activations' order (two byte permutes a dword).  Scales and
// zero points come in runs of 8 groups: a lane for each stored row loads its own in a run's last step and
// writes them, joined, to the one of two LDS buffers that the next run reads.
//
// Workgroups start at different runs and wrap around: all at one k, they would ask for
// the same columns of rows whose pitch is often a power of two.
//
// Bound by the products and the decoding, which share each SIMD's issue and start together behind
// the barrier: 64 x 28672 x 8192 takes 62 us, 54 without the copies and 35 with them alone (a step's
// 32 KB of activations and 16 KB of codes); without the sums of x, a third of the products, 52.  (Those
// sums made once for the four waves that share them, and subtracted a step later, took 65.)
// Rows of activations off 16-byte boundaries (or with pitches from 2^24 on) go through registers, on the
// smallest tile: 28672 x 8192, 32 rows 52 us, 64 93, 256 322.  Tiles of 32 x 128 and 64 x 128 through registers, timed
// but not built, are faster where there is work for them (28672 x 8191, 32 x 64, 32 x 128 and 64 x 128, us: 32 rows
// 55/50/71, 64 102/92/68, 256 330/300/264; 64 x 3584 37/43/63).
#include "strip.hpp"

namespace dgt {
namespace w4 {

namespace {

using mx4::static_for;
using strip::Params;

constexpr int NWAVE = 8, NS = 3, KS = 2, ROWB = 128, kRun = 8;
constexpr int STEPK = 2 * ROWB, CPS = ROWB / 16;      // k and chunks of a weight's row per step
constexpr int BPW = STEPK / 32 / KS;                  // blocks of 32 k per wave and step
constexpr int AROW = 2 * STEPK;                       // bytes of a row of activations per step

using uint32x2 = uint32_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ int swz_a(int r) { return r & 15; }
__device__ __forceinline__ int swz_b(int r) { return (r >> 1) & 7; }

template <int kPolicy>
__device__ __forceinline__ void copy_piece(const void* base, uint32_t range, uint8_t* lds,
                                           uint32_t voff) {
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, range, kBufferRsrcW3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (dma::lds_void*)lds, 16, voff, 0, 0, kPolicy);
}

// The 8 codes of a dword as 16-bit numbers in their order.
template <In T>
__device__ __forceinline__ u32x4 decode8(uint32_t q) {
    const uint32_t lo = q & 0x0f0f0f0fu, hi = (q >> 4) & 0x0f0f0f0fu;
    const uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u);  // codes 0 1 2 3, a byte each
    const uint32_t b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
    if constexpr (T == In::BF16) {
        return u32x4{
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, true)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, true))};
    } else {
        return u32x4{
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 512.0f, true)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.0f, true))};
    }
}

__device__ __forceinline__ uint32_t lds_address(const void* at) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)at;
}
// A step's codes of a stored row, or of two 16 apart (four dwords each, at the four addresses), and
// the factors of their G groups.  Read by hand: the compiler takes some of the
// copies on their way for writes of what it reads here, and waits for all of them.
template <int G, int CBW>
__device__ __forceinline__ void read_weight(const uint32_t (&at)[BPW], const uint32_t* factors,
                                            uint32_t (&q)[BPW][CBW], uint32_t (&f)[CBW][G]) {
    static_assert(BPW == 4 && 16 * kRun * 4 == 512 && 16 * ROWB == 8 * 64 * 4, "the offsets");
    static_assert((G == 1 || G == 2 || G == 4) && (CBW == 1 || CBW == 2), "a factor's read");
    using V = std::conditional_t<G == 1, uint32_t, std::conditional_t<G == 2, uint32x2, u32x4>>;
    V v[2];
    const uint32_t fat = lds_address(factors);
    if constexpr (CBW == 1) {
#define DGT_READ_WEIGHT(F)                                                                            \
    asm volatile("ds_read_b32 %0, %5\n\tds_read_b32 %1, %6\n\tds_read_b32 %2, %7\n\tds_read_b32 %3, %8\n\t" \
                 F " %4, %9\n\ts_waitcnt lgkmcnt(0)"                                                  \
                 : "=&v"(q[0][0]), "=&v"(q[1][0]), "=&v"(q[2][0]), "=&v"(q[3][0]), "=&v"(v[0])        \
                 : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(fat)                           \
                 : "memory")
        if constexpr (G == 1) DGT_READ_WEIGHT("ds_read_b32");
        else if constexpr (G == 2) DGT_READ_WEIGHT("ds_read_b64");
        else DGT_READ_WEIGHT("ds_read_b128");
#undef DGT_READ_WEIGHT
    } else {
        uint32x2 p[BPW];
#define DGT_READ_WEIGHT(F)                                                                      \
    asm volatile("ds_read2st64_b32 %0, %6 offset1:8\n\t"                                        \
                 "ds_read2st64_b32 %1, %7 offset1:8\n\t"                                        \
                 "ds_read2st64_b32 %2, %8 offset1:8\n\t"                                        \
                 "ds_read2st64_b32 %3, %9 offset1:8\n\t"                                        \
                 F " %4, %10\n\t"                                                               \
                 F " %5, %10 offset:512\n\t"                                                    \
                 "s_waitcnt lgkmcnt(0)"                                                         \
                 : "=&v"(p[0]), "=&v"(p[1]), "=&v"(p[2]), "=&v"(p[3]), "=&v"(v[0]), "=&v"(v[1]) \
                 : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(fat)                     \
                 : "memory")
        if constexpr (G == 1) DGT_READ_WEIGHT("ds_read_b32");
        else if constexpr (G == 2) DGT_READ_WEIGHT("ds_read_b64");
        else DGT_READ_WEIGHT("ds_read_b128");
#undef DGT_READ_WEIGHT
#pragma unroll
        for (int e = 0; e < BPW; ++e)
#pragma unroll
            for (int c = 0; c < CBW; ++c) q[e][c] = p[e][c];
    }
#pragma unroll
    for (int c = 0; c < CBW; ++c)
#pragma unroll
        for (int j = 0; j < G; ++j) {
            if constexpr (G == 1) f[c][j] = v[c];
            else f[c][j] = v[c][j];
        }
}

// 2^LG blocks of 32 k a scale group; RBT blocks of 16 rows of activations, CBW of the weight a wave.
// kAny: rows of activations that start anywhere go through registers, loaded at a step's start and stored
// to the free stage at its end.
template <In T, int LG, bool kGated, int RBT, int CBW, bool kAny>
// (two workgroups a CU of the smallest tile: registers for four waves a SIMD)
__global__ __launch_bounds__(NWAVE * 64, RBT * CBW == 2 ? 4 : 2) void w4_rows_kernel(Params p, int mchunks) {
    constexpr int GB = 1 << LG, GPS = STEPK / 32 / GB, GPW = GPS / KS, SPS = kRun / GPS;
    constexpr int ROWS = 16 * CBW * NWAVE / KS;      // stored rows of a strip
    constexpr int B_BYTES = ROWS * ROWB, IB = B_BYTES / 1024 / NWAVE;  // copies per wave
    constexpr int kPart = kGated ? ROWS / 2 : ROWS;  // stored rows of one matrix
    constexpr int A_BYTES = 16 * RBT * AROW, IA = A_BYTES / 1024 / NWAVE;
    constexpr int STAGE = B_BYTES + A_BYTES, COPIES = (kAny ? 0 : IA) + IB;
    static_assert(A_BYTES % (1024 * NWAVE) == 0, "whole copies per wave");
    // One object per stage, so that the compiler's wait-count pass can tell a
    // copy into one from reads of another.
    __shared__ __attribute__((aligned(1024))) uint8_t st0[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t st2[STAGE];
    // [run % 2][stored row][group of the run]: the scale as fp32, whose last 13
    // bits or more are zero, with the zero point in its last byte
    __shared__ __attribute__((aligned(16))) uint32_t factors[2 * ROWS * kRun];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, i = lane & 15;
    const int wk = wave % KS, wc = wave / KS;
    // the row chunks of one strip on one XCD, as in strip.hpp
    const int q8 = blockIdx.x / (8 * mchunks), r8 = blockIdx.x % (8 * mchunks);
    const int64_t first = (int64_t)(8 * q8 + r8 % 8) * kPart;
    if (first >= p.N) return;
    const int n0 = (int)first, nlim = min(n0 + kPart, p.N);
    const int mbase = (r8 / 8) * 16 * RBT;
    const int rows_x = min(16 * RBT, p.M - mbase);
    const int nsteps = (p.chunks + CPS - 1) / CPS, nruns = (nsteps + SPS - 1) / SPS;

    // Steps in order, run by run from the workgroup's first one: step k is the r-th of its run.
    struct Place {
        int run, r, k;
    };
    auto advance = [&](Place& at) DGT_INLINE {
        ++at.r;
        ++at.k;
        if (at.r == SPS || at.k == nsteps) {
            at.run = at.run + 1 == nruns ? 0 : at.run + 1;
            at.r = 0;
            at.k = at.run * SPS;
        }
    };
    Place now, ahead;
    now.run = (int)((unsigned)q8 % (unsigned)nruns);
    now.r = 0;
    now.k = now.run * SPS;
    ahead = now;

    const int pieces_x = (p.K + 7) / 8;  // 16-byte pieces of a row of activations
    const int64_t pitch_x = 2 * p.ldx;
    const uint8_t* base_x = reinterpret_cast<const uint8_t*>(p.X) + (int64_t)mbase * pitch_x;
    const uint32_t range_x = (uint32_t)((int64_t)(rows_x - 1) * pitch_x + 16 * (int64_t)pieces_x);
    const uint8_t* base_w[IB];
    uint32_t voff_w[IB], voff_x[IA], range_w;
    int cw[IB], cx[IA];  // the lane's piece within the step
    range_w = (uint32_t)((int64_t)(nlim - n0 - 1) * p.ldw[0] + 16 * (int64_t)p.chunks);
#pragma unroll
    for (int j = 0; j < IB; ++j) {  // 8 stored rows a copy
        const int row = 8 * (IB * wave + j) + lane / 8;
        const int m = 8 * (IB * wave + j) / kPart;  // uniform
        base_w[j] = (m ? p.W[1] : p.W[0]) + (int64_t)n0 * p.ldw[0];
        cw[j] = (lane % 8) ^ swz_b(row);
        voff_w[j] = (uint32_t)((row - kPart * m) * p.ldw[0] + 16 * cw[j]);
    }
#pragma unroll
    for (int j = 0; j < IA; ++j) {  // 2 rows a copy
        const int row = 2 * (IA * wave + j) + lane / 32;
        cx[j] = (lane % 32) ^ swz_a(row);
        voff_x[j] = (uint32_t)(row * pitch_x + 16 * cx[j]);
    }
    // Step k's copies into stage Q; with !real none of it (the copies are
    // counted, and read zeros without memory traffic).
    auto copy_step = [&](auto qc, int k, bool real) DGT_INLINE {
        uint8_t* st = dma::pick<decltype(qc)::value>(st0, st1, st2, st0);
        const int lim_w = real ? p.chunks - CPS * k : 0, lim_x = real ? pieces_x - 4 * CPS * k : 0;
#pragma unroll
        for (int j = 0; j < IB; ++j)
            copy_piece<2>(base_w[j], range_w, st + 1024 * (IB * wave + j),
                          cw[j] < lim_w ? voff_w[j] + (uint32_t)(ROWB * k) : 0xfffffff0u);
        if (kAny) return;
#pragma unroll
        for (int j = 0; j < IA; ++j)
            copy_piece<1>(base_x, range_x, st + B_BYTES + 1024 * (IA * wave + j),
                          cx[j] < lim_x ? voff_x[j] + (uint32_t)(AROW * k) : 0xfffffff0u);
    };

    // The same of the activations of any alignment: a piece that crosses a row's end or lies behind it is
    // the row's last 8 elements, shifted (rows past the last one are that one, and not stored).
    const uint16_t* row_x[IA];
#pragma unroll
    for (int j = 0; j < IA; ++j)
        row_x[j] = p.X + (mbase + min(2 * (IA * wave + j) + lane / 32, rows_x - 1)) * p.ldx;
    auto load_x = [&](int k, u32x4 (&v)[IA]) DGT_INLINE {
        if (p.K < 8) {  // uniform; then there is one step
#pragma unroll
            for (int j = 0; j < IA; ++j)
                v[j] = gated::gather8(row_x[j], STEPK * k + 8 * cx[j], p.K);
            return;
        }
#pragma unroll
        for (int j = 0; j < IA; ++j)
            v[j] = gated::load16(row_x[j] + min(STEPK * k + 8 * cx[j], p.K - 8));
    };
    auto store_x = [&](auto qc, int k, u32x4 (&v)[IA]) DGT_INLINE {
        uint8_t* st = dma::pick<decltype(qc)::value>(st0, st1, st2, st0);
        const bool cut = STEPK * (k + 1) > p.K && p.K >= 8;  // uniform
#pragma unroll
        for (int j = 0; j < IA; ++j) {
            const int past = min(max(STEPK * k + 8 * cx[j] - (p.K - 8), 0), 8);
            *reinterpret_cast<u32x4*>(st + B_BYTES + 1024 * (IA * wave + j) + 16 * lane) =
                cut ? gated::shift_out(v[j], past) : v[j];
        }
    };

    // Scales: lane tid's stored row.
    const bool loads_scales = wave < ROWS / 64;  // uniform
    const uint16_t* srow = nullptr;
    const uint8_t* zrow = nullptr;
    if (loads_scales) {
        const int m = tid / kPart;
        const int64_t out = min(n0 + tid % kPart, nlim - 1);  // rows past the strip: not stored
        srow = (m ? p.S[1] : p.S[0]) + out * p.lds;
        zrow = p.Z[0] ? (m ? p.Z[1] : p.Z[0]) + out * p.ldz : p.W[0];
    }
    const bool few = p.groups < kRun;  // then there is one run
    struct Scales {
        uint32_t s[kRun / 2], z[kRun / 4];
    };
    // A run's, or where the row ends in it the row's last ones.
    auto load_scales = [&](int run, Scales& o) DGT_INLINE {
        const int at = min(kRun * run, p.groups - kRun);
        __builtin_memcpy(o.s, srow + at, 2 * kRun);
        __builtin_memcpy(o.z, zrow + (p.Z[0] ? at : 0), kRun);
    };
    auto load_few = [&](Scales& o) DGT_INLINE {
#pragma unroll
        for (int d = 0; d < kRun / 2; ++d) o.s[d] = 0u;
#pragma unroll
        for (int d = 0; d < kRun / 4; ++d) o.z[d] = 0u;
#pragma unroll
        for (int e = 0; e + 1 < kRun; ++e) {  // past the last group: it again, not used
            const int at = min(e, p.groups - 1);
            o.s[e / 2] |= (uint32_t)srow[at] << (16 * (e % 2));
            o.z[e / 4] |= (uint32_t)zrow[p.Z[0] ? at : 0] << (8 * (e % 4));
        }
    };
    const uint32_t smask = p.s_bf16 ? 0xffffffffu : 0u;
    // Into the run's buffer; past the row's last group scales of 0 (their sums are
    // zero, but what is stored there may be anything).
    auto put_scales = [&](int run, int buf, Scales& o) DGT_INLINE {
        const int skip = few ? 0 : kRun * run - min(kRun * run, p.groups - kRun);
        const int left = p.groups - kRun * run;
        const uint32_t no_z = p.Z[0] ? 0u : 0xffffffffu;
#pragma unroll 1
        for (int t = 0; t < skip; ++t) {  // groups before the run
#pragma unroll
            for (int d = 0; d < kRun / 2; ++d)
                o.s[d] = (o.s[d] >> 16) | (d + 1 < kRun / 2 ? o.s[(d + 1) % (kRun / 2)] << 16 : 0u);
#pragma unroll
            for (int d = 0; d < kRun / 4; ++d)
                o.z[d] = (o.z[d] >> 8) | (d + 1 < kRun / 4 ? o.z[(d + 1) % (kRun / 4)] << 24 : 0u);
        }
        uint32_t f[kRun];
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
            const uint32_t bits = (o.s[e / 2] >> (16 * (e % 2))) & 0xffffu;
            const uint32_t half = __float_as_uint(scale_value(bits, false));
            const uint32_t z = (o.z[e / 4] >> (8 * (e % 4))) & 255u;
            f[e] = ((bits << 16) & smask) | (half & ~smask) | (z & ~no_z) | (8u & no_z);
            f[e] = e < left ? f[e] : 0u;
        }
        __builtin_memcpy(__builtin_assume_aligned(factors + (ROWS * buf + tid) * kRun, 16), f, 4 * kRun);
    };

    floatx4 acc[RBT][CBW];
#pragma unroll
    for (int rb = 0; rb < RBT; ++rb)
#pragma unroll
        for (int c = 0; c < CBW; ++c) acc[rb][c] = floatx4{0.f, 0.f, 0.f, 0.f};

    // The wave's part of step `at`, in stage st.
    auto compute = [&](const uint8_t* st, const Place& at, int buf) DGT_INLINE {
        const uint8_t* sx = st + B_BYTES;
        const int row0 = 16 * CBW * wc + i;  // the lane's row of the first block, and 16 on
        uint32_t from[BPW];
#pragma unroll
        for (int e = 0; e < BPW; ++e)
            from[e] = lds_address(st + row0 * ROWB + (((BPW * wk + e) ^ swz_b(row0)) << 4) + 4 * g);
        uint32_t q[BPW][CBW], f[CBW][GPW];
        read_weight<GPW, CBW>(from, factors + (ROWS * buf + row0) * kRun + GPS * at.r + GPW * wk, q, f);
#pragma unroll
        for (int j = 0; j < GPW; ++j) {
            floatx4 sum[RBT][CBW], xs[RBT];
#pragma unroll
            for (int rb = 0; rb < RBT; ++rb) {
                xs[rb] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < CBW; ++c) sum[rb][c] = floatx4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int e = GB * j; e < GB * (j + 1); ++e) {
                const int blk = BPW * wk + e;
                u32x4 a[RBT];
#pragma unroll
                for (int rb = 0; rb < RBT; ++rb) {
                    const int row = 16 * rb + i;
                    a[rb] = *reinterpret_cast<const u32x4*>(sx + row * AROW +
                                                            (((4 * blk + g) ^ swz_a(row)) << 4));
                }
#pragma unroll
                for (int rb = 0; rb < RBT; ++rb)
                    xs[rb] = mfma16x16x32<T>(a[rb], strip::ones<T>(), xs[rb]);
#pragma unroll
                for (int c = 0; c < CBW; ++c) {
                    const u32x4 w = decode8<T>(q[e][c]);
#pragma unroll
                    for (int rb = 0; rb < RBT; ++rb) sum[rb][c] = mfma16x16x32<T>(a[rb], w, sum[rb][c]);
                }
            }
#pragma unroll
            for (int c = 0; c < CBW; ++c) {
                const float s = __uint_as_float(f[c][j] & 0xffffff00u), z = (float)(f[c][j] & 255u);
#pragma unroll
                for (int rb = 0; rb < RBT; ++rb) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[rb][c][r] = fmaf(s, fmaf(-z, xs[rb][r], sum[rb][c][r]), acc[rb][c][r]);
                    // here and not later: the compiler would keep the groups' sums instead
                    asm volatile("" : "+v"(acc[rb][c]));
                }
            }
        }
    };
    auto fence = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // The s-th step, in stage Q; its run's scales are in buffer `buf`.  At the wait the
    // wave's copies of the step after it are newer than its own; waves that also load scales
    // wait for more.
    int buf = 0;
    auto step = [&](auto qc, int s) DGT_INLINE {
        constexpr int Q = decltype(qc)::value;
        DMA_WAIT_VMCNT_LGKM0(((NS - 2) * COPIES));
        dma::barrier();  // step s is in LDS for every wave; the stage of step s - 1 is free
        if (!kAny && p.K % 8 != 0 && now.k == nsteps - 1) {
            // what follows k = K - 1 in the rows' last pieces may be anything
            if (tid < 16 * RBT) {
                uint8_t* piece = dma::pick<Q>(st0, st1, st2, st0) + B_BYTES + tid * AROW +
                                 (((p.K / 8 - 4 * CPS * now.k) ^ swz_a(tid)) << 4);
                for (int e = p.K % 8; e < 8; ++e) reinterpret_cast<uint16_t*>(piece)[e] = 0;
            }
            fence();
            DMA_WAIT_VMCNT_LGKM0(0);
            dma::barrier();
        }
        Scales sc;
        // the last of its run, and there is another
        const bool last = !few && (now.r == SPS - 1 || now.k == nsteps - 1);
        const int next = now.run + 1 == nruns ? 0 : now.run + 1;
        if (loads_scales && last) load_scales(next, sc);
        fence();
        constexpr std::integral_constant<int, (Q + NS - 1) % NS> next_stage{};
        const int next_k = ahead.k;
        u32x4 v[IA];
        if constexpr (kAny) {
            load_x(next_k, v);
            fence();
        }
        copy_step(next_stage, next_k, s + NS - 1 < nsteps);
        advance(ahead);
        fence();
        const uint8_t* st = dma::pick<Q>(st0, st1, st2, st0);
        compute(st, now, buf);
        if constexpr (kAny) {
            fence();
            store_x(next_stage, next_k, v);
        }
        if (last) {
            buf ^= 1;
            if (loads_scales) put_scales(next, buf, sc);
        }
        fence();
        advance(now);
    };
    if (loads_scales) {
        Scales sc;
        if (few) load_few(sc);
        else load_scales(now.run, sc);
        put_scales(now.run, 0, sc);
    }
    fence();
    static_for<NS - 1>([&](auto qc) DGT_INLINE {
        if constexpr (kAny) {
            u32x4 v[IA];
            load_x(ahead.k, v);
            store_x(qc, ahead.k, v);
            fence();
        }
        copy_step(qc, ahead.k, decltype(qc)::value < nsteps);
        advance(ahead);
    });
    fence();
    // Stages are compile-time; whole rounds of them, then the rest.  (With steps that may be skipped in
    // the loop, the compiler counts the copies of ways through it that no run takes, and waits
    // for some that are still on their way.)
    int s = 0;
    for (; s + NS <= nsteps; s += NS)
        static_for<NS>([&](auto jc) DGT_INLINE { step(jc, s + decltype(jc)::value); });
    static_for<NS - 1>([&](auto jc) DGT_INLINE {
        constexpr int j = decltype(jc)::value;
        if (s + j < nsteps) step(jc, s + j);
    });
    DMA_WAIT_VMCNT_LGKM0(0);  // no copy may still target LDS: the stages are reused

    // The KS partial tiles, 16 rows at a time in stages 0 and 1 in turn (one
    // barrier per pass: a buffer is written again two passes later).
    static_assert(16 * KS * ROWS * 4 <= STAGE, "a pass fits a stage");
    dma::barrier();
    static_for<RBT>([&](auto rbc) DGT_INLINE {
        constexpr int rb = decltype(rbc)::value;
        if (16 * rb >= rows_x) return;  // uniform
        float* red = reinterpret_cast<float*>(dma::pick<rb % 2>(st0, st1, st0, st0));
#pragma unroll
        for (int c = 0; c < CBW; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                red[(16 * wk + 4 * g + r) * ROWS + ((16 * (CBW * wc + c) + i) ^ (16 * g))] =
                    acc[rb][c][r];
        __syncthreads();
        for (int e = tid; e < 16 * kPart; e += NWAVE * 64) {
            const int row = e / kPart, cl = e % kPart;
            const int64_t m = mbase + 16 * rb + row;
            const int n = n0 + cl;
            if (16 * rb + row >= rows_x || n >= nlim) continue;
            auto total = [&](int stored) DGT_INLINE {
                const int at = row * ROWS + (stored ^ (16 * (row >> 2)));
                return red[at] + red[16 * ROWS + at];
            };
            static_assert(KS == 2, "two parts");
            if constexpr (kGated) {
                float x = total(cl), u = total(kPart + cl);
                if (p.bg) x += p.bg[n];
                if (p.bu) u += p.bu[n];
                p.H[m * p.ldh + n] = gated::to_bits<T>(gated::act_of(p.act, x) * u);
            } else {
                float* c = p.C + m * p.ldc + n;
                const float sum = total(cl);
                const float r = p.beta == 0.0f ? p.alpha * sum : p.alpha * sum + p.beta * *c;
                *c = p.bias ? r + p.bias[n] : r;
            }
        }
    });
}

template <In T, int LG, bool kGated, int RBT, int CBW, bool kAny = false>
hipError_t launch(const Params& p, hipStream_t s) {
    constexpr int kCols = 16 * CBW * NWAVE / KS / (kGated ? 2 : 1);  // outputs of a strip
    const int64_t mchunks = ((int64_t)p.M + 16 * RBT - 1) / (16 * RBT);
    const int64_t strips = ((int64_t)p.N + kCols - 1) / kCols;
    const int64_t wgs = (strips + 7) / 8 * 8 * mchunks;
    if (wgs >= (int64_t(1) << 32) / (NWAVE * 64)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((w4_rows_kernel<T, LG, kGated, RBT, CBW, kAny>), dim3((unsigned)wgs), dim3(NWAVE * 64),
                       0, s, p, (int)mchunks);
    return hipGetLastError();
}

// Rows of activations by stored rows of a workgroup.  Its time does not depend on how many of them are
// there: 27, 37 and 55 us for K = 8192 (groups of 128; 27 becomes 42 where a CU has two of the smallest, whose LDS and
// registers allow that), so the tile is the one whose rounds of the CUs take least, and its strips are not narrowed where
// CUs are idle (narrowed against whole strips, us: 33 x 129 27.7/26.7, 64 x 3584 28.1/27.5, 64 x 28672 59.5/60.0).
// us, 32 x 64, 32 x 128 and 64 x 128 at K = 8192: 32 x 8192 28/37/52, 64 x 8192 28/38/56, 64 x 14336 43/39/56, 64 x 28672
// 83/76/59, 128 x 8192 44/39/56, 256 x 8192 85/76/61, 256 x 3584 42/38/56.  (64 x 64 takes as long as 32 x 128.)  Groups of
// 32 take longer at every tile and rank them alike: 64 x 8192 31/49/72, 64 x 14336 53/55/76, 64 x 28672 104/105/81,
// 128 x 8192 53/54/76, 256 x 8192 100/104/77, 256 x 3584 51/52/74; so do groups of 64, in between.
enum class Tile { R32x64, R32x128, R64x128 };
Tile tile_of(int64_t M, int64_t stored) {
    auto wgs = [&](int rows, int strip) { return (M + rows - 1) / rows * ((stored + strip - 1) / strip); };
    constexpr int64_t kCUs = dma::kCUs;
    const int64_t small = wgs(32, 64), rest = small % (2 * kCUs);
    const int64_t t32x64 = small / (2 * kCUs) * 42 + (rest == 0 ? 0 : rest <= kCUs ? 27 : 42);
    const int64_t t32x128 = (wgs(32, 128) + kCUs - 1) / kCUs * 37;
    const int64_t t64x128 = (wgs(64, 128) + kCUs - 1) / kCUs * 55;
    if (t64x128 < t32x64 && t64x128 < t32x128) return Tile::R64x128;
    return t32x128 < t32x64 ? Tile::R32x128 : Tile::R32x64;
}

template <In T, bool kGated>
hipError_t launch_group(const Params& p, int log_group, hipStream_t s) {
    const Tile tile = tile_of(p.M, (kGated ? 2 : 1) * (int64_t)p.N);
    const bool any = !rows_16b_aligned(p.X, p.ldx, 2) || p.ldx >= kMaxBufferPitch;
    auto rows = [&](auto lg) {
        constexpr int LG = decltype(lg)::value;
        if (any) return launch<T, LG, kGated, 2, 1, true>(p, s);
        if (tile == Tile::R64x128) return launch<T, LG, kGated, 4, 2>(p, s);
        return tile == Tile::R32x128 ? launch<T, LG, kGated, 2, 2>(p, s) : launch<T, LG, kGated, 2, 1>(p, s);
    };
    return log_group == 5   ? rows(std::integral_constant<int, 0>{})
           : log_group == 6 ? rows(std::integral_constant<int, 1>{})
                            : rows(std::integral_constant<int, 2>{});
}

}  // namespace

hipError_t launch_rows(In t, bool gate, int log_group, const Params& p, hipStream_t s) {
    if (t == In::BF16)
        return gate ? launch_group<In::BF16, true>(p, log_group, s)
                    : launch_group<In::BF16, false>(p, log_group, s);
    return gate ? launch_group<In::F16, true>(p, log_group, s)
                : launch_group<In::F16, false>(p, log_group, s);
}

}  // namespace w4
}  // namespace dgt
