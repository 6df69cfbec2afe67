// k_w4_strip.hip -- which strips (strip.hpp) a product of few rows with 4-bit
// weights takes.
#include "strip.hpp"

namespace dgt {
namespace w4 {

namespace {

using strip::Cfg;

// 2^LG blocks of 32 k a scale group.  Strips of at most as many rows as give every CU one
// (kGated: half as many outputs), wider ones where there are more rows than that: 16 to 128.  us, with this rule and
// with strips of 128 rows alone, K = 8192, one row of activations: 3584 8.8 and 20.6, 8192 12.2 and 20.7,
// 14336 15.6 and 21.4; gated 3584 12.0 and 20.1, 8192 17.4 and 22.6; 16 rows: 3584 14 and 25, 14336 21 and 28.
template <In T, int LG, bool kGated>
hipError_t launch_group(const strip::Params& p, hipStream_t s) {
    constexpr int kPair = kGated ? 2 : 1;
    constexpr int64_t kCUs = dma::kCUs;
    if (p.N <= 16 * kCUs) return strip::launch<T, Cfg<true, LG, kGated, 1, kPair, 16, 128>>(p, s);
    if constexpr (!kGated) {
        if (p.N <= 32 * kCUs) return strip::launch<T, Cfg<true, LG, false, 1, 2, 16, 128>>(p, s);
    }
    if (p.N <= 64 / kPair * kCUs) return strip::launch<T, Cfg<true, LG, kGated, 1, 4, 16, 128>>(p, s);
    return strip::launch<T, Cfg<true, LG, kGated, 1, 8, 16, 128>>(p, s);
}

template <bool kGated>
hipError_t launch_strips(In t, int log_group, const strip::Params& p, hipStream_t s) {
    // Strips load the activations once per strip and wave: more rows take the kernel that shares
    // them.  us, strips against it, K = 8192, groups of 128: 28672 x 32 44/41, x 64 80/59, x 256 285/228; 14336 x
    // 32 39/29, x 64 71/39; 8192 x 32 29/28, x 48 41/28, x 64 51/28; 3584 x 32 24/28, x 48 34/28, x 64 43/27; 4096
    // x 4096 x 32 15/16, x 64 27/16; gated 8192 x 32 39/29, gated 3584 x 32 28/28, x 64 50/28.
    const bool wide = (kGated ? 2 : 1) * (int64_t)p.N > 32 * dma::kCUs;
    if (p.M > 32 || (p.M > 16 && wide)) return launch_rows(t, kGated, log_group, p, s);
    auto go = [&](auto tc) {
        constexpr In T = decltype(tc)::value;
        return log_group == 5   ? launch_group<T, 0, kGated>(p, s)
               : log_group == 6 ? launch_group<T, 1, kGated>(p, s)
                                : launch_group<T, 2, kGated>(p, s);
    };
    return t == In::BF16 ? go(std::integral_constant<In, In::BF16>{})
                         : go(std::integral_constant<In, In::F16>{});
}

strip::Params of_weight(const Weight& w, int M, int N, int K, const uint16_t* X, int64_t ldx) {
    strip::Params p = {};
    p.M = M; p.N = N; p.K = K;
    p.X = X; p.ldx = ldx;
    p.chunks = mx4::blocks(K);
    p.groups = groups(K, w.log_group);
    p.lds = w.lds; p.ldz = w.ldz;
    p.s_bf16 = w.s_bf16;
    for (int m = 0; m < 2; ++m) {  // the second half's rows start at row N
        p.W[m] = w.Q + (int64_t)m * N * w.ldq;
        p.ldw[m] = w.ldq;
        p.S[m] = w.S + (int64_t)m * N * w.lds;
        p.Z[m] = w.Z ? w.Z + (int64_t)m * N * w.ldz : nullptr;
    }
    return p;
}

}  // namespace

hipError_t launch_product(In t, const Product& p, hipStream_t s) {
    strip::Params q = of_weight(p.w, p.M, p.N, p.K, p.A, p.lda);
    q.alpha = p.alpha; q.beta = p.beta;
    q.C = p.C; q.ldc = p.ldc;
    q.bias = p.bias;
    return launch_strips<false>(t, p.w.log_group, q, s);
}

hipError_t launch_gated(In t, const Gated& p, hipStream_t s) {
    strip::Params q = of_weight(p.w, p.M, p.N, p.K, p.X, p.ldx);
    q.act = p.act;
    q.bg = p.bg; q.bu = p.bu;
    q.H = p.H; q.ldh = p.ldh;
    return launch_strips<true>(t, p.w.log_group, q, s);
}

}  // namespace w4
}  // namespace dgt
