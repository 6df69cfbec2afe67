// k_gated_strip.hip -- which strips (strip.hpp) the gated projections of up to
// 64 rows take with 16-bit weights.
#include "strip.hpp"

namespace dgt {
namespace gated {

namespace {

// RB blocks of 16 rows, NG groups of GR stored rows of ROWB bytes a step.
template <int RB, int NG, int GR, int ROWB>
using Cfg = strip::Cfg<false, 0, true, RB, NG, GR, ROWB>;

}  // namespace

// 16-byte aligned rows of whole 16-byte pieces (a piece is then inside K or
// outside), and offsets of a group's rows below 2^31.
bool strip_eligible(const Forward& p) {
    auto rows_ok = [](const void* at, int64_t ld) {
        return rows_16b_aligned(at, ld, 2) && ld < kMaxBufferPitch;
    };
    return p.M <= kSkinnyMaxM && p.K > 0 && p.K % 8 == 0 && rows_ok(p.X, p.ldx) &&
           rows_ok(p.Wg, p.ldwg) && rows_ok(p.Wu, p.ldwu);
}

template <In T>
hipError_t launch_forward_strip(const Forward& p, hipStream_t s) {
    strip::Params q = {};
    q.M = p.M; q.N = p.N; q.K = p.K;
    q.X = p.X; q.ldx = p.ldx;
    q.W[0] = reinterpret_cast<const uint8_t*>(p.Wg); q.ldw[0] = 2 * p.ldwg;
    q.W[1] = reinterpret_cast<const uint8_t*>(p.Wu); q.ldw[1] = 2 * p.ldwu;
    q.chunks = p.K / 8;
    q.act = p.act;
    q.bg = p.bg; q.bu = p.bu;
    q.H = p.H; q.ldh = p.ldh;
    q.G = p.G; q.ldg = p.ldg;
    q.U = p.U; q.ldu = p.ldu;
    // Strips of 16 outputs where that gives every CU at most one, then of 32, then of 64.  us, this rule and
    // strips of 64 alone, K = 8192: 1 x 3584 21 and 30, 16 x 3584 22 and 34, 32 x 3584 28 and 43, 64 x 3584 42 and
    // 57, 16 x 8192 55 and 57, 32 x 8192 57 and 62, 64 x 8192 64 and 72 (strips of 16 there 83).
    const bool few = p.N <= 16 * dma::kCUs, some = p.N <= 32 * dma::kCUs;
    auto take = [&](auto narrow, auto middle, auto wide) {
        return few    ? strip::launch<T, decltype(narrow)>(q, s)
               : some ? strip::launch<T, decltype(middle)>(q, s)
                      : strip::launch<T, decltype(wide)>(q, s);
    };
    if (p.M > 32) return take(Cfg<4, 2, 16, 128>{}, Cfg<4, 2, 32, 128>{}, Cfg<4, 4, 32, 128>{});
    if (p.M > 16) return take(Cfg<2, 2, 16, 256>{}, Cfg<2, 4, 16, 256>{}, Cfg<2, 8, 16, 256>{});
    return take(Cfg<1, 2, 16, 256>{}, Cfg<1, 4, 16, 256>{}, Cfg<1, 8, 16, 256>{});
}
template hipError_t launch_forward_strip<In::BF16>(const Forward&, hipStream_t);
template hipError_t launch_forward_strip<In::F16>(const Forward&, hipStream_t);

}  // namespace gated
}  // namespace dgt
