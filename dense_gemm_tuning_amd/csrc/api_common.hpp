// api_common.hpp -- host-side helpers shared by the C entry points: input
// formats, argument ranges and overlap tests.
#pragma once

#include <cstdint>

#include "../../include/dgt_gemm.h"
#include "gemm_common.hpp"

namespace dgt {
namespace api {

enum class DType { F32, BF16, F16 };

inline int elem_size(DType t) { return t == DType::F32 ? 4 : 2; }

inline bool valid_flag(int f) { return f == 0 || f == 1; }

// Bytes spanned by a rows x cols row-major operand with leading dim ld.
inline uint64_t span_bytes(int rows, int cols, int ld, int esz) {
    if (rows == 0 || cols == 0) return 0;
    return ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * (uint64_t)esz;
}

// [lo, hi) byte range covered by `batch` problems of `span` bytes, `stride`
// bytes apart (empty when span == 0).
struct Range {
    uintptr_t lo, hi;
};
inline Range batch_range(const void* base, uint64_t span, int64_t stride_bytes, int batch) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(base);
    if (span == 0 || batch <= 0) return {b, b};
    return {b, b + (uint64_t)(batch - 1) * (uint64_t)stride_bytes + span};
}
inline bool overlaps(const Range& x, const Range& y) {
    return x.lo < x.hi && y.lo < y.hi && x.lo < y.hi && y.lo < x.hi;
}

// Strides beyond this (in elements) cannot describe device memory; rejecting
// them keeps the range arithmetic below from overflowing.
constexpr int64_t kMaxStride = int64_t(1) << 48;

inline bool valid_stride(int64_t s) { return s >= 0 && s < kMaxStride; }

// The format of a C dtype argument; false when it is none.
inline bool dtype_of(int dtype, DType& t) {
    if (dtype < GEMM_DTYPE_F32 || dtype > GEMM_DTYPE_F16) return false;
    t = dtype == GEMM_DTYPE_F32 ? DType::F32 : dtype == GEMM_DTYPE_BF16 ? DType::BF16 : DType::F16;
    return true;
}

}  // namespace api
}  // namespace dgt
