// Argument checks shared by the host layers: orders, the extents that
// matrices touch, and overlaps of such extents.  Nothing here calls HIP.
#pragma once

#include <cstdint>

#include "libgemm.h"

namespace libgemm {

inline bool valid_order(int o) { return o == GEMM_ROW_MAJOR || o == GEMM_COL_MAJOR; }

// Elements spanned by one rows x cols matrix stored with leading dimension ld.
inline int64_t span(int64_t rows, int64_t cols, int order, int64_t ld) {
    if (rows == 0 || cols == 0) return 0;
    const int64_t outer = order == GEMM_ROW_MAJOR ? rows : cols;
    const int64_t inner = order == GEMM_ROW_MAJOR ? cols : rows;
    return (outer - 1) * ld + inner;
}

// Byte range [lo, hi) that a batched operand touches.
struct Range {
    uintptr_t lo, hi;
};

inline Range range_of(const void *p, int64_t span_elems, int64_t batch, int64_t stride, int esize) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    const int64_t elems = span_elems == 0 ? 0 : (batch - 1) * stride + span_elems;
    return {lo, lo + static_cast<uintptr_t>(elems) * static_cast<uintptr_t>(esize)};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

// Product of non-negative dimensions overflowing int64 (or the 2^31 grid).
inline bool too_big(int64_t a, int64_t b) { return a != 0 && b > INT64_MAX / a; }

}  // namespace libgemm
