// Argument checks shared by the translation units of the C ABI.
#pragma once

#include "spg_common.h"

namespace spg {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
inline bool aligned2(const void *p) { return ((uintptr_t)p & 1u) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// [a0, a1) and [b0, b1) share a byte.
inline bool overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes)
{
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return abytes > 0 && bbytes > 0 && a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}
inline int64_t extent(int64_t rows, int64_t ld, int64_t cols) { return rows > 0 ? (rows - 1) * ld + cols : 0; }
// Byte extents of n pieces `stride` apart stay far inside 64 bits.
inline bool addressable(int64_t n, int64_t stride) { return n <= 1 || stride < (INT64_C(1) << 56) / n; }

struct Range {
    const void *p;
    int64_t bytes;
};
// An output (outs[0 .. n)) shares a byte with another or with an input.
inline bool any_overlap(const Range *outs, int n, const Range *ins, int m)
{
    for (int i = 0; i < n; ++i) {
        for (int j = i + 1; j < n; ++j)
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
        for (int j = 0; j < m; ++j)
            if (overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return true;
    }
    return false;
}

}  // namespace spg
