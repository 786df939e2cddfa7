// Argument checks shared by the C entries.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ssm_detail {

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

inline Range range_of(const void *p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + (uintptr_t)bytes};
}

inline bool overlaps(Range a, Range b) {
    if (a.lo == a.hi || b.lo == b.hi || a.lo == 0 || b.lo == 0) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a * b without overflow, both >= 0
inline bool mul_ok(int64_t a, int64_t b, int64_t *out) {
    if (a == 0 || b == 0) { *out = 0; return true; }
    if (a > INT64_MAX / b) return false;
    *out = a * b;
    return true;
}

// Whether a launch's work items stay below 2^32, the most that one may have
inline bool grid_ok(int64_t blocks, int threads) { return blocks <= (int64_t)(UINT32_MAX / (unsigned)threads); }

}  // namespace ssm_detail
