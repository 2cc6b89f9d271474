// Address-range and alignment checks shared by the C entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace q4 {

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + bytes};
}

inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace q4
