// Byte ranges of buffers, for the checks that a call's buffers do not overlap.  No HIP call.
#pragma once

#include <cstdint>

namespace adacomp {

struct Range {
    uintptr_t lo, hi;
};
inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }
inline Range range_of(const void* p, uint64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}

}  // namespace adacomp
