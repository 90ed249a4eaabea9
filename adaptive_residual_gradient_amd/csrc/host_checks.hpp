// Host-side argument checks shared by the C ABI's translation units.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/adacomp.h"

namespace adacomp {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
    uintptr_t lo, hi;
};
inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }
inline Range range_of(const void* p, uint64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}

inline int launch_status() {
    return hipGetLastError() == hipSuccess ? ADACOMP_OK : ADACOMP_ERR_HIP;
}

}  // namespace adacomp
