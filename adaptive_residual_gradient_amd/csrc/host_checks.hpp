// Host-side argument checks shared by the C ABI's translation units.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/adacomp.h"
#include "ranges.hpp"

namespace adacomp {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool aligned_to(const void* p, uint64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// Bytes of an element, 0 for what is no element type.
inline uint64_t type_size(int type) {
    return type == ADACOMP_FLOAT ? 4 : type == ADACOMP_BFLOAT || type == ADACOMP_HALF ? 2 : 0;
}
// No output may share a byte with any other buffer; the first `nout` ranges are outputs.
inline bool outputs_clash(const Range* r, int nout, int n) {
    for (int i = 0; i < nout; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlaps(r[i], r[j])) return true;
    return false;
}

inline int launch_status() {
    return hipGetLastError() == hipSuccess ? ADACOMP_OK : ADACOMP_ERR_HIP;
}

}  // namespace adacomp
