// Host-side argument checks shared by the C ABI's translation units.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/adacomp.h"
#include "ranges.hpp"

namespace adacomp {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int launch_status() {
    return hipGetLastError() == hipSuccess ? ADACOMP_OK : ADACOMP_ERR_HIP;
}

}  // namespace adacomp
