// What the operators along a sequence share: views, lengths and the logistic
// functions.
#pragma once

#include "elements.hpp"

namespace adacomp {

struct ScanView {
    void* p;
    uint64_t bs, ts;   // batch and time strides in elements
};

template <typename T>
__device__ __forceinline__ T* view_at(const ScanView& v, uint32_t b, uint64_t t, uint32_t c) {
    return static_cast<T*>(v.p) + uint64_t(b) * v.bs + t * v.ts + c;
}

// Steps of one sequence.
__device__ __forceinline__ uint64_t steps_of(const int32_t* lengths, uint64_t length, uint32_t b) {
    if (lengths == nullptr) return length;
    const int32_t n = lengths[b];
    return n <= 0 ? 0 : (uint64_t(n) < length ? uint64_t(n) : length);
}

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147182f, kLn2Low = -1.90465421e-9f;   // ln 2 = the sum of both

// exp(-z), to 2 units in the last place or so, for z that neither overflow nor leave nothing.
__device__ __forceinline__ float exp_of_minus(float z) {
    const float p = z * -kLog2e;
    const float e = __builtin_amdgcn_exp2f(p);
    // what the rounding of p leaves out, -z - p ln 2: without it e would be off by 2^-24 |z|
    return __builtin_fmaf(e, __builtin_fmaf(p, -kLn2Low, __builtin_fmaf(p, -kLn2, -z)), e);
}

}  // namespace adacomp
