// Element types of the training-step operators: vectors of float32, bfloat16
// and half in memory, float32 in registers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace adacomp {

typedef __bf16 bf16;
typedef _Float16 f16;

template <int N>
using FVec = float __attribute__((ext_vector_type(N)));

// Most bytes of a call's inputs (or output) that are worth a place in the 256 MB cache in front of the
// memory: beside them it holds what the calls around this one touch.
constexpr uint64_t kKeepBytes = 96u << 20;

// N elements at any address aligned to one element: gfx950 reads and writes
// 16 bytes from any address, so rows of odd widths keep wide accesses (a row
// that starts inside a 16-byte granule costs one more cache line, not a loop
// over its elements).
template <typename T, int N>
struct Packed {
    typedef T V __attribute__((ext_vector_type(N)));
    typedef V Any __attribute__((aligned(sizeof(T))));
};

template <int N, typename T>
__device__ __forceinline__ typename Packed<T, N>::V load_any(const T* p) {
    return *reinterpret_cast<const typename Packed<T, N>::Any*>(p);
}
template <int N, typename T>
__device__ __forceinline__ void store_any(T* p, typename Packed<T, N>::V v) {
    *reinterpret_cast<typename Packed<T, N>::Any*>(p) = v;
}
// The same, of data that is touched once.
template <int N, typename T>
__device__ __forceinline__ typename Packed<T, N>::V stream_load(const T* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const typename Packed<T, N>::Any*>(p));
}
template <int N, typename T>
__device__ __forceinline__ void stream_store(T* p, typename Packed<T, N>::V v) {
    __builtin_nontemporal_store(v, reinterpret_cast<typename Packed<T, N>::Any*>(p));
}
// Either, by NT (non-temporal).
template <int N, bool NT, typename T>
__device__ __forceinline__ typename Packed<T, N>::V load_hint(const T* p) {
    return NT ? stream_load<N>(p) : load_any<N>(p);
}
template <int N, bool NT, typename T>
__device__ __forceinline__ void store_hint(T* p, typename Packed<T, N>::V v) {
    if (NT) stream_store<N>(p, v);
    else store_any<N>(p, v);
}
template <int N, typename T>
__device__ __forceinline__ FVec<N> to_float(typename Packed<T, N>::V v) {
    return __builtin_convertvector(v, FVec<N>);
}
// rounded to nearest, ties to even
template <typename T, int N>
__device__ __forceinline__ typename Packed<T, N>::V from_float(FVec<N> v) {
    return __builtin_convertvector(v, typename Packed<T, N>::V);
}

}  // namespace adacomp
