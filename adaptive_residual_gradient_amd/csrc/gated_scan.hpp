// Gated linear recurrence along the sequence, and its gradients, for gfx950.
//
//   h_t = a_t h_(t-1) + k_t x_t            (forward, t ascending)
//   c_t = a_t (dh_t + c_(t+1))             (backward, t descending; l_t = dh_t + c_(t+1))
//
// Each is a chain of maps s -> A s + S, and maps compose: a sequence is cut
// into chunks, a first kernel forms each chunk's (A, S), a second carries the
// state through them, a third steps through the chunks from their carried
// states and writes the results.  Sequences of one chunk take the third
// kernel alone.
#pragma once

#include "common.hpp"
#include "elements.hpp"

namespace adacomp {

struct ScanView {
    void* p;
    uint64_t bs, ts;   // batch and time strides in elements
};

struct ScanArgs {
    ScanView gate, x, h, dh, dgate, dx;
    const float* h0;        // nullable
    const float* dh_last;   // nullable
    float* last;            // h_last or dh0; nullable
    const int32_t* lengths; // nullable
    float* agg_a;           // [batch][chunks][channels]
    float* agg_s;           // the same; then the carried states
    uint64_t length;
    uint32_t batch, channels, lanes, chunks, chunk;   // lanes per step; steps per chunk
};

constexpr int kScanBatch = 8;   // steps whose loads are requested together

// Factors on the state and on the input.  exp(-|z|) <= 1, so neither
// overflows and both keep their relative accuracy far from 0.  The hardware's
// exponential and reciprocal serve 16-bit types (their error, at most 2^-18 where
// |z| < 64, is far below those types' steps); float32 takes the full functions.
template <typename T, bool SIG>
__device__ __forceinline__ void gates(float z, float& a, float& k) {
    if (!SIG) {
        a = z;
        k = 1.f;
        return;
    }
    const bool full = sizeof(T) == 4;
    const float e = full ? expf(-fabsf(z)) : __builtin_amdgcn_exp2f(fabsf(z) * -1.44269504f);
    const float big = full ? 1.f / (1.f + e) : __builtin_amdgcn_rcpf(1.f + e);
    const float small = e * big;
    a = z >= 0.f ? big : small;
    k = z >= 0.f ? small : big;
}

template <typename T, int VW>
__device__ __forceinline__ FVec<VW> view_load(const ScanView& v, uint32_t b, uint64_t t, uint32_t c) {
    return to_float<VW, T>(load_any<VW>(static_cast<const T*>(v.p) + uint64_t(b) * v.bs + t * v.ts + c));
}
template <typename T, int VW>
__device__ __forceinline__ void view_store(const ScanView& v, uint32_t b, uint64_t t, uint32_t c, FVec<VW> x) {
    store_any<VW>(static_cast<T*>(v.p) + uint64_t(b) * v.bs + t * v.ts + c, from_float<T, VW>(x));
}

__device__ __forceinline__ uint64_t scan_steps(const ScanArgs& a, uint32_t b) {
    if (a.lengths == nullptr) return a.length;
    const int32_t n = a.lengths[b];
    return n <= 0 ? 0 : (uint64_t(n) < a.length ? uint64_t(n) : a.length);
}

// The thread's sequence, chunk and first channel.  Where the channels are no
// multiple of the vector the last lane moves back and repeats some of its
// neighbour's channels, with the same results.
struct ScanPlace {
    uint32_t b, k, c;
    uint64_t t0, t1, steps;   // the chunk's steps; the sequence's
    bool live;
};
template <int VW>
__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& a) {
    ScanPlace p;
    const uint64_t i = uint64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    const uint32_t lane = uint32_t(i % a.lanes);
    const uint64_t r = i / a.lanes;
    p.k = uint32_t(r % a.chunks);
    const uint64_t b = r / a.chunks;
    p.live = b < a.batch;
    p.b = p.live ? uint32_t(b) : 0;
    const uint32_t c = lane * VW;
    p.c = c + VW <= a.channels ? c : a.channels - VW;
    p.t0 = uint64_t(p.k) * a.chunk;
    const uint64_t t1 = p.t0 + a.chunk;
    p.t1 = t1 < a.length ? t1 : a.length;
    p.steps = p.live ? scan_steps(a, p.b) : 0;
    return p;
}

template <typename T, int VW, bool SIG, bool BACK>
__global__ __launch_bounds__(256) void k_scan_sum(ScanArgs a) {
    const ScanPlace p = scan_place<VW>(a);
    if (!p.live) return;
    const uint64_t end = p.t1 < p.steps ? p.t1 : p.steps;
    FVec<VW> A = 1.f, S = 0.f;
    for (uint64_t i = p.t0; i < end; i += kScanBatch) {
        FVec<VW> z[kScanBatch], x[kScanBatch];
#pragma unroll
        for (int u = 0; u < kScanBatch; ++u) {
            const uint64_t t = BACK ? p.t0 + (end - 1 - (i + u)) : i + u;
            if (i + u < end) {
                z[u] = view_load<T, VW>(a.gate, p.b, t, p.c);
                x[u] = view_load<T, VW>(BACK ? a.dh : a.x, p.b, t, p.c);
            }
        }
#pragma unroll
        for (int u = 0; u < kScanBatch; ++u) {
            if (i + u >= end) break;
#pragma unroll
            for (int v = 0; v < VW; ++v) {
                float f, k;
                gates<T, SIG>(z[u][v], f, k);
                S[v] = BACK ? f * (x[u][v] + S[v]) : __builtin_fmaf(f, S[v], k * x[u][v]);
                A[v] *= f;
            }
        }
    }
    const uint64_t at = (uint64_t(p.b) * a.chunks + p.k) * a.channels + p.c;
    store_any<VW>(a.agg_a + at, A);
    store_any<VW>(a.agg_s + at, S);
}

// agg_s becomes the state carried into each chunk.
template <bool BACK>
__global__ __launch_bounds__(64) void k_scan_carry(ScanArgs a) {
    const uint64_t i = uint64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    const uint64_t b = i / a.channels;
    if (b >= a.batch) return;
    const uint32_t c = uint32_t(i % a.channels);
    const float* start = BACK ? a.dh_last : a.h0;
    float s = start ? start[i] : 0.f;
    for (uint32_t n = 0; n < a.chunks; n += kScanBatch) {
        float A[kScanBatch], S[kScanBatch];
#pragma unroll
        for (int u = 0; u < kScanBatch; ++u) {
            if (n + u >= a.chunks) break;
            const uint32_t k = BACK ? a.chunks - 1 - (n + u) : n + u;
            const uint64_t at = (b * a.chunks + k) * a.channels + c;
            A[u] = a.agg_a[at];
            S[u] = a.agg_s[at];
        }
#pragma unroll
        for (int u = 0; u < kScanBatch; ++u) {
            if (n + u >= a.chunks) break;
            const uint32_t k = BACK ? a.chunks - 1 - (n + u) : n + u;
            a.agg_s[(b * a.chunks + k) * a.channels + c] = s;
            s = __builtin_fmaf(A[u], s, S[u]);
        }
    }
}

// The state carried into the thread's chunk.
template <int VW, bool BACK>
__device__ __forceinline__ FVec<VW> scan_start(const ScanArgs& a, const ScanPlace& p) {
    if (a.chunks > 1) return load_any<VW>(a.agg_s + (uint64_t(p.b) * a.chunks + p.k) * a.channels + p.c);
    const float* start = BACK ? a.dh_last : a.h0;
    FVec<VW> s = 0.f;
    if (start) s = load_any<VW>(start + uint64_t(p.b) * a.channels + p.c);
    return s;
}

template <typename T, int VW, bool SIG>
__global__ __launch_bounds__(256) void k_scan_forward(ScanArgs a) {
    const ScanPlace p = scan_place<VW>(a);
    if (!p.live) return;
    const uint64_t end = p.t1 < p.steps ? p.t1 : p.steps;
    FVec<VW> s = scan_start<VW, false>(a, p);
    for (uint64_t i = p.t0; i < end; i += kScanBatch) {
        FVec<VW> z[kScanBatch], x[kScanBatch];
#pragma unroll
        for (int u = 0; u < kScanBatch; ++u)
            if (i + u < end) {
                z[u] = view_load<T, VW>(a.gate, p.b, i + u, p.c);
                x[u] = view_load<T, VW>(a.x, p.b, i + u, p.c);
            }
#pragma unroll
        for (int u = 0; u < kScanBatch; ++u) {
            if (i + u >= end) break;
#pragma unroll
            for (int v = 0; v < VW; ++v) {
                float f, k;
                gates<T, SIG>(z[u][v], f, k);
                s[v] = __builtin_fmaf(f, s[v], k * x[u][v]);
            }
            view_store<T, VW>(a.h, p.b, i + u, p.c, s);
        }
    }
    const FVec<VW> zero = 0.f;
    for (uint64_t t = p.t0 > end ? p.t0 : end; t < p.t1; ++t) view_store<T, VW>(a.h, p.b, t, p.c, zero);
    if (a.last && p.k == a.chunks - 1) store_any<VW>(a.last + uint64_t(p.b) * a.channels + p.c, s);
}

template <typename T, int VW, bool SIG>
__global__ __launch_bounds__(256) void k_scan_backward(ScanArgs a) {
    const ScanPlace p = scan_place<VW>(a);
    if (!p.live) return;
    const uint64_t end = p.t1 < p.steps ? p.t1 : p.steps;
    FVec<VW> s = scan_start<VW, true>(a, p);
    const FVec<VW> zero = 0.f;
    for (uint64_t t = p.t0 > end ? p.t0 : end; t < p.t1; ++t) {
        view_store<T, VW>(a.dgate, p.b, t, p.c, zero);
        view_store<T, VW>(a.dx, p.b, t, p.c, zero);
    }
    for (uint64_t i = p.t0; i < end; i += kScanBatch) {
        FVec<VW> z[kScanBatch], x[kScanBatch], d[kScanBatch], before[kScanBatch];
#pragma unroll
        for (int u = 0; u < kScanBatch; ++u)
            if (i + u < end) {
                const uint64_t t = p.t0 + (end - 1 - (i + u));
                z[u] = view_load<T, VW>(a.gate, p.b, t, p.c);
                d[u] = view_load<T, VW>(a.dh, p.b, t, p.c);
                if (SIG) x[u] = view_load<T, VW>(a.x, p.b, t, p.c);
                before[u] = 0.f;
                if (t > 0) before[u] = view_load<T, VW>(a.h, p.b, t - 1, p.c);
                else if (a.h0) before[u] = load_any<VW>(a.h0 + uint64_t(p.b) * a.channels + p.c);
            }
#pragma unroll
        for (int u = 0; u < kScanBatch; ++u) {
            if (i + u >= end) break;
            const uint64_t t = p.t0 + (end - 1 - (i + u));
            FVec<VW> dg, dx;
#pragma unroll
            for (int v = 0; v < VW; ++v) {
                float f, k;
                gates<T, SIG>(z[u][v], f, k);
                const float l = d[u][v] + s[v];
                dg[v] = SIG ? l * (before[u][v] - x[u][v]) * f * k : l * before[u][v];
                dx[v] = l * k;
                s[v] = f * l;
            }
            view_store<T, VW>(a.dgate, p.b, t, p.c, dg);
            view_store<T, VW>(a.dx, p.b, t, p.c, dx);
        }
    }
    if (a.last && p.k == 0) store_any<VW>(a.last + uint64_t(p.b) * a.channels + p.c, s);
}

}  // namespace adacomp
