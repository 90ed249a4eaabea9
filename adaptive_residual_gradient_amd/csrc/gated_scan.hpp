// Gated linear recurrence along the sequence, and its gradients, for gfx950.
//
//   h_t = a_t h_(t-1) + k_t x_t            (forward, t ascending)
//   c_t = a_t (dh_t + c_(t+1))             (backward, t descending; l_t = dh_t + c_(t+1))
//
// Each step is a map s -> a s + b of the carried state, and maps compose: the
// steps of a tile are composed without knowing the state carried into it, and
// every result is then one multiply-add of that state.  A tile is up to 256
// steps (more where a sequence has few channels) of 32 or 64 channels: 512
// threads, each with 4 bytes of channels and 16 (backward 8) consecutive steps whose local
// state and gate product stay in registers between the two halves, so inputs
// are read once and results written once.  The tile's threads join their
// steps through LDS.  The state travels from tile to tile
//   - not at all, where one tile holds the whole sequence (kScanWhole);
//   - through one 8-byte word a channel that each tile leaves for its
//     successor (kScanChain), where there are enough independent chains of
//     tiles to hide that hop;
//   - through a pass of its own over the tiles' compositions (kScanSum,
//     k_scan_carry, kScanCarry), which reads the gates twice, for a few long
//     sequences.
// Sequences of at most kScanShort steps take one thread per 4 bytes of
// channels (k_scan_short).
#pragma once

#include "common.hpp"
#include "elements.hpp"

namespace adacomp {

// Steps a thread holds: backward, their gates, states and gradients are held as
// well, and 16 steps would take more than the 128 registers of four wavefronts a SIMD.
constexpr int scan_thread_steps(bool back) { return back ? 8 : 16; }
constexpr uint32_t kScanShort = 16;     // longest sequence of the short kernels
constexpr uint32_t kScanThreads = 512;  // most threads of a tile
constexpr uint32_t kScanQueues = 64;    // tickets of kScanChain
constexpr uint32_t kScanCountBytes = kScanQueues * 64;   // each on a line of its own
constexpr int kScanWhole = 0, kScanSum = 1, kScanCarry = 2, kScanChain = 3;

struct ScanView {
    void* p;
    uint64_t bs, ts;   // batch and time strides in elements
};

struct ScanArgs {
    ScanView gate, x, h, dh, dgate, dx;
    const float* h0;         // nullable
    const float* dh_last;    // nullable
    float* last;             // h_last or dh0; nullable
    const int32_t* lengths;  // nullable
    uint32_t* tickets;       // kScanChain
    uint64_t* words;         // kScanChain: [chain][tile][slot] {state, 1 once it is there}
    float* agg_a;            // kScanSum, kScanCarry: [chain][tile][slot]
    float* agg_s;            // the same; then the carried states
    uint64_t length;
    uint32_t batch, channels;
    uint32_t lanes, groups, tiles, steps;   // lanes a step, channel groups, tiles a chain, steps a tile
};

// Factors on the state and on the input.  With e = exp(-z), a = 1 / (1 + e)
// and k = e a keep their relative accuracy far from 0; z is held from below
// (NaN stays NaN) where e would overflow: a is below 2e-35 there.
template <typename T, bool SIG>
__device__ __forceinline__ void gates(float z, float& a, float& k) {
    if (!SIG) {
        a = z;
        k = 1.f;
        return;
    }
    constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.69314718f;
    z = __builtin_elementwise_maximum(z, -80.f);
    if (sizeof(T) == 4) z = __builtin_elementwise_minimum(z, 100.f);   // e is 0 from there on
    const float p = z * -kLog2e;
    float e = __builtin_amdgcn_exp2f(p);
    if (sizeof(T) == 4) {
        // the product's rounding, which the exponential turns into a relative error; 16-bit types do
        // without (it is at most 2^-18 where |z| < 64)
        const float r = __builtin_fmaf(z, -kLog2e, -p) + z * -kLog2eLow;
        e = __builtin_fmaf(e * kLn2, r, e);
    }
    const float d = 1.f + e;
    a = __builtin_amdgcn_rcpf(d);
    if (sizeof(T) == 4) a = __builtin_fmaf(a, __builtin_fmaf(-d, a, 1.f), a);
    k = e * a;
}

__device__ __forceinline__ uint64_t scan_steps(const ScanArgs& a, uint32_t b) {
    if (a.lengths == nullptr) return a.length;
    const int32_t n = a.lengths[b];
    return n <= 0 ? 0 : (uint64_t(n) < a.length ? uint64_t(n) : a.length);
}

template <typename T>
__device__ __forceinline__ T* view_at(const ScanView& v, uint32_t b, uint64_t t, uint32_t c) {
    return static_cast<T*>(v.p) + uint64_t(b) * v.bs + t * v.ts + c;
}

// ---- tiles ----

// The state of slot `s` that the predecessor left.  It is there sooner or
// later: a tile waits only for tiles whose tickets were taken before its own,
// so the earliest unfinished one waits for nobody.  The count bounds the wait
// all the same; past it (seconds) the results become NaN.
__device__ __forceinline__ float wait_for_state(const uint64_t* word) {
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        const uint64_t w = __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (w >> 32) return __uint_as_float(uint32_t(w));
        __builtin_amdgcn_s_sleep(1);
    }
    return __builtin_nanf("");
}

// One thread's pointers step through time; where the channels are no multiple
// of the vector the last lanes move back and repeat their neighbours'
// channels, with the same results.
template <typename T, int VW, bool SIG, bool BACK, int MODE>
__global__ __launch_bounds__(kScanThreads, 4) void k_scan_tile(ScanArgs a) {
    typedef typename Packed<T, VW>::V V;
    constexpr int kScanSteps = scan_thread_steps(BACK);
    __shared__ float sa[kScanThreads * VW], ss[kScanThreads * VW];   // [sub-chunk][slot]
    __shared__ uint32_t ticket;
    const uint32_t tid = threadIdx.x, R = a.lanes, slots = R * VW;
    const uint32_t r = tid % R, g = tid / R, G = blockDim.x / R;
    uint32_t chain, k;   // k: the tile along the chain's direction of travel
    if (MODE == kScanChain) {
        const uint32_t q = blockIdx.x % kScanQueues;
        const uint32_t chains = a.batch * a.groups, mine = (chains - q + kScanQueues - 1) / kScanQueues;
        if (tid == 0)
            ticket = __hip_atomic_fetch_add(a.tickets + q * 16, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        const uint32_t n = ticket;
        if (n >= mine * a.tiles) return;
        chain = q + kScanQueues * (n % mine);
        k = n / mine;
    } else {
        chain = blockIdx.x % (a.batch * a.groups);
        k = blockIdx.x / (a.batch * a.groups);
    }
    const uint32_t b = chain / a.groups, group = chain % a.groups;
    if (BACK) k = a.tiles - 1 - k;
    const uint64_t n = scan_steps(a, b);
    const uint64_t t0 = uint64_t(k) * a.steps;
    const uint64_t t1 = t0 + a.steps < a.length ? t0 + a.steps : a.length;
    const uint64_t tend = t1 < n ? t1 : (t0 < n ? n : t0);   // the tile's steps of the sequence end here
    const uint32_t count = uint32_t(tend - t0);
    const uint32_t c = min(group * slots + r * VW, a.channels - VW);

    // zeros past the sequence's end
    if (MODE != kScanSum && tend < t1) {
        const V zero = {};
        for (uint64_t t = tend + g; t < t1; t += G) {
            if (BACK) {
                store_any<VW>(view_at<T>(a.dgate, b, t, c), zero);
                store_any<VW>(view_at<T>(a.dx, b, t, c), zero);
            } else {
                store_any<VW>(view_at<T>(a.h, b, t, c), zero);
            }
        }
    }
    const bool first = BACK ? tend == n : k == 0;    // nothing is carried in but the given state
    const bool last = BACK ? k == 0 : tend == n;     // the carried-out state is the call's
    if (count == 0 && !(n == 0 && k == 0)) return;   // no step of the sequence (an empty one has its tile 0)

    // position i of the direction of travel is step t0 + i, or tend - 1 - i
    const int64_t dir = BACK ? -1 : 1;
    const uint32_t i0 = g * kScanSteps;
    const uint64_t ta = BACK ? tend - 1 - i0 : t0 + i0;   // wraps where the thread has no step
    const int left = int(count) - int(i0);               // steps the thread has
    V zr[kScanSteps], xr[kScanSteps];
    {
        const T* z = view_at<T>(a.gate, b, ta, c);
        const T* x = view_at<T>(BACK ? a.dh : a.x, b, ta, c);
        const int64_t zs = dir * int64_t(a.gate.ts), xs = dir * int64_t(BACK ? a.dh.ts : a.x.ts);
        if (left >= kScanSteps) {
#pragma unroll
            for (int u = 0; u < kScanSteps; ++u) {
                zr[u] = load_any<VW>(z + u * zs);
                xr[u] = load_any<VW>(x + u * xs);
            }
        } else {
#pragma unroll
            for (int u = 0; u < kScanSteps; ++u) {
                zr[u] = xr[u] = V{};
                if (u < left) {
                    zr[u] = load_any<VW>(z + u * zs);
                    xr[u] = load_any<VW>(x + u * xs);
                }
            }
        }
    }
    // what the gradients need besides, requested before the wait
    constexpr bool kGrad = BACK && MODE != kScanSum;
    V hr[kGrad ? kScanSteps : 1], ur[kGrad && SIG ? kScanSteps : 1];
    if (kGrad) {
        const T* h = view_at<T>(a.h, b, ta - 1, c);
        const T* x = SIG ? view_at<T>(a.x, b, ta, c) : nullptr;
#pragma unroll
        for (int u = 0; u < kScanSteps; ++u) {
            hr[kGrad ? u : 0] = V{};
            if (SIG) ur[kGrad && SIG ? u : 0] = V{};
            if (u < left) {
                // step 0 has no earlier state in h
                if (ta != uint64_t(u)) hr[kGrad ? u : 0] = load_any<VW>(h - u * int64_t(a.h.ts));
                if (SIG) ur[kGrad && SIG ? u : 0] = load_any<VW>(x - u * int64_t(a.x.ts));
            }
        }
    }

    // the thread's steps composed: s the state from 0, p the product of gates.  Backward keeps
    // what reaches step t: q = dh + s before it, and p before it.
    FVec<VW> S = 0.f, P = 1.f, sv[kScanSteps], pv[kScanSteps];
#pragma unroll
    for (int u = 0; u < kScanSteps; ++u) {
        const FVec<VW> z = to_float<VW, T>(zr[u]), x = to_float<VW, T>(xr[u]);
#pragma unroll
        for (int v = 0; v < VW; ++v) {
            float f, m;
            gates<T, SIG>(z[v], f, m);
            const bool on = u < left;
            f = on ? f : 1.f;     // steps past the end leave the state as it is
            if (BACK) {
                const float l = x[v] + S[v];   // x is 0 there
                sv[u][v] = l;
                pv[u][v] = P[v];
                S[v] = f * l;
                P[v] *= f;
            } else {
                S[v] = __builtin_fmaf(f, S[v], on ? m * x[v] : 0.f);
                P[v] *= f;
                sv[u][v] = S[v];
                pv[u][v] = P[v];
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VW; ++v) {
        sa[g * slots + r * VW + v] = P[v];
        ss[g * slots + r * VW + v] = S[v];
    }
    __syncthreads();
    if (tid < slots) {
        float A = 1.f, C = 0.f;
#pragma unroll 8
        for (uint32_t i = 0; i < G; ++i) {
            const float f = sa[i * slots + tid];
            C = __builtin_fmaf(f, C, ss[i * slots + tid]);
            A *= f;
        }
        const uint64_t at = (uint64_t(chain) * a.tiles + k) * slots + tid;
        if (MODE == kScanSum) {
            a.agg_a[at] = A;
            a.agg_s[at] = C;
            return;
        }
        const uint32_t sc = min(group * slots + tid / VW * VW, a.channels - VW) + tid % VW;   // the slot's channel
        const uint64_t state = uint64_t(b) * a.channels + sc;
        float s = 0.f;
        if (first) {
            const float* start = BACK ? a.dh_last : a.h0;
            if (start) s = start[state];
        } else if (MODE == kScanCarry) {
            s = a.agg_s[at];
        } else if (MODE == kScanChain) {
            s = wait_for_state(a.words + (BACK ? at + slots : at - slots));
        }
        const float out = __builtin_fmaf(A, s, C);
        if (MODE == kScanChain && !last)
            __hip_atomic_store(a.words + at, (uint64_t(1) << 32) | __float_as_uint(out), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        if (last && a.last) a.last[state] = count ? out : s;
        // the state each sub-chunk starts from takes the place of its product
#pragma unroll 8
        for (uint32_t i = 0; i < G; ++i) {
            const float f = sa[i * slots + tid];
            sa[i * slots + tid] = s;
            s = __builtin_fmaf(f, s, ss[i * slots + tid]);
        }
    }
    if (MODE == kScanSum) return;
    __syncthreads();
    FVec<VW> s;
#pragma unroll
    for (int v = 0; v < VW; ++v) s[v] = sa[g * slots + r * VW + v];
    if (!BACK) {
        T* h = view_at<T>(a.h, b, ta, c);
#pragma unroll
        for (int u = 0; u < kScanSteps; ++u) {
            FVec<VW> o;
#pragma unroll
            for (int v = 0; v < VW; ++v) o[v] = __builtin_fmaf(pv[u][v], s[v], sv[u][v]);
            if (u < left) store_any<VW>(h + u * a.h.ts, from_float<T, VW>(o));
        }
    } else {
        T* dg = view_at<T>(a.dgate, b, ta, c);
        T* dx = view_at<T>(a.dx, b, ta, c);
#pragma unroll
        for (int u = 0; u < kScanSteps; ++u) {
            if (u >= left) continue;
            FVec<VW> z = to_float<VW, T>(zr[u]), before = to_float<VW, T>(hr[kGrad ? u : 0]), og, ox;
            if (ta == uint64_t(u)) {
                before = 0.f;
                if (a.h0) before = load_any<VW>(a.h0 + uint64_t(b) * a.channels + c);
            }
            if (SIG) before -= to_float<VW, T>(ur[kGrad && SIG ? u : 0]);
#pragma unroll
            for (int v = 0; v < VW; ++v) {
                float f, m;
                gates<T, SIG>(z[v], f, m);
                const float l = __builtin_fmaf(pv[u][v], s[v], sv[u][v]);
                og[v] = SIG ? l * before[v] * f * m : l * before[v];
                ox[v] = l * m;
            }
            store_any<VW>(dg - u * int64_t(a.dgate.ts), from_float<T, VW>(og));
            store_any<VW>(dx - u * int64_t(a.dx.ts), from_float<T, VW>(ox));
        }
    }
}

// Clears the tickets and words of kScanChain.
__global__ __launch_bounds__(256) void k_scan_clear(uint4* p, uint64_t n) {
    for (uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += uint64_t(gridDim.x) * 256)
        p[i] = uint4{0, 0, 0, 0};
}

// agg_s becomes the state carried into each tile: a workgroup takes one chain,
// 1024 / slots sections of its tiles at once, joined through LDS.
template <bool BACK>
__global__ __launch_bounds__(1024) void k_scan_carry(ScanArgs a, uint32_t vw) {
    __shared__ float sa[1024], ss[1024];
    const uint32_t slots = a.lanes * vw, slot = threadIdx.x % slots, part = threadIdx.x / slots;
    const uint32_t parts = blockDim.x / slots, chain = blockIdx.x, b = chain / a.groups;
    const uint32_t tiles = uint32_t((scan_steps(a, b) + a.steps - 1) / a.steps);   // those with steps
    const uint32_t per = (tiles + parts - 1) / parts;
    const uint32_t n0 = min(part * per, tiles), n1 = min(n0 + per, tiles);
    const uint64_t base = uint64_t(chain) * a.tiles * slots + slot;
    auto at = [&](uint32_t n) { return base + uint64_t(BACK ? tiles - 1 - n : n) * slots; };
    float A = 1.f, S = 0.f;
#pragma unroll 8
    for (uint32_t n = n0; n < n1; ++n) {
        const float f = a.agg_a[at(n)];
        S = __builtin_fmaf(f, S, a.agg_s[at(n)]);
        A *= f;
    }
    sa[threadIdx.x] = A;
    ss[threadIdx.x] = S;
    __syncthreads();
    const uint32_t c = min((chain % a.groups) * slots + slot / vw * vw, a.channels - vw) + slot % vw;
    const float* start = BACK ? a.dh_last : a.h0;
    float s = start ? start[uint64_t(b) * a.channels + c] : 0.f;
    for (uint32_t i = 0; i < part; ++i) s = __builtin_fmaf(sa[i * slots + slot], s, ss[i * slots + slot]);
#pragma unroll 8
    for (uint32_t n = n0; n < n1; ++n) {
        const float f = a.agg_a[at(n)], d = a.agg_s[at(n)];
        a.agg_s[at(n)] = s;
        s = __builtin_fmaf(f, s, d);
    }
}

// ---- short sequences ----

template <typename T, int VW, bool SIG, bool BACK>
__global__ __launch_bounds__(256) void k_scan_short(ScanArgs a) {
    const uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x;
    const uint32_t b = uint32_t(i / a.lanes);
    if (b >= a.batch) return;
    const uint32_t c = min(uint32_t(i % a.lanes) * VW, a.channels - VW);
    const uint32_t n = uint32_t(scan_steps(a, b)), T1 = uint32_t(a.length);
    const uint64_t state = uint64_t(b) * a.channels + c;
    const float* start = BACK ? a.dh_last : a.h0;
    FVec<VW> s = 0.f;
    if (start) s = load_any<VW>(start + state);
    const typename Packed<T, VW>::V zero = {};
    if (!BACK) {
#pragma unroll 4
        for (uint32_t t = 0; t < n; ++t) {
            const FVec<VW> z = to_float<VW, T>(load_any<VW>(view_at<T>(a.gate, b, t, c)));
            const FVec<VW> x = to_float<VW, T>(load_any<VW>(view_at<T>(a.x, b, t, c)));
#pragma unroll
            for (int v = 0; v < VW; ++v) {
                float f, m;
                gates<T, SIG>(z[v], f, m);
                s[v] = __builtin_fmaf(f, s[v], m * x[v]);
            }
            store_any<VW>(view_at<T>(a.h, b, t, c), from_float<T, VW>(s));
        }
        for (uint32_t t = n; t < T1; ++t) store_any<VW>(view_at<T>(a.h, b, t, c), zero);
    } else {
        for (uint32_t t = n; t < T1; ++t) {
            store_any<VW>(view_at<T>(a.dgate, b, t, c), zero);
            store_any<VW>(view_at<T>(a.dx, b, t, c), zero);
        }
#pragma unroll 4
        for (uint32_t i1 = 0; i1 < n; ++i1) {
            const uint32_t t = n - 1 - i1;
            const FVec<VW> z = to_float<VW, T>(load_any<VW>(view_at<T>(a.gate, b, t, c)));
            const FVec<VW> d = to_float<VW, T>(load_any<VW>(view_at<T>(a.dh, b, t, c)));
            FVec<VW> before = 0.f, og, ox;
            if (t > 0) before = to_float<VW, T>(load_any<VW>(view_at<T>(a.h, b, t - 1, c)));
            else if (a.h0) before = load_any<VW>(a.h0 + state);
            if (SIG) before -= to_float<VW, T>(load_any<VW>(view_at<T>(a.x, b, t, c)));
#pragma unroll
            for (int v = 0; v < VW; ++v) {
                float f, m;
                gates<T, SIG>(z[v], f, m);
                const float l = d[v] + s[v];
                og[v] = SIG ? l * before[v] * f * m : l * before[v];
                ox[v] = l * m;
                s[v] = f * l;
            }
            store_any<VW>(view_at<T>(a.dgate, b, t, c), from_float<T, VW>(og));
            store_any<VW>(view_at<T>(a.dx, b, t, c), from_float<T, VW>(ox));
        }
    }
    if (a.last) store_any<VW>(a.last + state, s);
}

}  // namespace adacomp
