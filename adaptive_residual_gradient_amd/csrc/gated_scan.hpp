// Gated linear recurrence along the sequence, and its gradients, for gfx950.
//
//   h_t = a_t h_(t-1) + k_t x_t            (forward, t ascending)
//   c_t = a_t (dh_t + c_(t+1))             (backward, t descending; l_t = dh_t + c_(t+1))
//
// Each step is a map s -> a s + b of the carried state, and maps compose: the
// steps of a tile are composed without knowing the state carried into it.  Once
// it is known every forward result is one multiply-add of it, and the backward
// recurrence runs again.  A tile is at most 128 steps (64 backward with the
// sigmoid; more where a sequence has few channels) of 64 float32 or 128 16-bit
// channels: 512 threads, each with 4 bytes of channels and up to 16 consecutive
// steps that stay in registers between the two halves, so inputs are read once
// and results written once.  The tile's threads join their steps through LDS.
// The state travels from tile to tile
//   - not at all, where one tile holds the whole sequence (kScanAlone);
//   - through one word a channel that each tile leaves for its successor
//     (kScanChain), where there are enough independent chains of tiles to hide
//     that hop of about 1.3 us;
//   - of few long chains, through the compositions of the tiles and of groups of
//     tiles before, many at a time (kScanBack).
// Sequences of at most kScanShort steps take one thread per 4 bytes of
// channels (k_scan_short).
//
// Memory bounds it: 8 x 4096 x 2048 bf16 takes 82.5 us (4.9 TB/s), the gradients
// of 1 x 65536 x 256 float32 69.4 us (4.8 TB/s).  The accesses of a tile alone, rows
// of 256 bytes in 128 steps, run at 6.0 TB/s.
#pragma once

#include "common.hpp"
#include "elements.hpp"

namespace adacomp {

// Steps a thread holds.  Backward with the sigmoid 8: 16 of them take more registers than there are (8 x
// 4096 x 2048 bf16 238 us against 145), or one workgroup a CU fewer (1 x 65536 x 256 f32 83 against 95, but
// 8 x 4096 x 2048 f32 296 against 278).  The others 16, for fewer tiles on the way of the state (backward without the sigmoid, 1 x 65536 x 256 f32
// 71 us against 86 with 8, though 8 x 4096 x 2048 f32 270 against 236).
constexpr int scan_thread_steps(bool sigmoid, bool back) { return sigmoid && back ? 8 : 16; }
constexpr uint32_t kScanShort = 16;     // longest sequence of the short kernels
constexpr uint32_t kScanThreads = 512;  // most threads of a tile
constexpr uint32_t kScanQueues = 64;    // most ticket counters
constexpr uint32_t kScanCountBytes = kScanQueues * 64;   // each on a line of its own
constexpr int kScanAlone = 0, kScanChain = 1, kScanBack = 2;
// Words that a thread of kScanBack looks at together, of tiles and of groups of tiles each.  8 tiles' forward
// takes 114 registers instead of 77 (1 x 20000 x 1000 f32 58.5 us and 53.1), or more than there are
// (4 x 8000 x 512 bf16 36.8 and 27.5).
constexpr uint32_t kScanWindow = 4;

// Accesses: non-temporal; non-temporal results and inputs of at most kKeepBytes, which the call before
// has just written, through the cache (8 x 2048 x 1024 bf16, again and again on one set of buffers, 23.1 us
// and 27.1 past it; its gradient's 134 MB, past the bound, 43.6 us and 36.2 through the cache); all
// through the cache.
constexpr int kScanStream = 0, kScanKeepIn = 1, kScanCached = 2;

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
    uint32_t* tickets;       // one counter a queue, 64 bytes apart
    void* words;             // [chain][tile][slot]: uint32_t (kScanChain) or uint64_t (kScanBack)
    void* group_words;       // kScanBack: uint64_t [chain][group of tiles][slot]
    uint64_t length;
    uint32_t batch, channels;
    uint32_t lanes, groups, tiles, steps, queues;   // lanes a step, channel groups, tiles a chain, steps a tile
    uint32_t span, spans, most;                     // kScanBack: tiles a group, groups a chain, groups looked at
};

// Factors on the state and on the input, each within 8 roundings of float32 whatever the type: the states
// that they form are float32.  With e = exp(-z), a = 1 / (1 + e) and k = e a keep their relative accuracy
// far from 0.  z is held (NaN stays NaN) from below where e would overflow: a stays at 1.6e-38 from there
// on; and from above where e is 0.
template <typename T, bool SIG>
__device__ __forceinline__ void gates(float z, float& a, float& k) {
    if (!SIG) {
        a = z;
        k = 1.f;
        return;
    }
    constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147182f, kLn2Low = -1.90465421e-9f;   // ln 2 = the sum of both
    z = __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -87.f), 100.f);
    const float p = z * -kLog2e;
    float e = __builtin_amdgcn_exp2f(p);
    // what the rounding of p leaves out, -z - p ln 2: without it e would be off by 2^-24 |z|
    e = __builtin_fmaf(e, __builtin_fmaf(p, -kLn2Low, __builtin_fmaf(p, -kLn2, -z)), e);
    const float d = 1.f + e;
    a = __builtin_amdgcn_rcpf(d);
    // the hardware's reciprocal is off by one unit in the last place, which float32 calls take out too
    // (8 x 4096 x 2048 bf16 85.6 us with it, 84.6 without)
    if (sizeof(T) == 4) a = __builtin_fmaf(a, __builtin_fmaf(-d, a, 1.f), a);
    k = e * a;
}

// Product of two gate products.  Of gates that are not 0 it never becomes 0, so that an infinite state
// stays infinite under them (0 times infinity is NaN); to any other state the smallest number adds no more
// than that product's own rounding may.  With the sigmoid no gate is 0 or below.
template <bool SIG>
__device__ __forceinline__ float gate_product(float p, float f) {
    const float least = __uint_as_float(1u), q = p * f;
    if (SIG) return __builtin_elementwise_maximum(q, least);
    const float size = __builtin_elementwise_minimum(__builtin_elementwise_minimum(fabsf(p), fabsf(f)), least);
    return copysignf(__builtin_elementwise_maximum(fabsf(q), size), q);
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

// A state on its way to the next tile: its bits, of which this NaN's stand for
// "not there yet".
constexpr uint32_t kScanEmpty = 0xFFFFFFFFu;
__device__ __forceinline__ void leave_state(uint32_t* word, float s) {
    const uint32_t bits = __float_as_uint(s);
    __hip_atomic_store(word, bits == kScanEmpty ? 0x7FC00000u : bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The state that the predecessor leaves.  It is there sooner or later: a tile
// waits only for tiles whose tickets were taken before its own, so the earliest
// unfinished one waits for nobody.  The count bounds the wait all the same;
// past it (seconds) the results become NaN.
__device__ __forceinline__ float wait_for_state(const uint32_t* word) {
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        const uint32_t w = __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (w != kScanEmpty) return __uint_as_float(w);
        __builtin_amdgcn_s_sleep(1);
    }
    return __builtin_nanf("");
}

// kScanBack: `span` tiles that follow each other on the way of the state make a group.  A tile looks at
// the words of its own group's tiles and of the group's before, which those tiles leave as soon as they
// have composed their steps, and at the groups' words before that; a group's word is left by the tile
// behind it.  A word is a composition (two floats), or a known state where none is needed: the first
// tile's, and that of every `most`-th group, at which the look ends.  So the state carried into a tile
// is always joined from the same words in the same order, whichever of them are there first.
constexpr uint32_t kScanKnown = 0xFFFFFFFEu;   // the high half of a word that holds a state
__device__ __forceinline__ void leave_pair(uint64_t* word, uint32_t high, float s) {
    __hip_atomic_store(word, uint64_t(high) << 32 | __float_as_uint(s), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t composed(float a) {
    const uint32_t bits = __float_as_uint(a);
    return bits >= kScanKnown ? 0x7FC00000u : bits;
}

// The n words (at most subs * WINDOW) before a place, word `d` of which (1 the nearest) is at
// base + d * stride.  All threads look: the subs of a slot take WINDOW words each, nearest first, and
// join their maps through LDS.
template <bool SIG>
struct LookBack {
    static constexpr uint32_t WINDOW = kScanWindow;
    const uint64_t* base;
    int64_t stride;
    uint32_t n, d0;
    uint64_t w[WINDOW];
    __device__ __forceinline__ uint64_t word(uint32_t d) const {
        return __hip_atomic_load(base + int64_t(d) * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ LookBack(const uint64_t* words, int64_t step, uint32_t count, uint32_t slots)
        : base(words + threadIdx.x % slots), stride(step), n(count), d0(threadIdx.x / slots * WINDOW + 1) {
        if (n > 0) request();
    }
    __device__ __forceinline__ void request() {
#pragma unroll
        for (uint32_t u = 0; u < WINDOW; ++u) w[u] = word(min(d0 + u, n));
    }
    // Whether a word was not there yet at the last request.
    __device__ __forceinline__ bool missing() const {
        bool any = false;
#pragma unroll
        for (uint32_t u = 0; u < WINDOW; ++u) any |= uint32_t(w[u] >> 32) == kScanEmpty;
        return any;
    }
    // Waits for the words.  Their map is A s + S; where the farthest is a known state S is the state itself,
    // and A means nothing.  For the first `slots` threads.
    __device__ __forceinline__ void join(uint32_t slots, float (&la)[kScanThreads], float (&ls)[kScanThreads], float& A,
                                         float& S) {
        const uint32_t tid = threadIdx.x;
        A = 1.f;
        S = 0.f;
        if (n == 0) return;
        for (uint32_t i = 0; missing() && i < (1u << 22); ++i) {   // past the bound a NaN's bits
            __builtin_amdgcn_s_sleep(1);
            request();   // all together: one by one each would wait a load's time again
        }
        float a = 1.f, s = 0.f;
#pragma unroll
        for (uint32_t u = 0; u < WINDOW; ++u) {
            if (d0 + u > n) continue;
            s = __builtin_fmaf(a, __uint_as_float(uint32_t(w[u])), s);
            a = gate_product<SIG>(a, __uint_as_float(uint32_t(w[u] >> 32)));
        }
        la[tid] = a;
        ls[tid] = s;
        __syncthreads();
        if (tid >= slots) return;
        for (uint32_t j = 0; j < (n + WINDOW - 1) / WINDOW; ++j) {
            S = __builtin_fmaf(A, ls[j * slots + tid], S);
            A = gate_product<SIG>(A, la[j * slots + tid]);
        }
    }
};

// Workgroups go to the 8 chiplets in turn.  Of 64 consecutive ones each
// chiplet's eight take eight neighbouring chains: neighbouring channels of the
// same rows.
__device__ __forceinline__ uint32_t chiplet_order(uint32_t i) { return (i & ~63u) | (i & 7u) << 3 | (i >> 3 & 7u); }

// A tile's place.
struct ScanTile {
    uint32_t chain, b, k, slot0;      // slot0: the channel of the group's first slot
    uint64_t tend;                    // the tile's steps of the sequence end here
    uint32_t count;                   // and are so many
    uint32_t before;                  // tiles with steps before it in the direction of travel
    bool first, last;                 // first: nothing is carried in but the given state;
                                      // last: the state carried out is the call's
};

// One tile.  FULL: every thread has all its steps.  Else those past the
// sequence's end read the last one again and leave the state as it is, so that
// no load stands under a condition (one that does is waited for at once).
// Where the channels are no multiple of the vector the last lanes move back and
// repeat their neighbours' channels, with the same results.
template <typename T, int VW, bool SIG, bool BACK, int MODE, int ACCESS, bool FULL>
__device__ __forceinline__ void scan_tile(const ScanArgs& a, const ScanTile& tile, float* sa, float* ss) {
    typedef typename Packed<T, VW>::V V;
    constexpr int N = scan_thread_steps(SIG, BACK);
    const uint32_t tid = threadIdx.x, R = a.lanes, slots = R * VW;
    const uint32_t r = tid % R, g = tid / R, G = blockDim.x / R, b = tile.b;
    const uint32_t c = min(tile.slot0 + r * VW, a.channels - VW);
    // position i of the direction of travel is step t0 + i, or tend - 1 - i
    const uint32_t i0 = g * N;
    const int left = FULL ? N : int(tile.count) - int(i0);   // steps the thread has
    const uint32_t at = FULL ? i0 : min(i0, tile.count - 1);
    const uint64_t ta = BACK ? tile.tend - 1 - at : tile.tend - tile.count + at;
    auto walk = [&](const ScanView& view, uint64_t t, V(&v)[N]) {
        const T* p = view_at<T>(view, b, t, c);
        const int64_t step = BACK ? -int64_t(view.ts) : int64_t(view.ts);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            v[u] = load_hint<VW, ACCESS == kScanStream>(p);
            if (u + 1 < N) p += FULL || u + 1 < left ? step : 0;
        }
    };
    V zr[N], xr[N], hr[N], ur[N];
    walk(a.gate, ta, zr);
    walk(BACK ? a.dh : a.x, ta, xr);
    FVec<VW> h0 = 0.f;
    if (BACK) {   // requested before the wait
        if (SIG) walk(a.x, ta, ur);
        // the earlier states, the given one before step 0 (whose place reads step 0's)
        const T* p = view_at<T>(a.h, b, ta, c);
        uint64_t t = ta;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if ((FULL || u < left) && t > 0) {
                p -= a.h.ts;
                --t;
            }
            hr[u] = load_hint<VW, ACCESS == kScanStream>(p);
        }
        if (tile.k == 0 && a.h0) h0 = load_any<VW>(a.h0 + uint64_t(b) * a.channels + c);
    }

    // the thread's steps composed: S the state from 0, P the product of gates.  Forward keeps both
    // after every step.
    FVec<VW> S = 0.f, P = 1.f, sv[BACK ? 1 : N], pv[BACK ? 1 : N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const FVec<VW> z = to_float<VW, T>(zr[u]), x = to_float<VW, T>(xr[u]);
        const bool on = FULL || u < left;
#pragma unroll
        for (int v = 0; v < VW; ++v) {
            float f, m;
            gates<T, SIG>(z[v], f, m);
            f = on ? f : 1.f;
            S[v] = BACK ? f * ((on ? x[v] : 0.f) + S[v]) : __builtin_fmaf(f, S[v], on ? m * x[v] : 0.f);
            P[v] = gate_product<SIG>(P[v], f);
        }
        if (!BACK) {
            sv[u] = S;
            pv[u] = P;
        }
    }
#pragma unroll
    for (int v = 0; v < VW; ++v) {
        sa[g * slots + r * VW + v] = P[v];
        ss[g * slots + r * VW + v] = S[v];
    }
    __syncthreads();
    float A = 1.f, C = 0.f, s0 = 0.f;
    const uint64_t word = (uint64_t(tile.chain) * a.tiles + tile.k) * slots;
    if (tid < slots) {
#pragma unroll 8
        for (uint32_t i = 0; i < G; ++i) {
            const float f = sa[i * slots + tid];
            C = __builtin_fmaf(f, C, ss[i * slots + tid]);
            A = gate_product<SIG>(A, f);
        }
    }
    uint64_t* known_at = nullptr;   // kScanBack: where the state carried out goes, if anywhere
    if (MODE == kScanBack) {
        uint64_t* words = static_cast<uint64_t*>(a.words) + word;
        const uint32_t group = tile.before / a.span, place = tile.before % a.span;
        if (tid < slots && !tile.first && !tile.last) leave_pair(words + tid, composed(A), C);
        if (tile.first && !tile.last) known_at = words;
        // the groups' words by their place on the way of the state, from the group before on
        uint64_t* groups =
            static_cast<uint64_t*>(a.group_words) + (uint64_t(tile.chain) * a.spans + (group ? group - 1 : 0)) * slots;
        LookBack<SIG> near(words, BACK ? int64_t(slots) : -int64_t(slots), group < 2 ? tile.before : place + a.span, slots);
        LookBack<SIG> far(groups, -int64_t(slots),
                     group < 2 ? 0 : group <= a.most ? group - 1 : (group - 1) % a.most + 1, slots);
        __shared__ float la[2][kScanThreads], ls[2][kScanThreads];
        float ga, gs, none;
        near.join(slots, la[0], ls[0], ga, gs);
        const bool leaves = group > 0 && place == 0 && tid < slots, known = group == 1 || group % a.most == 0;
        if (leaves && !known) leave_pair(groups + tid, composed(ga), gs);
        s0 = gs;
        if (group > 1) {
            far.join(slots, la[1], ls[1], none, s0);
            s0 = __builtin_fmaf(ga, s0, gs);
        }
        if (leaves && known) leave_pair(groups + tid, kScanKnown, s0);
    }
    if (tid < slots) {
        const uint32_t sc = min(tile.slot0 + tid / VW * VW, a.channels - VW) + tid % VW;   // the slot's channel
        const uint64_t state = uint64_t(b) * a.channels + sc;
        if (tile.first) {
            const float* start = BACK ? a.dh_last : a.h0;
            if (start) s0 = start[state];
        } else if (MODE == kScanChain) {
            s0 = wait_for_state(static_cast<const uint32_t*>(a.words) + (BACK ? word + slots : word - slots) + tid);
        }
        const float out = __builtin_fmaf(A, s0, C);
        if (MODE == kScanChain && !tile.last) leave_state(static_cast<uint32_t*>(a.words) + word + tid, out);
        if (MODE == kScanBack && known_at) leave_pair(known_at + tid, kScanKnown, out);
        if (tile.last && a.last) a.last[state] = out;
        // the state each sub-chunk starts from takes the place of its product
#pragma unroll 8
        for (uint32_t i = 0; i < G; ++i) {
            const float f = sa[i * slots + tid];
            sa[i * slots + tid] = s0;
            s0 = __builtin_fmaf(f, s0, ss[i * slots + tid]);
        }
    }
    __syncthreads();
    FVec<VW> s;
#pragma unroll
    for (int v = 0; v < VW; ++v) s[v] = sa[g * slots + r * VW + v];
    if (!BACK) {
        T* h = view_at<T>(a.h, b, ta, c);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            FVec<VW> o;
#pragma unroll
            for (int v = 0; v < VW; ++v) o[v] = __builtin_fmaf(pv[u][v], s[v], sv[u][v]);
            if (FULL || u < left) store_hint<VW, ACCESS != kScanCached>(h, from_float<T, VW>(o));
            h += a.h.ts;
        }
    } else {
        // the recurrence again, now from the state that is carried in: the gates are needed here in any
        // case, and no step's composition has to wait in registers
        T* dg = view_at<T>(a.dgate, b, ta, c);
        T* dx = view_at<T>(a.dx, b, ta, c);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const FVec<VW> z = to_float<VW, T>(zr[u]), d = to_float<VW, T>(xr[u]);
            FVec<VW> before = to_float<VW, T>(hr[u]), og, ox;
            // only a tile's last thread can hold step 0, as its last step
            if (!FULL || u == N - 1) before = ta == uint64_t(u) ? h0 : before;
            if (SIG) before -= to_float<VW, T>(ur[u]);
#pragma unroll
            for (int v = 0; v < VW; ++v) {
                float f, m;
                gates<T, SIG>(z[v], f, m);
                const float l = d[v] + s[v];
                s[v] = f * l;
                og[v] = SIG ? s[v] * before[v] * m : l * before[v];
                ox[v] = l * m;
            }
            if (FULL || u < left) {
                store_hint<VW, ACCESS != kScanCached>(dg, from_float<T, VW>(og));
                store_hint<VW, ACCESS != kScanCached>(dx, from_float<T, VW>(ox));
            }
            dg -= a.dgate.ts;
            dx -= a.dx.ts;
        }
    }
}

template <typename T, int VW, bool SIG, bool BACK, int MODE, int ACCESS>
__global__ __launch_bounds__(kScanThreads, 4) void k_scan_tile(ScanArgs a) {
    __shared__ float sa[kScanThreads * VW], ss[kScanThreads * VW];   // [sub-chunk][slot]
    __shared__ uint32_t ticket;
    const uint32_t tid = threadIdx.x, slots = a.lanes * VW;
    ScanTile tile;
    uint32_t k;   // along the direction of travel
    const uint32_t chains = a.batch * a.groups;
    if (MODE != kScanAlone) {
        // tickets of a queue go through its chains tile by tile
        const uint32_t q = blockIdx.x % a.queues, at = a.queues == kScanQueues ? chiplet_order(q) : q;
        const uint32_t mine = (chains - at + a.queues - 1) / a.queues;
        if (tid == 0)
            ticket = __hip_atomic_fetch_add(a.tickets + q * 16, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        const uint32_t n = __builtin_amdgcn_readfirstlane(ticket);
        if (n >= mine * a.tiles) return;
        tile.chain = at + a.queues * (n % mine);
        k = n / mine;
    } else {
        const uint32_t i = blockIdx.x;
        tile.chain = i < (chains & ~63u) ? chiplet_order(i) : i;
        k = 0;
    }
    tile.b = tile.chain / a.groups;
    tile.slot0 = tile.chain % a.groups * slots;
    tile.k = BACK ? a.tiles - 1 - k : k;
    const uint64_t n = scan_steps(a, tile.b);
    const uint64_t t0 = uint64_t(tile.k) * a.steps;
    const uint64_t t1 = t0 + a.steps < a.length ? t0 + a.steps : a.length;
    tile.tend = t1 < n ? t1 : (t0 < n ? n : t0);
    tile.count = uint32_t(tile.tend - t0);
    tile.first = BACK ? tile.tend == n : tile.k == 0;
    tile.before = BACK ? uint32_t((n + a.steps - 1) / a.steps) - 1 - tile.k : tile.k;
    tile.last = BACK ? tile.k == 0 : tile.tend == n;

    // zeros past the sequence's end
    if (tile.tend < t1) {
        const uint32_t r = tid % a.lanes, c = min(tile.slot0 + r * VW, a.channels - VW);
        const typename Packed<T, VW>::V zero = {};
        for (uint64_t t = tile.tend + tid / a.lanes; t < t1; t += blockDim.x / a.lanes) {
            if (BACK) {
                store_hint<VW, ACCESS != kScanCached>(view_at<T>(a.dgate, tile.b, t, c), zero);
                store_hint<VW, ACCESS != kScanCached>(view_at<T>(a.dx, tile.b, t, c), zero);
            } else {
                store_hint<VW, ACCESS != kScanCached>(view_at<T>(a.h, tile.b, t, c), zero);
            }
        }
    }
    if (tile.count == a.steps) {
        scan_tile<T, VW, SIG, BACK, MODE, ACCESS, true>(a, tile, sa, ss);
    } else if (tile.count > 0) {
        scan_tile<T, VW, SIG, BACK, MODE, ACCESS, false>(a, tile, sa, ss);
    } else if (n == 0 && tile.k == 0 && a.last && tid < slots) {   // an empty sequence
        const uint32_t c = min(tile.slot0 + tid / VW * VW, a.channels - VW) + tid % VW;
        const uint64_t state = uint64_t(tile.b) * a.channels + c;
        const float* start = BACK ? a.dh_last : a.h0;
        a.last[state] = start ? start[state] : 0.f;
    }
}

// Makes the tickets (the first kScanCountBytes) 0 and the words empty.
__global__ __launch_bounds__(256) void k_scan_clear(uint4* p, uint64_t n) {
    const uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x;
    const uint32_t v = i < kScanCountBytes / 16 ? 0u : kScanEmpty;
    if (i < n) p[i] = uint4{v, v, v, v};
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
