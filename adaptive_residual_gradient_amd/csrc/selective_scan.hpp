// Selective state space scan along the sequence, and its gradients, for gfx950.
//
//   h_n <- e_n h_n + u b_n,  e_n = exp(s a_n),  u = s x       (forward, t ascending)
//   y = (sum_n c_n h_n + d x) silu(z)
//   l_n = r c_n + f_n,  f_n <- e_n l_n,  r = dy silu(z)        (backward, t descending; f_n is carried)
//   dc_n = sum r h_n,  db_n = sum l_n u  (over channels),  du = sum_n l_n b_n,
//   q_n = f_n h_n(before),  ds = sum_n q_n a_n + du x,  da_n = sum q_n s,  dx = du s + d r
//
// The exponentials and the states' updates bound it, not the memory: forward takes
// an exponential and four multiplies and adds for every step, channel and state,
// backward an exponential and about 12, and the sums across lanes.  So a lane has one channel and a block of
// its states in registers, nothing is reduced across lanes on the way to y, and b
// and c, which all channels share, come through scalar registers: a kernel before
// lays them out as float32 rows (k_ssm_rows).
//
// A long sequence is cut into chunks, for there are too few channels to fill the
// chip.  A first pass forms each chunk's states from 0 (k_ssm_forward, ENDS), a
// second joins them (k_ssm_join): the decay of a whole chunk is exp(a_n sum s).
// Then the chunks run on their own.  Backward does the same with f.
//
// Backward needs the states of every step.  Forward keeps every 8th, and a
// block of 8 steps is formed again in registers: 4 states a wavefront, whose
// decays and states of 8 steps leave room for several wavefronts a SIMD.  A
// workgroup is 64 channels and all their states' blocks, which share s, u and r
// and add up du, ds and y through LDS.  The sums over channels of db and dc are
// formed by exchanging halves of the values with halves of the lanes, until
// each of the 64 lanes has one of the 64 sums of a block of 8 steps.
//
// 8 x 2048 x 2048 bf16, 16 states, gated: forward 148 us for the chunks' ends,
// 12 to join them and 166 for y; backward 148, 11 and 479, and 25 us for
// the joined sums of db, dc, da and dd.  The vector units are busy 63% of the
// forward ends' time, 69% of y's, 73% of the backward ends' and 88% of the
// gradients', which take 26 vector instructions a step and state, and spill 3 (not gated) or 6 of their 128
// registers with 16 states a channel, 10 or 24 with 8, none with more.
#pragma once

#include "sequence.hpp"

namespace adacomp {

constexpr uint32_t kSsmKeep = 8;        // steps from one kept state to the next; also a block of the kernels
constexpr uint32_t kSsmBlock = 16;      // states of a wavefront forward (8 where there are no more)
constexpr uint32_t kSsmBackBlock = 4;   // and backward
constexpr uint32_t kSsmShort = 8;       // longest sequence of the short kernel

struct SsmArgs {
    ScanView x, dt, z, y, dy, dx, ddt, dz;   // z.p nullable
    ScanView b, c, db, dc;
    const float* a;          // [channels][states]
    const float* d;          // nullable
    const float* dt_bias;    // nullable
    const float* h0;         // nullable; backward: dh_last
    float* last;             // nullable: h_last, or dh0
    float* kept;             // [batch][length / 8][padded][channels], nullable forward
    const int32_t* lengths;  // nullable
    float* rows;             // [batch][length][2][padded]: b and c
    float* ends;             // [batch][chunk][padded][channels]: a chunk's end from 0, then what is carried in
    float* sums;             // [batch][chunk][channels]: sum of s
    float* steps_of;         // [batch][length][channels]: s, where the sequence is in chunks
    float* part_rows;        // [group of 64 channels][batch][length][2][padded]: db and dc
    float* part_a;           // [batch][chunk][padded + 2][channels]: da, dd, ddt_bias
    uint64_t length;
    uint32_t batch, channels, states, padded;   // padded: states in whole blocks of the forward pass
    uint32_t chunks, steps;                     // steps a chunk, a multiple of 8
    uint32_t groups, blocks;                    // wavefronts that cover the channels, and the states
    bool softplus;
};

template <int N>
struct Const {
    static constexpr int value = N;
};

// log(1 + exp(v)), and its derivative 1 / (1 + exp(-v)) from the same exponential.
__device__ __forceinline__ float softplus(float v, float* slope = nullptr) {
    const float e = exp_of_minus(__builtin_elementwise_minimum(__builtin_fabsf(v), 100.f));
    const float w = 1.f + e, r = __builtin_amdgcn_rcpf(w);
    // what the rounding of 1 + e leaves out, relative to it
    const float l = __builtin_fmaf(__builtin_amdgcn_logf(w), kLn2, (e - (w - 1.f)) * r);
    if (slope) *slope = (v < 0.f ? e : 1.f) * __builtin_fmaf(r, __builtin_fmaf(-w, r, 1.f), r);
    return __builtin_elementwise_maximum(v, 0.f) + l;
}
// 1 / (1 + exp(-v)); below -87, where exp(-v) comes to overflow, 0: a gate of the type's lowest value lets nothing
// pass, and v times it is off by less than 1.5e-36.
__device__ __forceinline__ float logistic(float v) {
    const float p = __builtin_elementwise_minimum(__builtin_elementwise_maximum(v, -87.f), 100.f);
    const float w = 1.f + exp_of_minus(p), r = __builtin_amdgcn_rcpf(w);
    return v < -87.f ? 0.f : __builtin_fmaf(r, __builtin_fmaf(-w, r, 1.f), r);
}

// b and c as float32 rows of whole blocks, zeros behind the states.
template <typename T>
__global__ __launch_bounds__(256) void k_ssm_rows(SsmArgs a) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;   // fewer than 2^32, as in the kernels below
    const uint32_t n = i % a.padded, which = i / a.padded & 1u;
    const uint32_t row = i / (2 * a.padded), b = row / uint32_t(a.length), t = row % uint32_t(a.length);
    if (b >= a.batch) return;
    float v = 0.f;
    if (n < a.states && t < steps_of(a.lengths, a.length, b)) v = float(*view_at<T>(which ? a.c : a.b, b, t, n));
    a.rows[i] = v;
}

// A wavefront's place in its workgroup, as a number that all its lanes share.
__device__ __forceinline__ uint32_t wave_of() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// b and c are the same for all lanes and are not written while a kernel reads them: scalar loads, of a
// whole block of states.
template <int NB>
__device__ __forceinline__ FVec<NB> ssm_row(const float* p) {
    typedef const FVec<NB> __attribute__((address_space(4))) Row;
    return *reinterpret_cast<Row*>(reinterpret_cast<uintptr_t>(p));
}

// The place of a wavefront.
struct SsmPlace {
    uint32_t b, chunk, group, block, c, lane;
    uint64_t t0, t1, n;      // the chunk's steps of the tensor, and the sequence's steps
    __device__ __forceinline__ SsmPlace(const SsmArgs& a) {
        // a workgroup's wavefronts: the blocks of one group of channels, then the next group's
        const uint32_t wave = wave_of(), per = blockDim.x / 64 / a.blocks, wide = (a.groups + per - 1) / per;
        lane = threadIdx.x % 64;
        block = wave % a.blocks;
        group = blockIdx.x % wide * per + wave / a.blocks;
        const uint32_t at = blockIdx.x / wide;
        chunk = at % a.chunks;
        b = at / a.chunks;
        c = min(group * 64 + lane, a.channels - 1);
        n = steps_of(a.lengths, a.length, b);
        t0 = uint64_t(chunk) * a.steps;
        t1 = t0 + a.steps < a.length ? t0 + a.steps : a.length;
    }
};

// A rate in units of log 2.  That of a state that keeps nothing, -infinity, is taken for the lowest number, whose decays
// are 0 too: times no step at all, or in a gradient times 0, it would be NaN.
__device__ __forceinline__ float ssm_rate(float a) { return __builtin_elementwise_maximum(a * kLog2e, -3.40282347e38f); }

// The rates a_n of a block; zeros behind the states.
template <int NB>
__device__ __forceinline__ void ssm_rates(const SsmArgs& a, const SsmPlace& w, float (&a2)[NB]) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const uint32_t at = w.block * NB + n;
        a2[n] = at < a.states ? ssm_rate(a.a[uint64_t(w.c) * a.states + at]) : 0.f;
    }
}

// The kernel's arguments where the launch left them (they are its first and only ones), read again at each
// use: kept in scalar registers over a loop they would not fit beside b and c, and be spilled lane by lane.
typedef const SsmArgs __attribute__((address_space(4))) SsmArgsAt;
__device__ __forceinline__ SsmArgsAt& ssm_args_again() {
    SsmArgsAt* p = (SsmArgsAt*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *p;
}

// A sequence's rows of a view, for lanes that each have one channel: a row's address is the same for all
// lanes, a channel's a 32-bit offset from it.
template <typename T>
struct SsmRows {
    char* p;          // step 0's row
    uint64_t step;    // bytes
    __device__ __forceinline__ SsmRows(const ScanView& v, uint32_t b)
        : p(static_cast<char*>(v.p) + uint64_t(b) * v.bs * sizeof(T)), step(v.ts * sizeof(T)) {}
    __device__ __forceinline__ SsmRows(const ScanView __attribute__((address_space(4)))& v, uint32_t b)
        : p(static_cast<char*>(v.p) + uint64_t(b) * v.bs * sizeof(T)), step(v.ts * sizeof(T)) {}
    __device__ __forceinline__ T& at(uint64_t t, uint32_t offset) const {
        return *reinterpret_cast<T*>(p + t * step + offset);
    }
};

// Forward.  kSsmEnds: only the states at the chunk's end, from 0, and s, which kSsmChunks takes; kSsmWhole:
// sequences of one chunk.
constexpr int kSsmEnds = 0, kSsmChunks = 1, kSsmWhole = 2;
template <typename T, int NB, int MODE, bool GATED>
__global__ __launch_bounds__(256) void k_ssm_forward(SsmArgs a) {
    constexpr int S = kSsmKeep;
    constexpr bool ENDS = MODE == kSsmEnds, FORMED = MODE == kSsmChunks;
    extern __shared__ float lds[];   // [2][wavefront][S][64], where a channel's states are several blocks
    const SsmPlace w(a);
    const uint32_t c = w.c, b = w.b, off = c * uint32_t(sizeof(T)), wave = wave_of(), first = wave - w.block;
    const bool mine = w.group < a.groups;
    float a2[NB], h[NB], total = 0.f;
    ssm_rates<NB>(a, w, a2);
    const uint64_t end = w.t1 < w.n ? w.t1 : w.n;
    const uint64_t ends = ((uint64_t(b) * a.chunks + w.chunk) * a.padded + w.block * NB) * a.channels + c;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        h[n] = 0.f;
        const uint32_t at = w.block * NB + n;
        if (ENDS) continue;
        if (FORMED) {
            h[n] = a.ends[ends + uint64_t(n) * a.channels];
        } else if (a.h0 != nullptr && at < a.states) {
            h[n] = a.h0[(uint64_t(b) * a.channels + c) * a.states + at];
        }
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, d = a.d ? a.d[c] : 0.f;
    const bool soft = a.softplus, keep = !ENDS && a.kept != nullptr && mine;
    const uint64_t keeps = (a.length + S - 1) / S;
    uint32_t turn = 0;
    // b and c, requested a step ahead
    const float* const rows = a.rows + uint64_t(b) * a.length * 2 * a.padded + w.block * NB;
    FVec<NB> bn, cn;
    auto request = [&](uint64_t t) {
        const float* row = rows + (t < end ? t : end - 1) * 2 * a.padded;
        bn = ssm_row<NB>(row);
        if (!ENDS) cn = ssm_row<NB>(row + a.padded);
    };
    // U steps from t on
    auto steps = [&](uint64_t t, auto count) {
        constexpr int U = decltype(count)::value;
        T xr[U], zr[U];
        float s[U], y[U];
        SsmArgsAt& again = ssm_args_again();
        const SsmRows<T> xs(again.x, b), ds(again.dt, b), zs(again.z, b);
        float* sp = a.steps_of + (uint64_t(b) * a.length + t) * a.channels;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xr[u] = xs.at(t + u, off);
            if (FORMED) s[u] = sp[uint64_t(u) * a.channels + c];
            else s[u] = float(ds.at(t + u, off));
            if (!ENDS && GATED) zr[u] = zs.at(t + u, off);
        }
        if (keep && t % S == 0) {
            float* k = a.kept + ((uint64_t(b) * keeps + t / S) * a.padded + w.block * NB) * a.channels;
#pragma unroll
            for (int n = 0; n < NB; ++n) k[uint64_t(n) * a.channels + c] = h[n];
        }
        if (!FORMED) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u] += bias;
                const float p = softplus(s[u]);
                s[u] = soft ? p : s[u];
                total += s[u];
            }
            if (ENDS && w.block == 0 && mine)
#pragma unroll
                for (int u = 0; u < U; ++u) sp[uint64_t(u) * a.channels + c] = s[u];
        }
        // no branch from here on: the compiler would move all steps' work behind it, and spill their rows
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            y[u] = 0.f;
            const FVec<NB> bs = bn, cs = cn;
            request(t + u + 1);
            const float v = s[u] * float(xr[u]);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(s[u] * a2[n]), h[n], v * bs[n]);
                if (!ENDS) y[u] = __builtin_fmaf(cs[n], h[n], y[u]);
            }
            __builtin_amdgcn_sched_barrier(0);   // or the rows of all steps are requested at once and spilled
        }
        if (ENDS) return;
        const SsmRows<T> ys(ssm_args_again().y, b);
        auto finish = [&](int u, float sum) {
            sum = __builtin_fmaf(d, float(xr[u]), sum);
            if (GATED) {
                const float z = float(zr[u]);
                sum *= z * logistic(z);
            }
            if (mine) ys.at(t + u, off) = T(sum);
        };
        if (a.blocks == 1) {
#pragma unroll
            for (int u = 0; u < U; ++u) finish(u, y[u]);
        } else {
            float* at = lds + turn * blockDim.x * S;
            turn ^= 1u;
#pragma unroll
            for (int u = 0; u < U; ++u) at[(wave * S + u) * 64 + w.lane] = y[u];
            __syncthreads();   // the other half is free again: whoever writes it next has passed this
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u % a.blocks != w.block) continue;
                float sum = 0.f;
                for (uint32_t j = 0; j < a.blocks; ++j) sum += at[((first + j) * S + u) * 64 + w.lane];
                finish(u, sum);
            }
        }
    };
    uint64_t t = w.t0;
    if (t < end) request(t);
    for (; t + S <= end; t += S) steps(t, Const<S>{});
    for (; t < end; ++t) steps(t, Const<1>{});
    if (!mine) return;
    if (ENDS) {
#pragma unroll
        for (int n = 0; n < NB; ++n) a.ends[ends + uint64_t(n) * a.channels] = h[n];
        if (w.block == 0) a.sums[(uint64_t(b) * a.chunks + w.chunk) * a.channels + c] = total;
        return;
    }
    if (!FORMED && a.last != nullptr)
#pragma unroll
        for (int n = 0; n < NB; ++n)
            if (w.block * NB + n < a.states) a.last[(uint64_t(b) * a.channels + c) * a.states + w.block * NB + n] = h[n];
    if (w.block == 0)
        for (t = end > w.t0 ? end : w.t0; t < w.t1; ++t) SsmRows<T>(a.y, b).at(t, off) = T(0.f);
}

// h exp2(p) + add: the power of two goes to h's exponent, for float32 need not hold the decay of a whole chunk where it
// holds h before and behind it.  Within 2^-600 .. 2^600 the decay is neither 0 nor infinite, as its steps' own need
// not have been: an infinite state times 0, or none times infinity, would be NaN.
__device__ __forceinline__ float decayed(float h, float p, float add) {
    const float whole = floorf(fminf(fmaxf(p, -600.f), 600.f));   // a number of NaN too
    p = __builtin_elementwise_minimum(__builtin_elementwise_maximum(p, -600.f), 600.f);   // NaN
    return __builtin_fmaf(__builtin_amdgcn_exp2f(p - whole), __builtin_amdgcn_ldexpf(h, int(whole)), add);
}

// What is carried into each chunk takes the place of its end from 0; backward
// (BACK) from the last chunk to the first.  One thread a sequence, state and channel.
template <bool BACK>
__global__ __launch_bounds__(256) void k_ssm_join(SsmArgs a) {
    const uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x;
    const uint32_t c = uint32_t(i % a.channels), n = uint32_t(i / a.channels % a.padded);
    const uint64_t b = i / a.channels / a.padded;
    if (b >= a.batch) return;
    const uint64_t place = (b * a.channels + c) * a.states + n;
    float h = 0.f, a2 = 0.f;
    if (n < a.states) {
        a2 = ssm_rate(a.a[uint64_t(c) * a.states + n]);
        if (a.h0 != nullptr) h = a.h0[place];
    }
    constexpr uint32_t U = 16;   // chunks requested together, while the ones before are joined
    float* const ends = a.ends + (b * a.chunks * a.padded + n) * a.channels + c;
    const float* const sums = a.sums + b * a.chunks * a.channels + c;
    const uint64_t step = uint64_t(a.padded) * a.channels;
    float end[U], sum[U];
    auto request = [&](uint32_t k) {
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t at = min(k + u, a.chunks - 1), chunk = BACK ? a.chunks - 1 - at : at;
            end[u] = ends[chunk * step];
            sum[u] = sums[uint64_t(chunk) * a.channels];
        }
    };
    request(0);
    for (uint32_t k = 0; k < a.chunks; k += U) {
        float now[U], s[U];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            now[u] = end[u];
            s[u] = sum[u];
        }
        if (k + U < a.chunks) request(k + U);
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            if (k + u >= a.chunks) continue;
            const uint32_t chunk = BACK ? a.chunks - 1 - (k + u) : k + u;
            ends[chunk * step] = h;
            h = decayed(h, s[u] * a2, now[u]);
        }
    }
    if (a.last != nullptr && n < a.states) a.last[place] = h;
}

// Sequences of at most kSsmShort steps: `quads` lanes a channel with 4 states each.
template <typename T>
__global__ __launch_bounds__(256) void k_ssm_short(SsmArgs a, uint32_t quads) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, q = i % quads, unit = i / quads, units = a.batch * a.channels;
    const bool mine = unit < units;
    // lanes past the end go along with the last channel: the sum over the quads takes all lanes
    const uint32_t at = mine ? unit : units - 1, c = at % a.channels, b = at / a.channels;
    const uint32_t n0 = q * 4, left = n0 < a.states ? min(a.states - n0, 4u) : 0;
    const uint32_t n = uint32_t(steps_of(a.lengths, a.length, b));
    FVec<4> h = 0.f, a2 = 0.f;
    const uint64_t place = uint64_t(at) * a.states + n0;
    if (left == 4) {
        a2 = load_any<4>(a.a + uint64_t(c) * a.states + n0);
        if (a.h0) h = load_any<4>(a.h0 + place);
    } else {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            if (k >= left) continue;
            a2[k] = a.a[uint64_t(c) * a.states + n0 + k];
            if (a.h0) h[k] = a.h0[place + k];
        }
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, d = a.d ? a.d[c] : 0.f;
    for (uint32_t t = 0; t < n; ++t) {
        const T* bp = view_at<T>(a.b, b, t, n0);
        const T* cp = view_at<T>(a.c, b, t, n0);
        FVec<4> bv = 0.f, cv = 0.f;
        if (left == 4) {
            bv = to_float<4, T>(load_any<4>(bp));
            cv = to_float<4, T>(load_any<4>(cp));
        } else {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                if (k >= left) continue;
                bv[k] = float(bp[k]);
                cv[k] = float(cp[k]);
            }
        }
        const float x = float(*view_at<T>(a.x, b, t, c));
        const float z = a.z.p ? float(*view_at<T>(a.z, b, t, c)) : 0.f;
        float s = float(*view_at<T>(a.dt, b, t, c)) + bias, y = 0.f;
        if (a.softplus) s = softplus(s);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(s * ssm_rate(a2[k])), h[k], s * x * bv[k]);
            y = __builtin_fmaf(cv[k], h[k], y);
        }
        for (uint32_t m = 1; m < quads; m *= 2) y += __shfl_xor(y, int(m));
        y = __builtin_fmaf(d, x, y);
        if (a.z.p != nullptr) y *= z * logistic(z);
        if (mine && q == 0) *view_at<T>(a.y, b, t, c) = T(y);
    }
    if (!mine) return;
    if (q == 0)
        for (uint64_t t = n; t < a.length; ++t) *view_at<T>(a.y, b, t, c) = T(0.f);
    if (a.last == nullptr) return;
    if (left == 4) {
        store_any<4>(a.last + place, h);
    } else {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
            if (k < left) a.last[place + k] = h[k];
    }
}

// ---- backward ----

// f at each chunk's first step from 0 at its end, and the sum of s.
template <typename T, int NB, bool GATED>
__global__ __launch_bounds__(256) void k_ssm_back_ends(SsmArgs a) {
    constexpr int S = kSsmKeep;
    const SsmPlace w(a);
    if (w.group >= a.groups) return;
    const uint32_t c = w.c, b = w.b, off = c * uint32_t(sizeof(T));
    float a2[NB], f[NB], total = 0.f;
    ssm_rates<NB>(a, w, a2);
#pragma unroll
    for (int n = 0; n < NB; ++n) f[n] = 0.f;
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    const bool soft = a.softplus;
    const uint64_t end = w.t1 < w.n ? w.t1 : w.n;
    const SsmRows<T> rs(a.dy, b), ds(a.dt, b), zs(a.z, b);
    // U steps from t on, the last one first
    auto steps = [&](uint64_t t, auto count) {
        constexpr int U = decltype(count)::value;
        T rr[U], sr[U], zr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rr[u] = rs.at(t + u, off);
            sr[u] = ds.at(t + u, off);
            if (GATED) zr[u] = zs.at(t + u, off);
        }
        const float* row = a.rows + ((uint64_t(b) * a.length + t) * 2 + 1) * a.padded + w.block * NB;
#pragma unroll
        for (int u = U - 1; u >= 0; --u) {
            const FVec<NB> cs = ssm_row<NB>(row + uint64_t(u) * 2 * a.padded);
            const float v = float(sr[u]) + bias, p = softplus(v), s = soft ? p : v;
            total += s;
            float r = float(rr[u]);
            if (GATED) {
                const float z = float(zr[u]);
                r *= z * logistic(z);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
                f[n] = __builtin_amdgcn_exp2f(s * a2[n]) * __builtin_fmaf(r, cs[n], f[n]);
            __builtin_amdgcn_sched_barrier(0);   // or the rows of all steps are requested at once and spilled
        }
    };
    if (w.t0 < end) {
        uint64_t t = end;
        while ((t - w.t0) % S != 0) steps(--t, Const<1>{});
        while (t > w.t0) steps(t -= S, Const<S>{});
    }
    const uint64_t ends = ((uint64_t(b) * a.chunks + w.chunk) * a.padded + w.block * NB) * a.channels + c;
#pragma unroll
    for (int n = 0; n < NB; ++n) a.ends[ends + uint64_t(n) * a.channels] = f[n];
    if (w.block == 0) a.sums[(uint64_t(b) * a.chunks + w.chunk) * a.channels + c] = total;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false));
}

// The sums over lanes of v[0..15], each over a quarter of 16 lanes: lane l has value
// 8 (l / 32) + 4 (l / 16 % 2) + 2 (l / 8 % 2) + l / 4 % 2, summed over the lanes that are congruent to l modulo 4.
__device__ __forceinline__ float sum_halves(float (&v)[16]) {
    typedef unsigned int Pair __attribute__((ext_vector_type(2)));
    float p[8], q[4], r[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // the lower 32 lanes keep v[i], the upper ones v[i + 8]
        const Pair x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 8]), false, false);
        p[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // rows of 16 lanes
        const Pair x = __builtin_amdgcn_permlane16_swap(__float_as_uint(p[i]), __float_as_uint(p[i + 4]), false, false);
        q[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    }
    auto move = [](float old, float from, auto ctrl, auto banks) {
        return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
            static_cast<int>(__float_as_uint(old)), static_cast<int>(__float_as_uint(from)), decltype(ctrl)::value, 0xf,
            decltype(banks)::value, false)));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // halves of a row: row_ror:8
        const float own = move(q[i], q[i + 2], Const<0x128>{}, Const<0xc>{});
        const float other = move(q[i + 2], q[i], Const<0x128>{}, Const<0x3>{});
        r[i] = own + other;
    }
    // quarters: row_shr:4 and row_shl:4.  own: in the odd quarters r[1] of the lane 4 before; other: in the
    // even ones r[0] of the lane 4 behind
    const float own = move(r[0], r[1], Const<0x114>{}, Const<0xa>{});
    const float other = move(r[1], r[0], Const<0x104>{}, Const<0x5>{});
    return own + other;
}
// Of four such values the sums over the four lanes: lane l has that of value l % 4.
__device__ __forceinline__ float sum_quads(float v0, float v1, float v2, float v3, uint32_t lane) {
    auto swap1 = [](float x) {   // quad_perm:[1,0,3,2]
        return __uint_as_float(dpp_move<0xB1>(__float_as_uint(x)));
    };
    auto swap2 = [](float x) {   // quad_perm:[2,3,0,1]
        return __uint_as_float(dpp_move<0x4E>(__float_as_uint(x)));
    };
    const bool hi = lane & 2u, odd = lane & 1u;
    const float a = (hi ? v2 : v0) + swap2(hi ? v0 : v2);   // lanes 0, 1: v0; 2, 3: v2
    const float b = (hi ? v3 : v1) + swap2(hi ? v1 : v3);
    return (odd ? b : a) + swap1(odd ? a : b);
}

// A workgroup is 64 channels, a wavefront kSsmBackBlock of their states.  Of a block of 8 steps each
// wavefront prepares OWN (s, u and r, which all of them take from LDS) and finishes the same ones, from the sums
// over the wavefronts of du, ds and s that lie in LDS then.
template <typename T, int OWN, bool GATED>
__global__ __launch_bounds__(OWN == 1 ? 1024 : 256, 4) void k_ssm_backward(SsmArgs a) {
    constexpr int S = kSsmKeep, NB = kSsmBackBlock, V = GATED ? 3 : 2;
    extern __shared__ float lds[];   // [3][S][64]: s, u, r;  [wavefront][V][S][64]: du, ds, sum
    float* const ready = lds;
    float* const parts = lds + 3 * S * 64;
    const SsmPlace w(a);
    const uint32_t c = w.c, b = w.b, off = c * uint32_t(sizeof(T)), lane = w.lane;
    // a lane past the last channel goes along with it, without a part in the sums over channels
    const bool mine = w.group * 64 + lane < a.channels;
    float a2[NB], f[NB], da[NB], dd = 0.f, dbias = 0.f;
    ssm_rates<NB>(a, w, a2);
    const uint64_t ends = ((uint64_t(b) * a.chunks + w.chunk) * a.padded + w.block * NB) * a.channels + c;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        da[n] = f[n] = 0.f;
        const uint32_t at = w.block * NB + n;
        if (a.chunks > 1) f[n] = a.ends[ends + uint64_t(n) * a.channels];
        else if (a.h0 != nullptr && at < a.states) f[n] = a.h0[(uint64_t(b) * a.channels + c) * a.states + at];
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, d = a.d ? a.d[c] : 0.f;
    const bool soft = a.softplus;
    const uint64_t end = w.t1 < w.n ? w.t1 : w.n, keeps = (a.length + S - 1) / S;
    for (uint64_t t = w.t0 < end ? (end - 1) / S * S : 0; w.t0 < end; t -= S) {
        const uint32_t left = end - t < uint64_t(S) ? uint32_t(end - t) : uint32_t(S);
        SsmArgsAt& again = ssm_args_again();
        const SsmRows<T> xs(again.x, b), ss(again.dt, b), rs(again.dy, b), zs(again.z, b);
        // what the wavefront keeps of its own steps
        float x[OWN], s[OWN], r[OWN], slope[OWN], back[OWN];
        T xr[OWN], sr[OWN], rr[OWN], zr[OWN];
        const float* k = a.kept + ((uint64_t(b) * keeps + t / S) * a.padded + w.block * NB) * a.channels;
        float h[S + 1][NB], e[S][NB];
#pragma unroll
        for (int i = 0; i < OWN; ++i) {   // past the end the last step again
            const uint32_t u = min(w.block + a.blocks * i, left - 1);
            xr[i] = xs.at(t + u, off);
            sr[i] = ss.at(t + u, off);
            rr[i] = rs.at(t + u, off);
            if (GATED) zr[i] = zs.at(t + u, off);
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) h[0][n] = k[uint64_t(n) * a.channels + c];
        // b and c of the whole block, requested before the barrier
        const float* row = a.rows + (uint64_t(b) * a.length + t) * 2 * a.padded + w.block * NB;
        FVec<NB> bs[S], cs[S];
#pragma unroll
        for (int u = 0; u < S; ++u) {
            const float* at = row + uint64_t(uint32_t(u) < left ? u : 0) * 2 * a.padded;
            bs[u] = ssm_row<NB>(at);
            cs[u] = ssm_row<NB>(at + a.padded);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const uint32_t u = w.block + a.blocks * i;
            x[i] = float(xr[i]);
            const float v = float(sr[i]) + bias, p = softplus(v, &slope[i]);
            s[i] = soft ? p : v;
            slope[i] = soft ? slope[i] : 1.f;
            r[i] = float(rr[i]);
            if (GATED) {
                const float z = float(zr[i]), q = logistic(z), g = z * q;
                back[i] = r[i] * __builtin_fmaf(g, 1.f - q, q);
                r[i] *= g;
            }
            if (u < S) {   // behind the sequence's end nothing moves
                const bool on = u < left;
                ready[u * 64 + lane] = on ? s[i] : 0.f;
                ready[(S + u) * 64 + lane] = on && mine ? s[i] * x[i] : 0.f;
                ready[(2 * S + u) * 64 + lane] = on && mine ? r[i] : 0.f;
            }
        }
        __syncthreads();
        // the block's decays and states
        float* part = parts + (w.block * V * S) * 64 + lane;
#pragma unroll
        for (int u = 0; u < S; ++u) {
            const float step = ready[u * 64 + lane], in = ready[(S + u) * 64 + lane];
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                e[u][n] = __builtin_amdgcn_exp2f(step * a2[n]);
                h[u + 1][n] = __builtin_fmaf(e[u][n], h[u][n], in * bs[u][n]);
                if (GATED) sum = __builtin_fmaf(cs[u][n], h[u + 1][n], sum);
            }
            if (GATED) part[(2 * S + u) * 64] = sum;
            __builtin_amdgcn_sched_barrier(0);
        }
        float v[16], quad[S / 2];
#pragma unroll
        for (int u = S - 1; u >= 0; --u) {
            const float step = ready[u * 64 + lane], in = ready[(S + u) * 64 + lane], out = ready[(2 * S + u) * 64 + lane];
            float du = 0.f, ds = 0.f;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const float l = __builtin_fmaf(out, cs[u][n], f[n]);
                f[n] = e[u][n] * l;
                const float q = f[n] * h[u][n];
                du = __builtin_fmaf(l, bs[u][n], du);
                ds = __builtin_fmaf(q, a2[n], ds);
                da[n] = __builtin_fmaf(q, step, da[n]);
                v[u % 2 * 4 + n] = l * in;
                v[8 + u % 2 * 4 + n] = out * h[u + 1][n];
            }
            part[u * 64] = du;
            part[(S + u) * 64] = ds;
            if (u % 2 == 0) {
                quad[u / 2] = sum_halves(v);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        {   // lane l has the sum of step 2 (l % 4) + l / 16 % 2, state l / 4 % 4, of b or (from lane 32 on) of c
            const float total = sum_quads(quad[0], quad[1], quad[2], quad[3], lane);
            const uint32_t u = 2 * (lane % 4) + lane / 16 % 2;
            if (u < left)
                a.part_rows[(((uint64_t(w.group) * a.batch + b) * a.length + t + u) * 2 + lane / 32) * a.padded +
                            w.block * NB + lane / 4 % 4] = total;
        }
        __syncthreads();
        SsmArgsAt& outs = ssm_args_again();
        const SsmRows<T> dxs(outs.dx, b), dss(outs.ddt, b), dzs(outs.dz, b);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const uint32_t u = w.block + a.blocks * i;
            if (u >= left) continue;
            float sums[V] = {};
            for (uint32_t j = 0; j < a.blocks; ++j)
#pragma unroll
                for (int q = 0; q < V; ++q) sums[q] += parts[((j * V + q) * S + u) * 64 + lane];
            const float dx = __builtin_fmaf(sums[0], s[i], d * r[i]);
            const float dv = slope[i] * __builtin_fmaf(sums[1], kLn2, sums[0] * x[i]);   // the rates were in units of log 2
            dd = __builtin_fmaf(r[i], x[i], dd);
            dbias += dv;
            if (!mine) continue;
            dxs.at(t + u, off) = T(dx);
            dss.at(t + u, off) = T(dv);
            if (GATED) dzs.at(t + u, off) = T(back[i] * __builtin_fmaf(d, x[i], sums[V - 1]));
        }
        if (t == w.t0) break;
    }
    // sums over the chunk's steps
    float* part = a.part_a + (uint64_t(b) * a.chunks + w.chunk) * (a.padded + 2) * a.channels + c;
    if (mine)
#pragma unroll
        for (int n = 0; n < NB; ++n) part[uint64_t(w.block * NB + n) * a.channels] = da[n];
    __syncthreads();
    lds[(w.block * 2 + 0) * 64 + lane] = dd;
    lds[(w.block * 2 + 1) * 64 + lane] = dbias;
    __syncthreads();
    if (!mine) return;
    if (w.block == 0) {
        dd = dbias = 0.f;
        for (uint32_t j = 0; j < a.blocks; ++j) {
            dd += lds[(j * 2 + 0) * 64 + lane];
            dbias += lds[(j * 2 + 1) * 64 + lane];
        }
        part[uint64_t(a.padded) * a.channels] = dd;
        part[uint64_t(a.padded + 1) * a.channels] = dbias;
        for (uint64_t t = end > w.t0 ? end : w.t0; t < w.t1; ++t) {
            SsmRows<T>(a.dx, b).at(t, off) = T(0.f);
            SsmRows<T>(a.ddt, b).at(t, off) = T(0.f);
            if (GATED) SsmRows<T>(a.dz, b).at(t, off) = T(0.f);
        }
    }
    if (a.chunks == 1 && a.last != nullptr)
#pragma unroll
        for (int n = 0; n < NB; ++n)
            if (w.block * NB + n < a.states) a.last[(uint64_t(b) * a.channels + c) * a.states + w.block * NB + n] = f[n];
}

// db and dc: the groups' sums over their channels joined.
template <typename T>
__global__ __launch_bounds__(256) void k_ssm_row_grad(SsmArgs a) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;   // fewer than 2^32, as in the kernels below
    const uint32_t n = i % a.padded, which = i / a.padded & 1u;
    const uint32_t row = i / (2 * a.padded), b = row / uint32_t(a.length), t = row % uint32_t(a.length);
    if (b >= a.batch || n >= a.states) return;
    float s = 0.f;
    if (t < steps_of(a.lengths, a.length, b)) {
        const uint64_t stride = uint64_t(a.batch) * a.length * 2 * a.padded;
#pragma unroll 8
        for (uint32_t g = 0; g < a.groups; ++g) s += a.part_rows[g * stride + i];
    }
    *view_at<T>(which ? a.dc : a.db, b, t, n) = T(s);
}

// da, dd and ddt_bias: the chunks' sums over their steps joined.
__global__ __launch_bounds__(256) void k_ssm_channel_grad(const float* part, uint32_t rows, uint32_t padded,
                                                          uint32_t states, uint32_t channels, float* da, float* dd,
                                                          float* ddt_bias) {
    __shared__ double sums[16][17];
    const uint32_t lane = threadIdx.x % 16, sub = threadIdx.x / 16;
    const uint32_t c = blockIdx.x * 16 + lane, n = blockIdx.y;
    double s = 0.0;
    if (c < channels)
#pragma unroll 8
        for (uint32_t i = sub; i < rows; i += 16) s += part[(uint64_t(i) * (padded + 2) + n) * channels + c];
    sums[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || c >= channels) return;
    for (uint32_t j = 1; j < 16; ++j) s += sums[j][lane];
    if (n < states) da[uint64_t(c) * states + n] = float(s);
    else if (n == padded && dd != nullptr) dd[c] = float(s);
    else if (n == padded + 1 && ddt_bias != nullptr) ddt_bias[c] = float(s);
}

}  // namespace adacomp
