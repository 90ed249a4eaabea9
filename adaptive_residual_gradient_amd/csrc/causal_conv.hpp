// Short causal convolution along the sequence, one filter a channel, and its
// gradients, for gfx950.
//
//   p_t = bias + sum_k w_k x_(t-K+1+k),  y = p or p sigmoid(p)
//   g_t = dy_t (p's derivative),  dx_t = sum_k w_k g_(t+K-1-k),  dw_k = sum g_t x_(t-K+1+k)
//
// A thread has 8 bytes of channels and goes along the sequence with the last
// steps in registers: forward 4 to 32 steps, backward a longer stretch, so that the
// steps that two stretches both read, K - 1 of x (and of dy), are few.  The
// weight's gradient is summed in registers along the stretch, over a
// workgroup's stretches in LDS, written as one partial row a workgroup and
// joined in float64 by a second kernel.
//
// Memory bounds both directions: 8 x 4096 x 2048 bf16 of 4 taps takes 48 us
// forward (5.6 TB/s), 94 us backward (4.3 TB/s) and 7 us for the rows joined.  Backward the vector units are busy
// 63% of it: 1069 instructions for 8 steps, 88 of them integer products and 100 64-bit additions and selects, for
// addresses that are formed anew and the conditions of every step.  64 x 2048
// of one step take 4.4 us, most of it the round trips to the memory: all loads
// are requested together, the kept steps' among them (6.1 us with those behind the results).
#pragma once

#include "sequence.hpp"

namespace adacomp {

// Steps of a thread forward: the first of them that leaves enough threads (8 x 4096 x 2048 bf16, 4 taps, in us: 8
// steps 70, 12 63, 16 58, 24 53.5, 32 53, before the weights came in whole vectors).
constexpr uint32_t kConvRows[3] = {32, 12, 4};
constexpr uint32_t kConvThreads = 256;
// Partial rows of the weight's gradient: 3 wavefronts a SIMD, which the registers hold (8 x 4096 x 2048 bf16
// backward and the rows joined: 97 us, with 256 101, with 512 111).
constexpr uint32_t kConvMaxPartials = 384;
// The filters that kernels are made for: 2, 3 and 4 taps; 8, for every other number too.
constexpr uint32_t conv_kernel_taps(uint32_t taps) { return taps >= 2 && taps <= 4 ? taps : 8; }
// A thread's channels: 8 bytes, for more threads than with 16 (8 x 4096 x 2048 bf16 72 us forward and 109 backward
// against 98 and 118, before the other steps).
constexpr uint32_t kConvBytes = 8;

struct ConvArgs {
    ScanView x, y, dy, dx;
    const float* weight;     // [channels][taps]
    const float* bias;       // nullable
    const void* state;       // nullable [batch][taps - 1][channels]
    void* state_out;         // nullable
    void* dstate;            // nullable
    const int32_t* lengths;  // nullable
    float* partial;          // [workgroup][taps + 1][channels]
    uint64_t length;
    uint32_t batch, channels, taps;
    uint32_t lanes;          // threads that cover the channels
    uint32_t per;            // backward: threads of one stretch in a workgroup
    uint32_t pieces, rows;   // stretches of a sequence, and (backward) their steps
    bool past;               // results go past the cache
};

// p's logistic function.  Below -87, where exp(-p) comes to overflow, it is 0: a gate of the type's lowest value lets
// nothing pass, and p times it is off by less than 1.5e-36.  Of 16-bit calls, whose results are rounded far coarser,
// without the corrections of the exponential's argument and of the reciprocal: off by 2^-24 (|p| + 4).
template <typename T>
__device__ __forceinline__ float conv_gate(float p) {
    if (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(p * -kLog2e));
    const float v = __builtin_elementwise_minimum(__builtin_elementwise_maximum(p, -87.f), 100.f);
    const float d = 1.f + exp_of_minus(v);
    const float r = __builtin_amdgcn_rcpf(d);
    return p < -87.f ? 0.f : __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.f), r);
}

// The weights of a thread's channels by tap, those of the KT - taps taps that are not there 0.
template <int KT, int VW>
__device__ __forceinline__ void conv_weights(const ConvArgs& a, uint32_t c, FVec<VW> (&w)[KT]) {
    if (KT <= 4) {   // their own kernels: KT taps of VW channels, which lie together
        FVec<VW> all[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) all[k] = load_any<VW>(a.weight + uint64_t(c) * KT + k * VW);
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int v = 0; v < VW; ++v) w[k][v] = all[(v * KT + k) / VW][(v * KT + k) % VW];
        return;
    }
    const uint32_t skip = KT - a.taps;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int v = 0; v < VW; ++v)
            w[k][v] = uint32_t(k) < skip ? 0.f : a.weight[uint64_t(c + v) * a.taps + k - skip];
}

// x at a step before step 0: from the state, of which it is the (taps - 1 - back)-th; 0 before that or without.
template <typename T, int VW>
__device__ __forceinline__ typename Packed<T, VW>::V conv_before(const ConvArgs& a, uint32_t b, uint32_t c,
                                                                 uint32_t back) {
    typename Packed<T, VW>::V v = {};
    if (a.state != nullptr && back < a.taps)
        v = load_any<VW>(static_cast<const T*>(a.state) +
                         (uint64_t(b) * (a.taps - 1) + (a.taps - 1 - back)) * a.channels + c);
    return v;
}

// One product of the filter.  KT past 4 stands for fewer taps too: what lies under the ones that are not
// there, which may be NaN, has no part.
template <int KT, int VW>
__device__ __forceinline__ FVec<VW> conv_sum(const ConvArgs& a, const FVec<VW> (&w)[KT], const FVec<VW>* x,
                                             FVec<VW> sum) {
    const uint32_t skip = KT - a.taps;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        if (KT > 4 && uint32_t(k) < skip) continue;
#pragma unroll
        for (int v = 0; v < VW; ++v) sum[v] = __builtin_fmaf(w[k][v], x[k][v], sum[v]);
    }
    return sum;
}

// Workgroups go to the 8 chiplets in turn: each chiplet takes a run of them, whose stretches follow each
// other, so that the steps that two stretches read come from its cache.
__device__ __forceinline__ uint32_t conv_workgroup() {
    const uint32_t each = gridDim.x / 8, rest = gridDim.x % 8, xcd = blockIdx.x % 8;
    return xcd * each + min(xcd, rest) + blockIdx.x / 8;
}

// ROWS steps of one sequence.
template <typename T, int VW, int KT, int ROWS>
__global__ __launch_bounds__(kConvThreads) void k_conv(ConvArgs a, bool silu) {
    typedef typename Packed<T, VW>::V V;
    const uint32_t i = conv_workgroup() * kConvThreads + threadIdx.x;   // fewer than 2^32
    const uint32_t r = i % a.lanes, unit = i / a.lanes, piece = unit % a.pieces, b = unit / a.pieces;
    if (b >= a.batch) return;
    const uint32_t c = min(r * VW, a.channels - VW);
    const uint64_t n = steps_of(a.lengths, a.length, b), t0 = uint64_t(piece) * ROWS;
    const int steps = int(t0 + ROWS < a.length ? ROWS : a.length - t0);   // of the tensor
    const int live = t0 < n ? int(n - t0 < uint64_t(ROWS) ? n - t0 : ROWS) : 0;   // of the sequence
    // the steps before step n, requested with the others; [j]: KT - 1 - j steps before it
    const bool keeps = piece == 0 && a.state_out != nullptr;
    V kept[KT > 1 ? KT - 1 : 1];
    if (keeps)
#pragma unroll
        for (int j = 0; j < KT - 1; ++j) {
            const uint32_t back = KT - 1 - j;
            if (back >= a.taps) continue;
            if (n >= back) kept[j] = load_any<VW>(view_at<T>(a.x, b, n - back, c));
            else kept[j] = conv_before<T, VW>(a, b, c, uint32_t(back - n));
        }
    if (live > 0) {
        V raw[KT - 1 + ROWS];
        const T* p = view_at<T>(a.x, b, t0, c);
        if (t0 >= KT - 1) {
#pragma unroll
            for (int u = 0; u < KT - 1; ++u) raw[u] = load_any<VW>(p - uint64_t(KT - 1 - u) * a.x.ts);
        } else {
#pragma unroll
            for (int u = 0; u < KT - 1; ++u) {
                const uint32_t back = KT - 1 - u;
                if (t0 >= back) raw[u] = load_any<VW>(p - uint64_t(back) * a.x.ts);
                else raw[u] = conv_before<T, VW>(a, b, c, uint32_t(back - t0));
            }
        }
        // past the sequence's end its last step again, so that no load stands under a condition
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            raw[KT - 1 + u] = load_any<VW>(p);
            p += u + 1 < live ? a.x.ts : 0;
        }
        FVec<VW> w[KT], bias = 0.f, x[KT - 1 + ROWS];
        conv_weights<KT, VW>(a, c, w);
        if (a.bias) bias = load_any<VW>(a.bias + c);
        T* y = view_at<T>(a.y, b, t0, c);
#pragma unroll
        for (int u = 0; u < KT - 1 + ROWS; ++u) x[u] = to_float<VW, T>(raw[u]);
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            FVec<VW> s = conv_sum<KT, VW>(a, w, x + u, bias);
            if (silu)
#pragma unroll
                for (int v = 0; v < VW; ++v) s[v] *= conv_gate<T>(s[v]);
            if (u < live) {
                if (a.past) stream_store<VW>(y, from_float<T, VW>(s));
                else store_any<VW>(y, from_float<T, VW>(s));
            }
            y += a.y.ts;
        }
    }
    for (int u = live; u < steps; ++u) store_any<VW>(view_at<T>(a.y, b, t0 + u, c), V{});
    if (keeps) {
        T* out = static_cast<T*>(a.state_out) + uint64_t(b) * (a.taps - 1) * a.channels + c;
#pragma unroll
        for (int j = 0; j < KT - 1; ++j)
            if (uint32_t(j) >= KT - a.taps) store_any<VW>(out + uint64_t(j - (KT - a.taps)) * a.channels, kept[j]);
    }
}

// The gradients of a stretch of a.rows steps: g is formed from its first step
// on, and for the KT - 1 steps behind it, which dx needs too.  A workgroup is
// `subs` stretches of `per` threads.
template <typename T, int VW, int KT>
__global__ __launch_bounds__(kConvThreads) void k_conv_backward(ConvArgs a, bool silu) {
    typedef typename Packed<T, VW>::V V;
    constexpr int U = 8;   // steps requested together
    constexpr uint32_t HALO = KT - 1;
    __shared__ float sums[kConvThreads * VW];   // [stretch][channel of a thread][thread of the stretch]
    const uint32_t per = a.per, subs = kConvThreads / per, sub = threadIdx.x / per, lane = threadIdx.x % per;
    const uint32_t groups = (a.lanes + per - 1) / per, row = blockIdx.x / groups;
    const uint64_t unit = uint64_t(row) * subs + sub, units = uint64_t(a.batch) * a.pieces;
    const uint32_t r = blockIdx.x % groups * per + lane;
    const uint32_t c = min(r * VW, a.channels - VW), skip = KT - a.taps;
    FVec<VW> dw[KT], db = 0.f;
#pragma unroll
    for (int k = 0; k < KT; ++k) dw[k] = 0.f;
    if (sub < subs && unit < units && r < a.lanes) {
        const uint32_t b = uint32_t(unit / a.pieces), piece = uint32_t(unit % a.pieces);
        FVec<VW> w[KT], bias = 0.f;
        conv_weights<KT, VW>(a, c, w);
        if (a.bias) bias = load_any<VW>(a.bias + c);
        const uint64_t n = steps_of(a.lengths, a.length, b), t0 = uint64_t(piece) * a.rows;
        const uint64_t t1 = t0 + a.rows < a.length ? t0 + a.rows : a.length;
        const uint64_t end = t1 < n ? t1 : n;   // dx is zero from here on
        // x and g at the last KT steps, the newest last
        FVec<VW> xw[KT], gw[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) xw[k] = gw[k] = 0.f;
        if (t0 < n) {
#pragma unroll
            for (int u = 1; u < KT; ++u) {
                const uint32_t back = KT - u;   // steps before t0
                if (t0 >= back) xw[u] = to_float<VW, T>(load_any<VW>(view_at<T>(a.x, b, t0 - back, c)));
                else xw[u] = to_float<VW, T>(conv_before<T, VW>(a, b, c, uint32_t(back - t0)));
            }
        }
        const uint64_t last = t0 < n ? end + HALO : t0;
        for (uint64_t t = t0; t < last; t += U) {
            V xr[U], dr[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {   // past the end the last step again
                const uint64_t at = t + u < n ? t + u : n - 1;
                xr[u] = load_any<VW>(view_at<T>(a.x, b, at, c));
                dr[u] = load_any<VW>(view_at<T>(a.dy, b, at, c));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint64_t s = t + u;
#pragma unroll
                for (int k = 0; k + 1 < KT; ++k) {
                    xw[k] = xw[k + 1];
                    gw[k] = gw[k + 1];
                }
                xw[KT - 1] = to_float<VW, T>(xr[u]);
                FVec<VW> g = to_float<VW, T>(dr[u]);
                if (silu) {
                    const FVec<VW> p = conv_sum<KT, VW>(a, w, xw, bias);
#pragma unroll
                    for (int v = 0; v < VW; ++v) {
                        const float q = conv_gate<T>(p[v]);
                        g[v] *= __builtin_fmaf(p[v] * q, 1.f - q, q);
                    }
                }
                if (s >= n) g = 0.f;
                gw[KT - 1] = g;
                if (s < end) {
                    db += g;
#pragma unroll
                    for (int k = 0; k < KT; ++k) {
                        if (KT > 4 && uint32_t(k) < skip) continue;
#pragma unroll
                        for (int v = 0; v < VW; ++v) dw[k][v] = __builtin_fmaf(g[v], xw[k][v], dw[k][v]);
                    }
                }
                // dx of step s - HALO: tap k of KT goes with g of step s - k
                if (s >= last || (t0 > 0 && s < t0 + HALO)) continue;
                FVec<VW> d = 0.f;
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    if (KT > 4 && uint32_t(k) < skip) continue;
#pragma unroll
                    for (int v = 0; v < VW; ++v) d[v] = __builtin_fmaf(w[k][v], gw[KT - 1 - k][v], d[v]);
                }
                if (s >= HALO) {
                    T* at = view_at<T>(a.dx, b, s - HALO, c);
                    if (a.past) stream_store<VW>(at, from_float<T, VW>(d));
                    else store_any<VW>(at, from_float<T, VW>(d));
                } else if (a.dstate != nullptr && HALO - s < a.taps) {   // so many steps before step 0
                    store_any<VW>(static_cast<T*>(a.dstate) +
                                      (uint64_t(b) * (a.taps - 1) + (a.taps - 1 - uint32_t(HALO - s))) * a.channels + c,
                                  from_float<T, VW>(d));
                }
            }
        }
        for (uint64_t t = end > t0 ? end : t0; t < t1; ++t) store_any<VW>(view_at<T>(a.dx, b, t, c), V{});
        if (piece == 0 && n == 0 && a.dstate != nullptr)
            for (uint32_t j = 0; j + 1 < a.taps; ++j)
                store_any<VW>(static_cast<T*>(a.dstate) + (uint64_t(b) * (a.taps - 1) + j) * a.channels + c, V{});
    }
    // over the workgroup's stretches, one tap after the other
    float* out = a.partial + uint64_t(row) * (a.taps + 1) * a.channels;
#pragma unroll
    for (int k = 0; k <= KT; ++k) {
        if (uint32_t(k) < skip) continue;
        const FVec<VW> own = k < KT ? dw[k < KT ? k : 0] : db;
        if (sub < subs)
#pragma unroll
            for (int v = 0; v < VW; ++v) sums[(sub * VW + v) * per + lane] = own[v];
        __syncthreads();
        if (sub == 0 && r < a.lanes) {
            FVec<VW> total = 0.f;
            for (uint32_t j = 0; j < subs; ++j)
#pragma unroll
                for (int v = 0; v < VW; ++v) total[v] += sums[(j * VW + v) * per + lane];
            store_any<VW>(out + uint64_t(k - skip) * a.channels + c, total);
        }
        __syncthreads();
    }
}

// Partial rows joined: dweight [channels][taps] and dbias.  64 threads an element.
__global__ __launch_bounds__(1024) void k_conv_weight_grad(const float* partial, uint32_t rows, uint32_t taps,
                                                           uint32_t channels, float* dweight, float* dbias) {
    __shared__ double part[64][17];
    const uint32_t lane = threadIdx.x % 16, sub = threadIdx.x / 16;
    const uint32_t c = blockIdx.x * 16 + lane, k = blockIdx.y;
    double s = 0.0;
    if (c < channels)
#pragma unroll 4
        for (uint32_t i = sub; i < rows; i += 64) s += partial[(uint64_t(i) * (taps + 1) + k) * channels + c];
    part[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || c >= channels) return;
    for (uint32_t j = 1; j < 64; ++j) s += part[j][lane];
    if (k < taps) dweight[uint64_t(c) * taps + k] = float(s);
    else if (dbias != nullptr) dbias[c] = float(s);
}

}  // namespace adacomp
