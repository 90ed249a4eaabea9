// Gradient norm and AdamW kernels for gfx950, over every tensor of a table in
// one launch.
//
// Per element, with the gradient's factor f (scale, times the clip factor):
//   g = f * grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   w = w * keep - size * (m / (sqrt(v) * rbc2 + eps))
// keep = 1 - lr_i wd_i, size = lr_i / (1 - b1^t), rbc2 = 1 / sqrt(1 - b2^t).
//
// About 15 operations per 28 bytes with float32 moments, about 80 per 18 bytes
// with 8-bit ones (float64 moments, the hash, two quantisations) and the bf16
// copy: memory bounds the first, and the second nearly so.  A work tile is
// 1024 elements of one tensor, 256 threads with one vector of four elements
// each; every buffer is touched once a step, so its accesses are non-temporal.
// 268 M elements with float32 moments take 1.19 ms (6.3 TB/s), 25.2 M with 8-bit
// moments, a bf16 gradient and the bf16 copy 66.2 us (6.1 TB/s).
#pragma once

#include "common.hpp"
#include "elements.hpp"
#include "optimizer_layout.hpp"

namespace adacomp {

struct AdamwArgs {
    const OptTile* tiles;
    float* w;
    const void* grad;
    void* m;
    void* v;
    uint8_t* scales;     // 8-bit moments
    bf16* w16;           // nullable
    const float* clip;   // nullable
    double beta1, beta2, omb1, omb2;
    double lr, inv_bc1;   // inv_bc1 = 1 / (1 - beta1^t)
    float rbc2, eps, scale;
    uint32_t key;        // hash of seed and step
};

template <typename V, bool NT>
__device__ __forceinline__ V load_as(const void* p) {
    if (NT) return __builtin_nontemporal_load(static_cast<const V*>(p));
    return *static_cast<const V*>(p);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Four gradient elements from e on.
template <typename G, bool NT>
__device__ __forceinline__ f32x4 load_grad(const void* grad, uint64_t e) {
    const G* p = static_cast<const G*>(grad) + e;
    if constexpr (sizeof(G) == 4) return load_as<f32x4, NT>(p);
    else return to_float<4, G>(__builtin_bit_cast(typename Packed<G, 4>::V, load_as<u32x2, NT>(p)));
}

// Four consecutive elements to memory, those below `left`.
template <typename T, typename V>
__device__ __forceinline__ void store_part(T* p, V v, int left) {
    if (left >= 4) {
        if constexpr (sizeof(V) == 16) __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
        else __builtin_nontemporal_store(__builtin_bit_cast(u32x2, v), reinterpret_cast<u32x2*>(p));
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < left) p[c] = v[c];
    }
}

// ---- norm ----

// One float64 partial sum of squares per workgroup: squares of float32 values
// are exact in float64, each thread adds its own in tile order, the workgroup
// joins its threads in a fixed order.  One tile at a time and 2048 workgroups:
// 1.07 GB are read at 6.3 TB/s, and at 5.2 to 5.7 with two to eight tiles at
// once, whose addresses lie further apart.
__device__ __forceinline__ double join_256(double sum, int tid) {
    __shared__ double part[4];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

template <typename G>
__global__ __launch_bounds__(256) void
k_grad_norm(const OptTile* __restrict__ tiles, uint32_t ntiles, const void* __restrict__ grad,
            double* __restrict__ partial) {
    const int tid = threadIdx.x;
    double sum = 0.0;
    OptTile tile = tiles[blockIdx.x];   // the grid holds at most one workgroup a tile
    for (uint32_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
        const int left = int(tile.count) - tid * 4;
        f32x4 g = {0.f, 0.f, 0.f, 0.f};
        if (left > 0) g = load_grad<G, false>(grad, tile.elem + uint64_t(tid) * 4);
        tile = tiles[min(t + gridDim.x, ntiles - 1)];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const double x = c < left ? double(g[c]) : 0.0;   // the padding of a last vector does not count
            sum = __builtin_fma(x, x, sum);
        }
    }
    sum = join_256(sum, tid);
    if (tid == 0) partial[blockIdx.x] = sum;
}

__global__ __launch_bounds__(256) void
k_grad_norm_finish(const double* __restrict__ partial, uint32_t n, double max_norm, double scale,
                   float* __restrict__ clip) {
    static_assert(kNormMaxBlocks == 8 * 256, "eight partial sums a thread");
    const int tid = threadIdx.x;
    double p[8], sum = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = uint32_t(j * 256 + tid) < n ? partial[j * 256 + tid] : 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += p[j];
    sum = join_256(sum, tid);
    if (tid == 0) {
        const double norm = sqrt(sum) * scale;
        clip[0] = float(norm);
        clip[1] = float(norm > max_norm ? max_norm / norm : 1.0);
    }
}

// A tile's step size and decay factor, formed in float64 and rounded once: six operations a thread,
// beside 60 and more on its elements.
struct Factors {
    float size, keep;
};
__device__ __forceinline__ Factors tile_factors(const AdamwArgs& a, const OptTile& tile) {
    const double lr = a.lr * double(tile.lr_scale);
    return {float(lr * a.inv_bc1), float(1.0 - lr * double(tile.weight_decay))};
}

// ---- float32 moments ----

template <typename G>
__global__ __launch_bounds__(256) void k_adamw(AdamwArgs a) {
    const OptTile tile = a.tiles[blockIdx.x];
    const int tid = threadIdx.x;
    const Factors f = tile_factors(a, tile);
    const float factor = a.clip ? a.clip[1] * a.scale : a.scale;
    const float b1 = float(a.beta1), b2 = float(a.beta2), omb1 = float(a.omb1), omb2 = float(a.omb2);
    float* m = static_cast<float*>(a.m);
    float* v = static_cast<float*>(a.v);
    const int left = int(tile.count) - tid * 4;
    if (left <= 0) return;
    const uint64_t at = tile.elem + uint64_t(tid) * 4;   // the padding of a last vector is readable
    f32x4 g4 = load_grad<G, true>(a.grad, at), w4 = load4<true>(a.w + at);
    f32x4 m4 = load4<true>(m + at), v4 = load4<true>(v + at);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float g = g4[c] * factor;
        m4[c] = __builtin_fmaf(b1, m4[c], omb1 * g);
        v4[c] = __builtin_fmaf(b2, v4[c], omb2 * (g * g));
        const float denom = __builtin_fmaf(sqrtf(v4[c]), a.rbc2, a.eps);
        w4[c] = __builtin_fmaf(w4[c], f.keep, -f.size * (m4[c] / denom));
    }
    store_part(a.w + at, w4, left);
    store_part(m + at, m4, left);
    store_part(v + at, v4, left);
    if (a.w16) store_part(a.w16 + at, from_float<bf16, 4>(w4), left);
}

// ---- 8-bit moments ----

// The 32-bit finaliser of MurmurHash3 (Appleby, public domain): every input
// bit reaches every output bit.
__host__ __device__ inline uint32_t fmix32(uint32_t h) {
    h ^= h >> 16;
    h *= 0x85EBCA6Bu;
    h ^= h >> 13;
    h *= 0xC2B2AE35u;
    h ^= h >> 16;
    return h;
}

__device__ __forceinline__ int high_word(double x) { return __double2hiint(x); }
// 2^k, k in -1022..1023
__device__ __forceinline__ double power_of_two(int k) { return __hiloint2double((k + 1023) << 20, 0); }

// Largest magnitude, by its high word, of the four values of each of the 8
// lanes that share a moment block.  High words without their sign are in
// magnitude order as float32 patterns too, so the float maximum takes the signs
// off by itself; infinities and NaN are NaN patterns there and drop out: they
// take no part in the scale that their neighbours share.
__device__ __forceinline__ int block_top(const double x[4]) {
    float t = __int_as_float(high_word(x[0])), u;
    asm("v_max3_f32 %0, |%1|, |%2|, |%3|"
        : "=v"(u) : "v"(t), "v"(__int_as_float(high_word(x[1]))), "v"(__int_as_float(high_word(x[2]))));
    asm("v_max_f32_e64 %0, |%1|, |%2|" : "=v"(t) : "v"(u), "v"(__int_as_float(high_word(x[3]))));
    int v = __float_as_int(t);
    v = v > 0x7F800000 ? 0 : v;                         // nothing but infinities and NaN
    v = max(v, int(dpp_u32<0xB1>(0u, uint32_t(v))));    // lane ^ 1
    v = max(v, int(dpp_u32<0x4E>(0u, uint32_t(v))));    // lane ^ 2
    v = max(v, int(dpp_u32<0x141>(0u, uint32_t(v))));   // mirrored in 8: the other quad
    return v;
}

// The biased scale of a block whose largest magnitude, 2^-SHIFT of x, has the
// high word `top`: the smallest exponent under which that magnitude, cut to 20
// fraction bits, is at most 448 = 1.75 * 2^8.
template <int SHIFT>
__device__ __forceinline__ int block_scale(int top) {
    const int exponent = ((top + 0x3FFFF) >> 20) - 1023 - 8 - SHIFT;
    return min(max(exponent + 127, 0), 254);
}

// e4m3 code of magnitude |x| * up, rounded up with the probability of its
// remainder: a code is the top of the value's bits (rebiased), so adding a
// random number to the 17 bits below it carries into it that often.  Below
// 2^-6 codes count steps of 2^-9; adding 2^-6 gives those values the exponent
// whose step that is, 8 codes higher.  Values past 448, infinities and NaN
// become the NaN code.  `random` is 2 * r + 1, r of 16 bits, less the rebiasing.
constexpr int kCodeBias = (1023 - 7) * 8;
__device__ __forceinline__ int e4m3_code(double x, double up, int random) {
    const double u = fabs(x) * up;
    const int sub = high_word(u + 0x1p-6) - (8 << 17);
    const int high = high_word(u) < ((1023 - 6) << 20) ? sub : high_word(u);
    return min((high + random) >> 17, 0x7F);
}

template <typename G>
__global__ __launch_bounds__(256) void k_adamw_packed(AdamwArgs a) {
    const OptTile tile = a.tiles[blockIdx.x];
    const int tid = threadIdx.x;
    const Factors f = tile_factors(a, tile);
    const double factor = a.clip ? double(a.clip[1]) * double(a.scale) : double(a.scale);
    uint8_t* mc = static_cast<uint8_t*>(a.m);
    uint8_t* vc = static_cast<uint8_t*>(a.v);
    const int left = int(tile.count) - tid * 4;
    const uint64_t at = tile.elem + uint64_t(tid) * 4;
    uint8_t* scales = a.scales + 2 * (tile.block + tid / 8);
    f32x4 g4 = {0.f, 0.f, 0.f, 0.f}, w4 = g4;
    uint32_t mcode = 0, vcode = 0, s2 = 0;
    if (left > 0) {
        g4 = load_grad<G, true>(a.grad, at);
        w4 = load4<true>(a.w + at);
        mcode = load_as<uint32_t, true>(mc + at);
        vcode = load_as<uint32_t, true>(vc + at);
        s2 = *reinterpret_cast<const uint16_t*>(scales);
        if (left < 4) {   // the padding of a last vector is readable and counts as 0
            const uint32_t keep_bytes = (1u << (8 * left)) - 1u;
            mcode &= keep_bytes;
            vcode &= keep_bytes;
#pragma unroll
            for (int c = 1; c < 4; ++c) g4[c] = c < left ? g4[c] : 0.f;
        }
    }
    // the hash of an element's index: its low word mixed with one key per high word
    const uint32_t high0 = uint32_t(tile.elem >> 32);
    const uint32_t key0 = fmix32(a.key ^ (high0 * 0x9E3779B9u));
    const uint32_t key1 = fmix32(a.key ^ ((high0 + 1u) * 0x9E3779B9u));
    const uint32_t key = uint32_t(at >> 32) == high0 ? key0 : key1;
    // Moments in float64: the rounding to 8 bits must not hang on the order of a sum.  A power of
    // two moves into a factor without a rounding: the scales into the betas, and 2^kUp into v, under
    // which its float32 root needs no care for subnormal numbers.
    constexpr int kUp = 30;
    const double b1 = a.beta1 * power_of_two(int(s2 & 0xFFu) - 127);
    const double b2 = a.beta2 * power_of_two(int(s2 >> 8) - 127 + kUp), omb2 = a.omb2 * power_of_two(kUp);
    const float rbc2 = a.rbc2 * 0x1p-15f;
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 mlo = __builtin_amdgcn_cvt_pk_f32_fp8(int(mcode), false);
    const f32x2 mhi = __builtin_amdgcn_cvt_pk_f32_fp8(int(mcode), true);
    const f32x2 vlo = __builtin_amdgcn_cvt_pk_f32_fp8(int(vcode), false);
    const f32x2 vhi = __builtin_amdgcn_cvt_pk_f32_fp8(int(vcode), true);
    double m[4] = {mlo[0], mlo[1], mhi[0], mhi[1]}, v[4] = {vlo[0], vlo[1], vhi[0], vhi[1]};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const double g = double(g4[c]) * factor;
        m[c] = b1 * m[c] + a.omb1 * g;
        v[c] = b2 * v[c] + omb2 * (g * g);
    }
    // The weights' step takes the hardware's root and reciprocal, each off by one unit in the last place of
    // a term that is far below the weight: rounded to nearest they are a dozen instructions each
    // (25.2 M elements with a bf16 gradient 73.3 us against 67.6).
    float q[4];
    bool far = false;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float u = float(v[c]);
        far |= u == __builtin_inff();
        q[c] = float(m[c]) * __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_amdgcn_sqrtf(u), rbc2, a.eps));
    }
    // v past 2^(128 - kUp), of gradients past 1e16 or so: root, denominator and m times 2^-65
    if (far) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (float(v[c]) != __builtin_inff()) continue;
            const float root = __builtin_amdgcn_sqrtf(float(v[c] * power_of_two(-130 - kUp)));
            q[c] = float(m[c] * 0x1p-65) * __builtin_amdgcn_rcpf(__builtin_fmaf(root, a.rbc2, a.eps * 0x1p-65f));
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) w4[c] = __builtin_fmaf(w4[c], f.keep, -f.size * q[c]);
    // every lane takes part: a block's lanes hold 0 past the end
    const int ms = block_scale<0>(block_top(m)), vs = block_scale<kUp>(block_top(v));
    const double m_up = power_of_two(127 - ms), v_up = power_of_two(127 - vs - kUp);
    mcode = vcode = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t bits = fmix32((uint32_t(at) + uint32_t(c)) ^ key);
        constexpr int kOffset = 1 - (kCodeBias << 17);
        int code = e4m3_code(m[c], m_up, int((bits << 1) & 0x1FFFEu) + kOffset);
        mcode |= (uint32_t(code) | ((uint32_t(high_word(m[c])) >> 24) & 0x80u)) << (8 * c);
        code = e4m3_code(v[c], v_up, int((bits >> 15) & 0x1FFFEu) + kOffset);
        code = max(code, min(high_word(v[c]) & 0x7FFFFFFF, 1));   // a second moment above zero stays above
        vcode |= uint32_t(code) << (8 * c);
    }
    if (left <= 0) return;
    store_part(a.w + at, w4, left);
    if (a.w16) store_part(a.w16 + at, from_float<bf16, 4>(w4), left);
    if (left >= 4) {
        __builtin_nontemporal_store(mcode, reinterpret_cast<uint32_t*>(mc + at));
        __builtin_nontemporal_store(vcode, reinterpret_cast<uint32_t*>(vc + at));
    } else {
        for (int c = 0; c < left; ++c) {
            mc[at + c] = uint8_t(mcode >> (8 * c));
            vc[at + c] = uint8_t(vcode >> (8 * c));
        }
    }
    if (tid % 8 == 0) *reinterpret_cast<uint16_t*>(scales) = uint16_t(ms | (vs << 8));
}

}  // namespace adacomp
