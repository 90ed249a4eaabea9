// Gradient norm and AdamW kernels for gfx950, over every tensor of a table in
// one launch.
//
// Per element, with the gradient's factor f (scale, times the clip factor):
//   g = f * grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   w = w * keep - size * (m / (sqrt(v) * rbc2 + eps))
// keep = 1 - lr_i wd_i, size = lr_i / (1 - b1^t), rbc2 = 1 / sqrt(1 - b2^t).
//
// About 15 operations per 28 bytes (float32 moments, float32 gradient) or 18
// bytes (8-bit moments with the bf16 copy): memory bounds it.  A work tile is
// 4096 elements of one tensor, 256 threads with four vectors of four elements
// each, all of a tile's loads requested before the first is used.
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
    double lr, inv_bc1;  // inv_bc1 = 1 / (1 - beta1^t)
    double beta1, beta2, omb1, omb2;
    float rbc2, eps, scale;
    uint32_t key;        // hash of seed and step
};

template <typename G>
__device__ __forceinline__ f32x4 load_grad(const void* grad, uint64_t e) {
    typedef typename Packed<G, 4>::V V;
    return to_float<4, G>(*reinterpret_cast<const V*>(static_cast<const G*>(grad) + e));
}

// Four consecutive elements to memory, those below `left`.
template <typename T, typename V>
__device__ __forceinline__ void store_part(T* p, V v, int left) {
    if (left >= 4) {
        *reinterpret_cast<V*>(p) = v;
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < left) p[c] = v[c];
    }
}

// ---- norm ----

// One float64 partial sum of squares per workgroup: squares of float32 values
// are exact in float64, each thread adds its own in tile order, the workgroup
// joins its threads in a fixed order.
template <typename G>
__global__ __launch_bounds__(256) void
k_grad_norm(const OptTile* __restrict__ tiles, uint32_t ntiles, const void* __restrict__ grad,
            double* __restrict__ partial) {
    const int tid = threadIdx.x;
    double sum = 0.0;
    for (uint32_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
        const OptTile tile = tiles[t];
        f32x4 g[kOptVecs];
#pragma unroll
        for (int j = 0; j < int(kOptVecs); ++j) {
            const int e = (j * int(kOptThreads) + tid) * 4;
            g[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (e < int(tile.count)) g[j] = load_grad<G>(grad, tile.elem + uint64_t(e));
        }
#pragma unroll
        for (int j = 0; j < int(kOptVecs); ++j) {
            const int left = int(tile.count) - (j * int(kOptThreads) + tid) * 4;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const double x = c < left ? double(g[j][c]) : 0.0;
                sum += x * x;
            }
        }
    }
    __shared__ double part[4];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    if (tid == 0) partial[blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(256) void
k_grad_norm_finish(const double* __restrict__ partial, uint32_t n, double max_norm, double scale,
                   float* __restrict__ clip) {
    const int tid = threadIdx.x;
    double sum = 0.0;
    for (uint32_t i = tid; i < n; i += 256) sum += partial[i];
    __shared__ double part[4];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    if (tid == 0) {
        const double norm = sqrt((part[0] + part[1]) + (part[2] + part[3])) * scale;
        clip[0] = float(norm);
        clip[1] = float(norm > max_norm ? max_norm / norm : 1.0);
    }
}

// ---- float32 moments ----

template <typename G>
__global__ __launch_bounds__(256) void k_adamw(AdamwArgs a) {
    const OptTile tile = a.tiles[blockIdx.x];
    const int tid = threadIdx.x;
    const double lr = a.lr * double(tile.lr_scale);
    const float size = float(lr * a.inv_bc1);
    const float keep = float(1.0 - lr * double(tile.weight_decay));
    const float factor = a.clip ? a.clip[1] * a.scale : a.scale;
    const float b1 = float(a.beta1), b2 = float(a.beta2), omb1 = float(a.omb1), omb2 = float(a.omb2);
    float* m = static_cast<float*>(a.m);
    float* v = static_cast<float*>(a.v);
    f32x4 w4[kOptVecs], g4[kOptVecs], m4[kOptVecs], v4[kOptVecs];
#pragma unroll
    for (int j = 0; j < int(kOptVecs); ++j) {
        const int e = (j * int(kOptThreads) + tid) * 4;
        if (e < int(tile.count)) {   // the padding of a last vector is readable
            const uint64_t at = tile.elem + uint64_t(e);
            g4[j] = load_grad<G>(a.grad, at);
            w4[j] = load4<false>(a.w + at);
            m4[j] = load4<false>(m + at);
            v4[j] = load4<false>(v + at);
        }
    }
#pragma unroll
    for (int j = 0; j < int(kOptVecs); ++j) {
        const int e = (j * int(kOptThreads) + tid) * 4;
        const int left = int(tile.count) - e;
        if (left <= 0) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float g = g4[j][c] * factor;
            m4[j][c] = __builtin_fmaf(b1, m4[j][c], omb1 * g);
            v4[j][c] = __builtin_fmaf(b2, v4[j][c], omb2 * (g * g));
            const float denom = __builtin_fmaf(sqrtf(v4[j][c]), a.rbc2, a.eps);
            w4[j][c] = __builtin_fmaf(w4[j][c], keep, -size * (m4[j][c] / denom));
        }
        const uint64_t at = tile.elem + uint64_t(e);
        store_part(a.w + at, w4[j], left);
        store_part(m + at, m4[j], left);
        store_part(v + at, v4[j], left);
        if (a.w16) store_part(a.w16 + at, from_float<bf16, 4>(w4[j]), left);
    }
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

// Largest value of the 8 lanes that share a moment block.
__device__ __forceinline__ int max_of_8_lanes(int v) {
    v = max(v, int(dpp_u32<0xB1>(0u, uint32_t(v))));    // lane ^ 1
    v = max(v, int(dpp_u32<0x4E>(0u, uint32_t(v))));    // lane ^ 2
    v = max(v, int(dpp_u32<0x141>(0u, uint32_t(v))));   // mirrored in 8: the other quad
    return v;
}

// The biased scale of a block whose largest magnitude has the high word
// `top`: the smallest exponent under which that magnitude, cut to 20 fraction
// bits, is at most 448 = 1.75 * 2^8.
__device__ __forceinline__ int block_scale(int top) {
    const int exponent = ((top + 0x3FFFF) >> 20) - 1023 - 8;
    return min(max(exponent + 127, 0), 254);
}

// e4m3 code of magnitude |x| * up, rounded up with the probability of its
// remainder: a code is the top of the value's bits (rebiased), so adding a
// random number to the 17 bits below it carries into it that often.  Below
// 2^-6 codes count steps of 2^-9; adding 2^-6 gives those values the exponent
// whose step that is.  Values past 448, infinities and NaN become the NaN code.
__device__ __forceinline__ uint32_t e4m3_code(double x, double up, uint32_t random16) {
    double u = fabs(x) * up;
    const bool small = u < 0x1p-6;
    u = small ? u + 0x1p-6 : u;
    int code = ((high_word(u) + int(2u * random16 + 1u)) >> 17) - (1023 - 7) * 8;
    code -= small ? 8 : 0;
    return uint32_t(min(code, 0x7F));
}

template <typename G>
__global__ __launch_bounds__(256) void k_adamw_packed(AdamwArgs a) {
    const OptTile tile = a.tiles[blockIdx.x];
    const int tid = threadIdx.x;
    const double lr = a.lr * double(tile.lr_scale);
    const float size = float(lr * a.inv_bc1);
    const float keep = float(1.0 - lr * double(tile.weight_decay));
    const double factor = a.clip ? double(a.clip[1]) * double(a.scale) : double(a.scale);
    uint8_t* mc = static_cast<uint8_t*>(a.m);
    uint8_t* vc = static_cast<uint8_t*>(a.v);
    f32x4 w4[kOptVecs], g4[kOptVecs];
    uint32_t m4[kOptVecs], v4[kOptVecs], s2[kOptVecs];
#pragma unroll
    for (int j = 0; j < int(kOptVecs); ++j) {
        const int e = (j * int(kOptThreads) + tid) * 4;
        g4[j] = w4[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        m4[j] = v4[j] = s2[j] = 0;
        if (e < int(tile.count)) {   // the padding of a last vector is readable
            const uint64_t at = tile.elem + uint64_t(e);
            g4[j] = load_grad<G>(a.grad, at);
            w4[j] = load4<false>(a.w + at);
            m4[j] = *reinterpret_cast<const uint32_t*>(mc + at);
            v4[j] = *reinterpret_cast<const uint32_t*>(vc + at);
            s2[j] = *reinterpret_cast<const uint16_t*>(a.scales + 2 * (tile.block + uint64_t(e) / ADACOMP_MOMENT_BLOCK));
        }
    }
    // the hash of an element's index: its low word mixed with one key per high word
    const uint32_t high0 = uint32_t(tile.elem >> 32);
    const uint32_t key0 = fmix32(a.key ^ (high0 * 0x9E3779B9u));
    const uint32_t key1 = fmix32(a.key ^ ((high0 + 1u) * 0x9E3779B9u));
#pragma unroll
    for (int j = 0; j < int(kOptVecs); ++j) {
        const int e = (j * int(kOptThreads) + tid) * 4;
        const int left = int(tile.count) - e;
        const uint64_t at = tile.elem + uint64_t(e);
        const uint32_t key = uint32_t(at >> 32) == high0 ? key0 : key1;
        const double m_scale = power_of_two(int(s2[j] & 0xFFu) - 127);
        const double v_scale = power_of_two(int(s2[j] >> 8) - 127);
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 mlo = __builtin_amdgcn_cvt_pk_f32_fp8(int(m4[j]), false);
        const f32x2 mhi = __builtin_amdgcn_cvt_pk_f32_fp8(int(m4[j]), true);
        const f32x2 vlo = __builtin_amdgcn_cvt_pk_f32_fp8(int(v4[j]), false);
        const f32x2 vhi = __builtin_amdgcn_cvt_pk_f32_fp8(int(v4[j]), true);
        double m[4] = {mlo[0], mlo[1], mhi[0], mhi[1]}, v[4] = {vlo[0], vlo[1], vhi[0], vhi[1]};
        int mtop = 0, vtop = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            // in float64: the rounding to 8 bits must not hang on the order of a sum
            const double g = double(g4[j][c]) * factor;
            m[c] = a.beta1 * (m[c] * m_scale) + a.omb1 * g;
            v[c] = a.beta2 * (v[c] * v_scale) + a.omb2 * (g * g);
            if (c >= left) m[c] = v[c] = 0.0;   // past the tensor's end
            const float denom = __builtin_fmaf(sqrtf(float(v[c])), a.rbc2, a.eps);
            w4[j][c] = __builtin_fmaf(w4[j][c], keep, -size * (float(m[c]) / denom));
            mtop = max(mtop, high_word(m[c]) & 0x7FFFFFFF);
            vtop = max(vtop, high_word(v[c]));
        }
        // every lane takes part: a block's lanes hold 0 past the end
        const int ms = block_scale(max_of_8_lanes(mtop)), vs = block_scale(max_of_8_lanes(vtop));
        const double m_up = power_of_two(127 - ms), v_up = power_of_two(127 - vs);
        uint32_t mcode = 0, vcode = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t bits = fmix32((uint32_t(at) + uint32_t(c)) ^ key);
            uint32_t code = e4m3_code(m[c], m_up, bits & 0xFFFFu);
            code |= m[c] < 0.0 ? 0x80u : 0u;
            mcode |= code << (8 * c);
            code = e4m3_code(v[c], v_up, bits >> 16);
            if (v[c] > 0.0 && code == 0u) code = 1u;   // a second moment above zero stays above
            vcode |= code << (8 * c);
        }
        if (left <= 0) continue;
        store_part(a.w + at, w4[j], left);
        if (a.w16) store_part(a.w16 + at, from_float<bf16, 4>(w4[j]), left);
        if (left >= 4) {
            *reinterpret_cast<uint32_t*>(mc + at) = mcode;
            *reinterpret_cast<uint32_t*>(vc + at) = vcode;
        } else {
            for (int c = 0; c < left; ++c) {
                mc[at + c] = uint8_t(mcode >> (8 * c));
                vc[at + c] = uint8_t(vcode >> (8 * c));
            }
        }
        if (e % int(ADACOMP_MOMENT_BLOCK) == 0)
            *reinterpret_cast<uint16_t*>(a.scales + 2 * (tile.block + uint64_t(e) / ADACOMP_MOMENT_BLOCK)) =
                uint16_t(ms | (vs << 8));
    }
}

}  // namespace adacomp
