// Layer norm and its gradients for gfx950.
//
//   y  = (x - mean) * rstd * weight + bias
//   dx = rstd * (g - mean(g) - xhat * mean(g * xhat)),  g = dy * weight
//   dweight = sum over rows of dy * xhat,  dbias = sum over rows of dy
//
// Memory bounds both (7 and 14 operations an element), so a row is read once
// and stays in registers between its statistics and its result.  A row of up
// to 1024 columns belongs to a team of 4 to 64 lanes of one wavefront, which
// joins its sums by lane moves alone; a wider one to a workgroup of one
// wavefront per 1024 columns, joined through LDS; past 16384 columns a
// workgroup reads the row once per pass.
#pragma once

#include "common.hpp"
#include "elements.hpp"

namespace adacomp {

constexpr int kNormElems = 16;                            // most elements of a row per lane
constexpr uint32_t kNormWaveCols = 64 * kNormElems;       // one wavefront's columns
constexpr uint32_t kNormRegCols = 16 * kNormWaveCols;     // a workgroup's
constexpr uint32_t kNormMaxPartials = 1024;               // workgroups of the weight gradients
constexpr uint32_t kNormWideThreads = 1024;

struct NormArgs {
    const void* x;
    const void* dy;
    void* out;             // y or dx
    const float* weight;   // nullable
    const float* bias;     // nullable
    float* mean;           // outputs (nullable) of the forward pass, inputs of the backward pass
    float* rstd;
    float* partial;        // [workgroups][2][cols]; null without dweight and dbias
    uint64_t x_stride, dy_stride, out_stride, rows;
    uint32_t cols;
    float eps, inv_cols;
};

// Sum over teams of LANES adjacent lanes, the same bits in each of them.
template <int LANES>
__device__ __forceinline__ float team_sum(float v) {
    auto moved = [](float x, uint32_t y) { return x + __uint_as_float(y); };
    if (LANES >= 2) v = moved(v, dpp_u32<0xB1>(0u, __float_as_uint(v)));    // lane ^ 1
    if (LANES >= 4) v = moved(v, dpp_u32<0x4E>(0u, __float_as_uint(v)));    // lane ^ 2
    if (LANES >= 8) v = moved(v, dpp_u32<0x141>(0u, __float_as_uint(v)));   // the other quad of 8
    if (LANES >= 16) v = moved(v, dpp_u32<0x140>(0u, __float_as_uint(v)));  // the other 8 of a row
    if (LANES >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if (LANES >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

// Sum over a workgroup's wavefronts (BLOCK) or over one team.  `slot`: 16
// floats of LDS that no earlier sum still reads.
template <int LANES, bool BLOCK>
__device__ __forceinline__ float row_sum(float v, float* slot) {
    v = team_sum<LANES>(v);
    if (BLOCK) {
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
        for (uint32_t i = 0; i < blockDim.x / 64; ++i) v += slot[i];
    }
    return v;
}

template <typename T>
constexpr int norm_vec() {
    return 16 / int(sizeof(T));
}

// VEC elements from column c on as float, 0 past the row's end.
template <typename T, int VEC>
__device__ __forceinline__ FVec<VEC> load_cols(const T* row, uint32_t c, uint32_t cols) {
    if (c + VEC <= cols) return to_float<VEC, T>(load_any<VEC>(row + c));
    FVec<VEC> v = 0.f;
#pragma unroll
    for (int k = 0; k < VEC; ++k)
        if (c + k < cols) v[k] = float(row[c + k]);
    return v;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_cols(T* row, uint32_t c, uint32_t cols, FVec<VEC> v) {
    const typename Packed<T, VEC>::V o = from_float<T, VEC>(v);
    if (c + VEC <= cols) {
        store_any<VEC>(row + c, o);
        return;
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k)
        if (c + k < cols) row[c + k] = o[k];
}

// ---- forward ----

template <typename T, int NV, int LANES, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void k_layer_norm(NormArgs a) {
    constexpr int VEC = norm_vec<T>();
    const uint32_t team = BLOCK ? blockDim.x : LANES;
    const uint32_t lane = BLOCK ? threadIdx.x : threadIdx.x % LANES;
    const uint64_t row = BLOCK ? blockIdx.x : uint64_t(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
    const bool live = BLOCK || row < a.rows;   // all lanes take part in the sums
    __shared__ float slots[2][16];
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    FVec<VEC> v[NV];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        v[j] = 0.f;
        if (live) v[j] = load_cols<T, VEC>(x, (j * team + lane) * VEC, a.cols);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum += v[j][k];
    const float mean = row_sum<LANES, BLOCK>(sum, slots[0]) * a.inv_cols;
    float square = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const bool in = (j * team + lane) * VEC + k < a.cols;
            v[j][k] = in ? v[j][k] - mean : 0.f;
            square = __builtin_fmaf(v[j][k], v[j][k], square);
        }
    const float var = row_sum<LANES, BLOCK>(square, slots[1]) * a.inv_cols;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (!live) return;
    T* y = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t c = (j * team + lane) * VEC;
        if (c >= a.cols) continue;
        FVec<VEC> w = 1.f, b = 0.f;
        if (a.weight) w = load_cols<float, VEC>(a.weight, c, a.cols);
        if (a.bias) b = load_cols<float, VEC>(a.bias, c, a.cols);
        FVec<VEC> o;
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = __builtin_fmaf(v[j][k] * rstd, w[k], b[k]);
        store_cols<T, VEC>(y, c, a.cols, o);
    }
    if (lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// Rows past kNormRegCols columns: one workgroup a row, read once per pass.
template <typename T>
__global__ __launch_bounds__(kNormWideThreads) void k_layer_norm_wide(NormArgs a) {
    constexpr int VEC = norm_vec<T>();
    __shared__ float slots[2][16];
    const uint64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    float sum = 0.f;
    for (uint32_t c = threadIdx.x * VEC; c < a.cols; c += kNormWideThreads * VEC) {
        const FVec<VEC> v = load_cols<T, VEC>(x, c, a.cols);
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum += v[k];
    }
    const float mean = row_sum<64, true>(sum, slots[0]) * a.inv_cols;
    float square = 0.f;
    for (uint32_t c = threadIdx.x * VEC; c < a.cols; c += kNormWideThreads * VEC) {
        const FVec<VEC> v = load_cols<T, VEC>(x, c, a.cols);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float d = c + k < a.cols ? v[k] - mean : 0.f;
            square = __builtin_fmaf(d, d, square);
        }
    }
    const float var = row_sum<64, true>(square, slots[1]) * a.inv_cols;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    T* y = static_cast<T*>(a.out) + row * a.out_stride;
    for (uint32_t c = threadIdx.x * VEC; c < a.cols; c += kNormWideThreads * VEC) {
        const FVec<VEC> v = load_cols<T, VEC>(x, c, a.cols);
        FVec<VEC> w = 1.f, b = 0.f, o;
        if (a.weight) w = load_cols<float, VEC>(a.weight, c, a.cols);
        if (a.bias) b = load_cols<float, VEC>(a.bias, c, a.cols);
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = __builtin_fmaf((v[k] - mean) * rstd, w[k], b[k]);
        store_cols<T, VEC>(y, c, a.cols, o);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// ---- backward ----

// Each team steps over rows and adds its columns' share of dweight and dbias
// in registers; the workgroup's teams are joined in LDS in team order and
// written as one partial row pair, which k_norm_weight_grad adds up.
template <typename T, int NV, int LANES, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void k_layer_norm_backward(NormArgs a) {
    constexpr int VEC = norm_vec<T>();
    constexpr uint32_t TEAMS = BLOCK ? 1 : 256 / LANES;
    const uint32_t team = BLOCK ? blockDim.x : LANES;
    const uint32_t lane = BLOCK ? threadIdx.x : threadIdx.x % LANES;
    const uint32_t mine = BLOCK ? 0 : threadIdx.x / LANES;
    __shared__ float slots[4][16];
    __shared__ float joined[BLOCK ? 1 : 2 * 256 * NV * VEC];
    FVec<VEC> w[NV], dw[NV], db[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t c = (j * team + lane) * VEC;
        dw[j] = db[j] = 0.f;
        w[j] = 1.f;
        if (a.weight) w[j] = load_cols<float, VEC>(a.weight, c, a.cols);
    }
    uint32_t turn = 0;
    for (uint64_t r0 = uint64_t(blockIdx.x) * TEAMS; r0 < a.rows; r0 += uint64_t(gridDim.x) * TEAMS) {
        const uint64_t row = r0 + mine;
        const bool live = row < a.rows;
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
        FVec<VEC> h[NV], g[NV];
        float mean = 0.f, rstd = 0.f;
        if (live) {
            mean = a.mean[row];
            rstd = a.rstd[row];
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * team + lane) * VEC;
            h[j] = g[j] = 0.f;
            if (live) {
                h[j] = load_cols<T, VEC>(x, c, a.cols);
                g[j] = load_cols<T, VEC>(dy, c, a.cols);
            }
        }
        float sum = 0.f, along = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                // past the row's end dy is 0: xhat does not count there
                h[j][k] = (h[j][k] - mean) * rstd;
                dw[j][k] = __builtin_fmaf(g[j][k], h[j][k], dw[j][k]);
                db[j][k] += g[j][k];
                g[j][k] *= w[j][k];
                sum += g[j][k];
                along = __builtin_fmaf(g[j][k], h[j][k], along);
            }
        const float c1 = row_sum<LANES, BLOCK>(sum, slots[turn]) * a.inv_cols;
        const float c2 = row_sum<LANES, BLOCK>(along, slots[turn + 1]) * a.inv_cols;
        turn ^= 2;   // a slot is written again two barriers after its last reader
        if (!live) continue;
        T* dx = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * team + lane) * VEC;
            if (c >= a.cols) continue;
            FVec<VEC> o;
#pragma unroll
            for (int k = 0; k < VEC; ++k) o[k] = rstd * (g[j][k] - c1 - h[j][k] * c2);
            store_cols<T, VEC>(dx, c, a.cols, o);
        }
    }
    if (a.partial == nullptr) return;
    float* out = a.partial + uint64_t(blockIdx.x) * 2 * a.cols;
    if (BLOCK) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * team + lane) * VEC;
            store_cols<float, VEC>(out, c, a.cols, dw[j]);
            store_cols<float, VEC>(out + a.cols, c, a.cols, db[j]);
        }
        return;
    }
    constexpr uint32_t SPAN = LANES * NV * VEC;   // columns a team holds
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const uint32_t c = (j * LANES + lane) * VEC + k;
            joined[mine * SPAN + c] = dw[j][k];
            joined[(TEAMS + mine) * SPAN + c] = db[j][k];
        }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < 2 * SPAN; i += 256) {
        const uint32_t which = i / SPAN, c = i % SPAN;
        if (c >= a.cols) continue;
        float s = 0.f;
        for (uint32_t t = 0; t < TEAMS; ++t) s += joined[(which * TEAMS + t) * SPAN + c];
        out[which * a.cols + c] = s;
    }
}

// Rows past kNormRegCols columns.
template <typename T>
__global__ __launch_bounds__(kNormWideThreads) void k_layer_norm_backward_wide(NormArgs a) {
    constexpr int VEC = norm_vec<T>();
    __shared__ float slots[2][16];
    const uint64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    T* dx = static_cast<T*>(a.out) + row * a.out_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float sum = 0.f, along = 0.f;
    for (uint32_t c = threadIdx.x * VEC; c < a.cols; c += kNormWideThreads * VEC) {
        const FVec<VEC> h = load_cols<T, VEC>(x, c, a.cols);
        FVec<VEC> g = load_cols<T, VEC>(dy, c, a.cols);
        if (a.weight) g *= load_cols<float, VEC>(a.weight, c, a.cols);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            sum += g[k];
            along = __builtin_fmaf(g[k], (h[k] - mean) * rstd, along);
        }
    }
    const float c1 = row_sum<64, true>(sum, slots[0]) * a.inv_cols;
    const float c2 = row_sum<64, true>(along, slots[1]) * a.inv_cols;
    for (uint32_t c = threadIdx.x * VEC; c < a.cols; c += kNormWideThreads * VEC) {
        const FVec<VEC> h = load_cols<T, VEC>(x, c, a.cols);
        FVec<VEC> g = load_cols<T, VEC>(dy, c, a.cols), o;
        if (a.weight) g *= load_cols<float, VEC>(a.weight, c, a.cols);
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = rstd * (g[k] - c1 - (h[k] - mean) * rstd * c2);
        store_cols<T, VEC>(dx, c, a.cols, o);
    }
}

// Their partial weight gradients: workgroup (x, y) adds rows y, y + gridDim.y,
// ... of 256 columns.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_partial_wide(NormArgs a) {
    const uint32_t c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.cols) return;
    float dw = 0.f, db = 0.f;
    for (uint64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float g = float(static_cast<const T*>(a.dy)[row * a.dy_stride + c]);
        const float h = (float(static_cast<const T*>(a.x)[row * a.x_stride + c]) - a.mean[row]) * a.rstd[row];
        dw = __builtin_fmaf(g, h, dw);
        db += g;
    }
    float* out = a.partial + uint64_t(blockIdx.y) * 2 * a.cols;
    out[c] = dw;
    out[a.cols + c] = db;
}

// dweight (blockIdx.y 0) and dbias (1) from the n partial rows: 64 columns by
// 16 groups of partial rows, in float64, joined in group order.
__global__ __launch_bounds__(1024) void
k_norm_weight_grad(const float* __restrict__ partial, uint32_t n, uint32_t cols, float* __restrict__ dweight,
                   float* __restrict__ dbias) {
    __shared__ double part[16][64];
    const uint32_t lane = threadIdx.x & 63, group = threadIdx.x >> 6;
    const uint32_t c = blockIdx.x * 64 + lane;
    double sum = 0.0;
    if (c < cols) {
        const float* p = partial + uint64_t(blockIdx.y) * cols + c;
#pragma unroll 4
        for (uint32_t i = group; i < n; i += 16) sum += double(p[uint64_t(i) * 2 * cols]);
    }
    part[group][lane] = sum;
    __syncthreads();
    if (group == 0 && c < cols) {
        sum = 0.0;
        for (int i = 0; i < 16; ++i) sum += part[i][lane];
        (blockIdx.y ? dbias : dweight)[c] = float(sum);
    }
}

}  // namespace adacomp
