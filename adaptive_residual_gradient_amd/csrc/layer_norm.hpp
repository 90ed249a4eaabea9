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
// workgroup reads the row once per pass.  16384 x 4096 bf16 takes 47 us (5.7
// TB/s), the gradients of 32768 x 1024 bf16 34.2 us (6.0 TB/s) and 4.8 us for
// the weight's partial rows.
#pragma once

#include "common.hpp"
#include "elements.hpp"

namespace adacomp {

constexpr int kNormElems = 16;                            // most elements of a row per lane
constexpr uint32_t kNormWaveCols = 64 * kNormElems;       // one wavefront's columns
constexpr uint32_t kNormRegCols = 16 * kNormWaveCols;     // a workgroup's
constexpr uint32_t kNormMaxWaves = 4096;                  // wavefronts of a forward launch
constexpr uint32_t kNormBackRegCols = 8 * kNormWaveCols;
constexpr uint32_t kNormMaxPartials = 256;                // workgroups of the weight gradients
constexpr uint32_t kNormWideThreads = 1024;
constexpr uint32_t kNormBackThreads = 512;                // most threads of a workgroup there

// What a call leaves to the 256 MB cache in front of the memory, the rest going past it by
// non-temporal accesses: its inputs, which the call before has just written, where they are at most
// kKeepBytes, else its output where that is.  Inputs kept against nothing kept: 4099 x 1000
// float32 gradient 14.6 us and 17.0, 32768 x 1024 bf16 21.6 and 24.9, but 16384 x 4096 bf16 52.0 and
// 48.3; the output kept: 32768 x 1024 bf16 gradient 38.9 us and 40.9.
constexpr int kNormKeepNone = 0, kNormKeepIn = 1, kNormKeepOut = 2;

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

// A thread's columns.  Vector j covers VEC columns from at[j] on, and at[j]
// never reaches past the row: where the columns are no multiple of the team's,
// the last vectors move back over columns that other lanes hold too.  Loads and
// results need no care then (both lanes form the same bits); sums leave the
// first skip[j] elements of a vector out.  Needs cols >= VEC.
template <int VEC, int NV>
struct NormCols {
    uint32_t at[NV];
    int skip[NV];
    bool ragged;   // some lane of the wavefront has elements to leave out
    __device__ NormCols(uint32_t cols, uint32_t lane, uint32_t team) {
        bool any = false;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * team + lane) * VEC;
            at[j] = min(c, cols - VEC);
            skip[j] = int(c - at[j]);
            any |= skip[j] > 0;
        }
        ragged = __any(any);
    }
};

// Weight or bias, which every row reads.
template <int VEC>
__device__ __forceinline__ FVec<VEC> load_param(const float* p, uint32_t c, float absent) {
    FVec<VEC> v = absent;
    if (p != nullptr) v = load_any<VEC>(p + c);
    return v;
}

// The thread's team of `team` lanes.  Whole wavefronts' is told to be the same in
// every lane, so that its rows' addresses and statistics take scalar registers.
template <int LANES>
__device__ __forceinline__ uint32_t team_index(uint32_t team) {
    const uint32_t i = threadIdx.x / team;
    return LANES == 64 ? uint32_t(__builtin_amdgcn_readfirstlane(int(i))) : i;
}

// ---- forward ----

// The next row is requested before the present one is joined; weight and bias
// stay in registers over a workgroup's rows (read anew for each row they are
// four times a 16-bit row's bytes).
template <typename T, int VEC, int NV, int LANES, bool BLOCK, int KEEP>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void k_layer_norm(NormArgs a) {
    typedef typename Packed<T, VEC>::V V;
    constexpr uint32_t TEAMS = BLOCK ? 1 : 256 / LANES;
    const uint32_t team = BLOCK ? blockDim.x : LANES, lane = threadIdx.x % team;
    const uint32_t mine = BLOCK ? 0 : team_index<LANES>(LANES);
    const NormCols<VEC, NV> cols(a.cols, lane, team);
    __shared__ float slots[2][16];
    FVec<VEC> w[NV], b[NV];
    V next[NV];
    auto request = [&](uint64_t row) {   // past the last row: the last row again
        const T* x = static_cast<const T*>(a.x) + min(row, a.rows - 1) * a.x_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) next[j] = load_hint<VEC, KEEP != kNormKeepIn>(x + cols.at[j]);
    };
    const uint64_t step = uint64_t(gridDim.x) * TEAMS;
    request(uint64_t(blockIdx.x) * TEAMS + mine);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        w[j] = load_param<VEC>(a.weight, cols.at[j], 1.f);
        b[j] = load_param<VEC>(a.bias, cols.at[j], 0.f);
    }
    for (uint64_t r0 = uint64_t(blockIdx.x) * TEAMS; r0 < a.rows; r0 += step) {
        const uint64_t row = r0 + mine;
        FVec<VEC> v[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = to_float<VEC, T>(next[j]);
        if (r0 + step < a.rows) request(row + step);
        float sum = 0.f, square = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < VEC; ++k) sum += cols.ragged && k < cols.skip[j] ? 0.f : v[j][k];
        // all lanes take part in the sums, those without a row too; the two sums' barriers keep
        // each slot until all have read it
        const float mean = row_sum<LANES, BLOCK>(sum, slots[0]) * a.inv_cols;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                v[j][k] -= mean;
                const float d = cols.ragged && k < cols.skip[j] ? 0.f : v[j][k];
                square = __builtin_fmaf(d, d, square);
            }
        const float var = row_sum<LANES, BLOCK>(square, slots[1]) * a.inv_cols;
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (row >= a.rows) continue;
        T* y = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            FVec<VEC> o;
#pragma unroll
            for (int k = 0; k < VEC; ++k) o[k] = __builtin_fmaf(v[j][k] * rstd, w[j][k], b[j][k]);
            if (cols.skip[j] < VEC) store_hint<VEC, KEEP != kNormKeepOut>(y + cols.at[j], from_float<T, VEC>(o));
        }
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// Rows past kNormRegCols columns: one workgroup a row, read once per pass.
template <typename T, int VEC, typename F>
__device__ __forceinline__ void each_vector(uint32_t cols, F f) {
    for (uint32_t c = threadIdx.x * VEC; c < cols; c += kNormWideThreads * VEC) {
        const uint32_t at = min(c, cols - VEC);
        f(at, int(c - at));
    }
}

template <typename T>
__global__ __launch_bounds__(kNormWideThreads) void k_layer_norm_wide(NormArgs a) {
    constexpr int VEC = norm_vec<T>();
    __shared__ float slots[2][16];
    const uint64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    float sum = 0.f, square = 0.f;
    each_vector<T, VEC>(a.cols, [&](uint32_t at, int skip) {
        const FVec<VEC> v = to_float<VEC, T>(load_any<VEC>(x + at));
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum += k < skip ? 0.f : v[k];
    });
    const float mean = row_sum<64, true>(sum, slots[0]) * a.inv_cols;
    each_vector<T, VEC>(a.cols, [&](uint32_t at, int skip) {
        const FVec<VEC> v = to_float<VEC, T>(load_any<VEC>(x + at));
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float d = k < skip ? 0.f : v[k] - mean;
            square = __builtin_fmaf(d, d, square);
        }
    });
    const float var = row_sum<64, true>(square, slots[1]) * a.inv_cols;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    T* y = static_cast<T*>(a.out) + row * a.out_stride;
    each_vector<T, VEC>(a.cols, [&](uint32_t at, int) {
        const FVec<VEC> v = to_float<VEC, T>(load_any<VEC>(x + at));
        const FVec<VEC> w = load_param<VEC>(a.weight, at, 1.f), b = load_param<VEC>(a.bias, at, 0.f);
        FVec<VEC> o;
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = __builtin_fmaf((v[k] - mean) * rstd, w[k], b[k]);
        store_any<VEC>(y + at, from_float<T, VEC>(o));
    });
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// ---- backward ----

// Each team steps over rows and adds its columns' share of dweight and dbias
// in registers; the workgroup's teams are joined in LDS in team order and
// written as one partial row pair, which k_norm_weight_grad adds up.  The
// next row is requested before the present one is joined (two rows ahead
// measured the same), and the weight waits in LDS; it is 0
// there in columns that another lane holds, which takes them out of the row's
// sums.  A team is LANES lanes of a wavefront or, BLOCK, one wavefront per 1024
// columns; a workgroup holds as many teams as kNormBackThreads lets it, for every
// workgroup costs a partial row pair.
template <typename T, int VEC, int NV, int LANES, bool BLOCK, int KEEP>
__global__ __launch_bounds__(kNormBackThreads) void k_layer_norm_backward(NormArgs a) {
    typedef typename Packed<T, VEC>::V V;
    const uint32_t waves = (a.cols + kNormWaveCols - 1) / kNormWaveCols;   // a team's, with BLOCK
    const uint32_t team = BLOCK ? waves * 64 : LANES, teams = blockDim.x / team;
    const uint32_t mine = team_index<LANES>(team), lane = threadIdx.x - mine * team;
    const NormCols<VEC, NV> cols(a.cols, lane, team);
    extern __shared__ float dynamic[];   // the weight and two sets of row sums, then the teams' sums
    const uint32_t span = team * NV * VEC;
    FVec<VEC> dw[NV], db[NV];
    struct Row {
        V x[NV], g[NV];
        float mean, rstd;
    } next;
    // The statistics take vector loads, in order with the row's: scalar ones would be waited for with
    // the weight's LDS reads, a row too early.
    uint32_t zero;
    asm("v_mov_b32 %0, 0" : "=v"(zero));
    auto request = [&](uint64_t row) {   // past the last row: the last row again
        const uint64_t r = min(row, a.rows - 1);
        next.mean = a.mean[r + zero];
        next.rstd = a.rstd[r + zero];
        const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
        const T* dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            next.x[j] = load_hint<VEC, KEEP != kNormKeepIn>(x + cols.at[j]);
            next.g[j] = load_hint<VEC, KEEP != kNormKeepIn>(dy + cols.at[j]);
        }
        if ((LANES < 64 || BLOCK) && row >= a.rows) {   // a team without a row beside teams that have one
            next.mean = next.rstd = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) next.x[j] = next.g[j] = V{};
        }
    };
    const uint64_t step = uint64_t(gridDim.x) * teams, first = uint64_t(blockIdx.x) * teams;
    request(first + mine);
    FVec<VEC>* wl = reinterpret_cast<FVec<VEC>*>(dynamic) + lane;   // vector j at wl[j * team]
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        dw[j] = db[j] = 0.f;
        FVec<VEC> w = load_param<VEC>(a.weight, cols.at[j], 1.f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] = k < cols.skip[j] ? 0.f : w[k];
        if (threadIdx.x < team) wl[j * team] = w;
    }
    __syncthreads();
    uint32_t turn = 0;
    for (uint64_t r0 = first; r0 < a.rows; r0 += step) {
        const uint64_t row = r0 + mine;
        if (LANES == 64 && !BLOCK && row >= a.rows) break;
        const float mean = next.mean, rstd = next.rstd;
        FVec<VEC> h[NV], g[NV];
        float sum = 0.f, along = 0.f;
        asm volatile("" ::: "memory");   // the weight stays in LDS, not in registers across rows
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            h[j] = to_float<VEC, T>(next.x[j]);
            g[j] = to_float<VEC, T>(next.g[j]);
        }
        if (r0 + step < a.rows) request(row + step);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const FVec<VEC> w = wl[j * team];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                h[j][k] = (h[j][k] - mean) * rstd;
                dw[j][k] = __builtin_fmaf(g[j][k], h[j][k], dw[j][k]);
                db[j][k] += g[j][k];
                g[j][k] *= w[k];
                sum += g[j][k];
                along = __builtin_fmaf(g[j][k], h[j][k], along);
            }
        }
        sum = team_sum<LANES>(sum);
        along = team_sum<LANES>(along);
        if (BLOCK) {
            float* slot = dynamic + span + turn;
            turn ^= 2 * kNormBackThreads / 64;   // a set is written again a barrier after its last reader
            if ((threadIdx.x & 63) == 0) {
                slot[threadIdx.x >> 6] = sum;
                slot[kNormBackThreads / 64 + (threadIdx.x >> 6)] = along;
            }
            __syncthreads();
            sum = along = 0.f;
            for (uint32_t i = mine * waves; i < (mine + 1) * waves; ++i) {
                sum += slot[i];
                along += slot[kNormBackThreads / 64 + i];
            }
        }
        if (row >= a.rows) continue;
        const float c1 = sum * a.inv_cols, c2 = along * a.inv_cols;
        T* dx = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            FVec<VEC> o;
#pragma unroll
            for (int k = 0; k < VEC; ++k) o[k] = rstd * (g[j][k] - c1 - h[j][k] * c2);
            const V out = from_float<T, VEC>(o);
            if (cols.skip[j] == 0) {
                store_hint<VEC, KEEP != kNormKeepOut>(dx + cols.at[j], out);
            } else {
#pragma unroll
                for (int k = 1; k < VEC; ++k)
                    if (k >= cols.skip[j]) dx[cols.at[j] + k] = out[k];
            }
        }
    }
    if (a.partial == nullptr) return;
    float* out = a.partial + uint64_t(blockIdx.x) * 2 * a.cols;
    // Whole vectors at their places of a row without moved-back ones, 16 bytes a lane; those that were
    // moved back are found there again.
    __syncthreads();   // the weight has been read
    FVec<VEC>* sums = reinterpret_cast<FVec<VEC>*>(dynamic) + lane;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        sums[mine * (span / VEC) + j * team] = dw[j];
        sums[(teams + mine) * (span / VEC) + j * team] = db[j];
    }
    __syncthreads();
    const uint32_t whole = a.cols / VEC * VEC;   // columns of vectors in their own place
    for (uint32_t i = threadIdx.x; i < 2 * a.cols; i += blockDim.x) {
        const uint32_t which = i >= a.cols, c = i - which * a.cols;
        const uint32_t at = c < whole ? c : whole + VEC - (a.cols - c);
        float s = 0.f;
#pragma unroll 4
        for (uint32_t t = 0; t < teams; ++t) s += dynamic[(which * teams + t) * span + at];
        out[i] = s;
    }
}

// Rows past kNormBackRegCols columns.
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
    each_vector<T, VEC>(a.cols, [&](uint32_t at, int skip) {
        const FVec<VEC> h = to_float<VEC, T>(load_any<VEC>(x + at));
        const FVec<VEC> g = to_float<VEC, T>(load_any<VEC>(dy + at)) * load_param<VEC>(a.weight, at, 1.f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            if (k < skip) continue;
            sum += g[k];
            along = __builtin_fmaf(g[k], (h[k] - mean) * rstd, along);
        }
    });
    const float c1 = row_sum<64, true>(sum, slots[0]) * a.inv_cols;
    const float c2 = row_sum<64, true>(along, slots[1]) * a.inv_cols;
    each_vector<T, VEC>(a.cols, [&](uint32_t at, int) {
        const FVec<VEC> h = to_float<VEC, T>(load_any<VEC>(x + at));
        const FVec<VEC> g = to_float<VEC, T>(load_any<VEC>(dy + at)) * load_param<VEC>(a.weight, at, 1.f);
        FVec<VEC> o;
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = rstd * (g[k] - c1 - (h[k] - mean) * rstd * c2);
        store_any<VEC>(dx + at, from_float<T, VEC>(o));
    });
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

// dweight (blockIdx.y 0) and dbias (1) from the n partial rows: 16 columns by
// 64 groups of partial rows, in float64, joined in group order.
__global__ __launch_bounds__(1024) void
k_norm_weight_grad(const float* __restrict__ partial, uint32_t n, uint32_t cols, float* __restrict__ dweight,
                   float* __restrict__ dbias) {
    __shared__ double part[64][16];
    const uint32_t lane = threadIdx.x % 16, group = threadIdx.x / 16;
    const uint32_t c = blockIdx.x * 16 + lane;
    double sum = 0.0;
    if (c < cols) {
        const float* p = partial + uint64_t(blockIdx.y) * cols + c;
        float v[8];
        for (uint32_t i0 = group; i0 < n; i0 += 8 * 64) {
#pragma unroll
            for (uint32_t u = 0; u < 8; ++u) v[u] = i0 + u * 64 < n ? p[uint64_t(i0 + u * 64) * 2 * cols] : 0.f;
#pragma unroll
            for (uint32_t u = 0; u < 8; ++u) sum += double(v[u]);
        }
    }
    part[group][lane] = sum;
    __syncthreads();
    if (threadIdx.x < 16 && c < cols) {
        sum = 0.0;
        for (int i = 0; i < 64; ++i) sum += part[i][lane];
        (blockIdx.y ? dbias : dweight)[c] = float(sum);
    }
}

}  // namespace adacomp
