// Losses over a large vocabulary straight from the hidden states, and their
// gradients, for gfx950: z = hidden weight^T / temperature is formed in tiles
// and never kept.
//
//   cross entropy   loss = lse - z_t,                dz_v = exp(z_v - lse) - [v = t]
//   distillation    loss = sum_k p_k (log p_k - z_k + lse),  p = softmax(teacher / temperature)
//                   dz_v = exp(z_v - lse) - sum of p_k over the picks k of word v
//   dhidden = dz weight,  dweight = dz^T hidden
//
// Forward is one product: a tile of 256 words leaves each row's largest logit and
// sum of exponentials (k_logits<false>), which k_loss joins; the logits at the
// targets or picks are dot products of their own (k_loss, k_picks).  Backward takes a
// piece of the vocabulary at a time: the product again, whose tiles leave dz in
// 16 bits (k_logits<true>), the target's or picks' elements put right from the
// forward call's float32 values (put_targets, k_pick_grad), and the two
// products from dz (k_product).  A pass is three products for the gradients and
// one for the loss, bound by the matrix cores.
//
// dz is rounded to the operands' 16 bits, for the matrix cores take no wider
// ones: each term of the gradients' sums is off by at most half a step of its
// type, as the rounded results are.  Of few rows, where it costs little, dz has a second
// plane of what the first leaves out.  The rows' factors are divided by the largest of them and
// brought up to 2^14: half's smallest numbers would not hold a probability over the number of
// rows, and equal factors are exact.  (In half an element of dz keeps its 11 bits down to 2^-28 of
// the largest factor: a probability of 2^-8 in a row whose factor is 2^-20 of that.)  float32 calls
// split every operand, dz too, into three bfloat16 planes (tile_product.hpp), and their products
// are as exact as float32's own.
#pragma once

#include "sequence.hpp"
#include "tile_product.hpp"

namespace adacomp {

constexpr uint32_t kLossMaxPicks = 1024;
// Most rows whose dz has a second plane.  Gradients of 512 x 1024 over 32000 words bf16 take 250 us with it and 155
// without, of 4096 rows 1432 and 854: up to here it adds 0.1 ms, past it 1.6 times the call.  With it the distillation's
// gradients are off by 0.0017 of their norm, as their own rounding is, without by 0.0023 to 0.0025, of 64 rows as of
// 4096; the cross entropy's, whose largest elements are -dloss and nearly exact, by 0.0017 either way.
constexpr uint32_t kLossFewRows = 512;

// Where a matrix of the caller's lies; T elements.
struct LossMatrix {
    const void* p;
    uint64_t stride;
};

struct LossArgs {
    LossMatrix hidden, weight;
    Operand x;                  // hidden as an operand, 16-bit
    const int64_t* ids;         // [rows][picks]; targets: one a row
    const float* teacher;       // [rows][picks], nullptr: cross entropy
    float* loss;
    float* lse;
    float* picked;              // [rows][picks]: z at the ids
    const float* dloss;
    float* factor;              // [rows]: dloss / temperature of the rows that count, over the largest, times 2^14
    float* scale;               // [1]: what a result from dz has to be multiplied by
    uint32_t* counts;           // [rows], backward of the distillation: whether a row counts
    float2* part;               // [tile of the vocabulary][rows]: largest logit in units of log 2, sum
    uint32_t rows, width, words, picks;
    float sharp;                // 1 / temperature
};

__device__ __forceinline__ bool is_word(int64_t id, uint32_t words) { return uint64_t(id) < words; }

// Whether a pick has a part in p: a word whose teacher's logit is not -infinity.  NaN has one, and makes the row NaN.
__device__ __forceinline__ bool is_pick(const LossArgs& a, uint64_t i) {
    return is_word(a.ids[i], a.words) && a.teacher[i] != -__builtin_inff();
}

// Whether a row's target is a word, or any of its picks has a part in p.
__device__ __forceinline__ bool row_counts(const LossArgs& a, uint32_t row) {
    return a.teacher ? a.counts[row] != 0 : is_word(a.ids[row], a.words);
}
// The picks' part of that, a wavefront a row.  (By the one workgroup that needs it of every row: 4096 rows of 64 picks
// 50 us.)
__global__ __launch_bounds__(256) void k_row_counts(LossArgs a) {
    const uint32_t row = blockIdx.x * 4 + threadIdx.x / 64, lane = threadIdx.x % 64;
    if (row >= a.rows) return;
    bool any = false;
    for (uint32_t k = lane; k < a.picks; k += 64) any |= is_pick(a, uint64_t(row) * a.picks + k);
    const bool counts = __any(any);
    if (lane == 0) a.counts[row] = counts;
}

// ---- operands ----

// Eight elements of a matrix as planes, or as a padded row: to [plane][rows][line], zeros behind the columns and,
// of rows that are not live, everywhere.
template <typename T, typename E, int PLANES>
__device__ __forceinline__ void pack_eight(const T* from, uint64_t stride, uint32_t rows, uint32_t cols, uint32_t line,
                                           uint64_t row, uint32_t c, bool live, E* to) {
    FVec<8> v = 0.f;
    if (live) {
        const T* p = from + row * stride + c;
        if (c + 8 <= cols) {
            v = to_float<8, T>(load_any<8>(p));
        } else {
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k)
                if (c + k < cols) v[k] = float(p[k]);
        }
    }
    E* out = to + row * line + c;
#pragma unroll
    for (int plane = 0; plane < PLANES; ++plane) {
        const Eight<E> part = __builtin_convertvector(v, Eight<E>);
        *reinterpret_cast<Eight<E>*>(out + plane * uint64_t(rows) * line) = part;
        if (PLANES == 1) break;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float rest = v[k] - float(part[k]);
            v[k] = __builtin_isfinite(float(part[k])) ? rest : 0.f;   // an infinity is whole in the first plane
        }
    }
}
template <typename T, typename E, int PLANES>
__global__ __launch_bounds__(256) void k_pack(const T* from, uint64_t stride, uint32_t rows, uint32_t cols, uint32_t line,
                                              E* to) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, per = line / 8;   // fewer than 2^32, as in the kernels below
    if (i / per < rows) pack_eight<T, E, PLANES>(from, stride, rows, cols, line, i / per, i % per * 8, true, to);
}

// The rows' factors: 0 of those that do not count.  An infinite one leaves them all as they are.  One workgroup.
__device__ __forceinline__ void row_factors(const LossArgs& a) {
    __shared__ float most[16];
    float m = 0.f;
    for (uint32_t row = threadIdx.x; row < a.rows; row += 1024) {
        const float f = row_counts(a, row) ? a.dloss[row] * a.sharp : 0.f;
        a.factor[row] = f;
        m = fmaxf(m, fabsf(f));
    }
    for (int s = 32; s > 0; s /= 2) m = fmaxf(m, __shfl_xor(m, s));
    if (threadIdx.x % 64 == 0) most[threadIdx.x / 64] = m;
    __syncthreads();
    for (int i = 0; i < 16; ++i) m = fmaxf(m, most[i]);
    const bool scaled = m > 0.f && m < __builtin_inff();
    if (scaled)
        for (uint32_t row = threadIdx.x; row < a.rows; row += 1024) a.factor[row] = a.factor[row] / m * 16384.f;
    if (threadIdx.x == 0) a.scale[0] = scaled ? m / 16384.f : 1.f;
}

// What the gradients start from: the factors, by the first workgroup, and the hidden states' rows that count, by the
// others.
template <typename T, typename E, int PLANES>
__global__ __launch_bounds__(1024) void k_loss_start(LossArgs a, uint32_t line, E* to) {
    if (blockIdx.x == 0) {
        row_factors(a);
        return;
    }
    const uint32_t i = (blockIdx.x - 1) * 1024 + threadIdx.x;
    const uint32_t per = line / 8;
    const uint32_t row = i / per;
    if (row >= a.rows) return;
    pack_eight<T, E, PLANES>(static_cast<const T*>(a.hidden.p), a.hidden.stride, a.rows, a.width, line, row,
                             i % per * 8, row_counts(a, row), to);
}

// ---- forward ----

// The rows' largest logits and sums of exponentials over a tile's words, in units of log 2: an exponential is
// one multiply-add before it.  WHOLE: every word of the tile is there.
template <bool WHOLE, typename P>
__device__ __forceinline__ void leave_sums(const P& p, const LossArgs& a, uint32_t word0, uint32_t m0, uint32_t n0,
                                           uint32_t tile, float2* lds) {
    const uint32_t lane = threadIdx.x % 64;
    const float k = a.sharp * kLog2e;
    auto there = [&](int i, int q) { return WHOLE || word0 + m0 + p.row() + i * 32 + p.block_row(q) < a.words; };
#pragma unroll
    for (int j = 0; j < P::NT; ++j) {
        float most = -__builtin_inff(), sum = 0.f;
#pragma unroll
        for (int i = 0; i < P::MT; ++i)
#pragma unroll
            for (int q = 0; q < 16; ++q) most = fmaxf(most, there(i, q) ? p.acc[i][j][q] : -__builtin_inff());
        most *= k;
        // exponentials from a finite number on, also where every logit is -infinity
        const float from = most == -__builtin_inff() ? 0.f : most;
#pragma unroll
        for (int i = 0; i < P::MT; ++i)
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(p.acc[i][j][q], k, -from));
                sum += there(i, q) ? e : 0.f;
            }
        const float other = __shfl_xor(most, 32), theirs = __shfl_xor(sum, 32), top = fmaxf(most, other);
        const float f0 = top == -__builtin_inff() ? 0.f : top;
        sum = sum * __builtin_amdgcn_exp2f(most - f0) + theirs * __builtin_amdgcn_exp2f(other - f0);
        if (lane < 32) lds[(p.wave() % P::WM) * P::TN + p.column() + j * 32 + lane] = make_float2(top, sum);
    }
    __syncthreads();
    for (uint32_t n = threadIdx.x; n < P::TN; n += P::THREADS) {
        if (n0 + n >= a.rows) continue;
        float2 s = lds[n];
        for (int w = 1; w < P::WM; ++w) {
            const float2 t = lds[w * P::TN + n];
            const float top = fmaxf(s.x, t.x), f0 = top == -__builtin_inff() ? 0.f : top;
            s.y = s.y * __builtin_amdgcn_exp2f(s.x - f0) + t.y * __builtin_amdgcn_exp2f(t.x - f0);
            s.x = top;
        }
        a.part[uint64_t(tile) * a.rows + n0 + n] = s;
    }
}

// Two groups of 4 consecutive rows of a tile's block that a lane and the lane 32 before or behind it have (rows 0 to
// 3 and 8 to 11, or 4 to 7 and 12 to 15) become 8 consecutive ones: 0 to 7 of the lower lane, 8 to 15 of the upper.
template <typename E>
__device__ __forceinline__ Eight<E> eight_rows(Four<E> low, Four<E> high) {
    typedef unsigned int Pair __attribute__((ext_vector_type(2)));
    typedef unsigned int Quad __attribute__((ext_vector_type(4)));
    const Pair l = __builtin_bit_cast(Pair, low), h = __builtin_bit_cast(Pair, high);
    const auto x = __builtin_amdgcn_permlane32_swap(l[0], h[0], false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(l[1], h[1], false, false);
    return __builtin_bit_cast(Eight<E>, Quad{x[0], y[0], x[1], y[1]});
}

// dz of a tile, scaled, into [plane][rows][line]: columns from the piece's first word on, zeros behind the last.
// One plane's exponentials take one multiply-add before them, whose rounding is far below the type's; three planes'
// are float32's own.  A row whose factor is 0, whose lse may be anything, gives 0 times 0.
template <bool WHOLE, typename P>
__device__ __forceinline__ void leave_dz(const P& p, const LossArgs& a, uint32_t word0, uint32_t m0, uint32_t n0,
                                         const Operand& dz, uint32_t planes) {
    typedef typename P::E E;
    const uint32_t lane = threadIdx.x % 64;
    const float k = a.sharp * kLog2e;
#pragma unroll
    for (int j = 0; j < P::NT; ++j) {
        const uint32_t row = n0 + p.column() + j * 32 + lane % 32;
        const bool on = row < a.rows;   // the lane 32 away has the same row
        const float f = on ? a.factor[row] : 0.f, lse = f != 0.f ? a.lse[row] : 1e30f, from = lse * kLog2e;
        E* out = static_cast<E*>(const_cast<void*>(dz.p)) + uint64_t(on ? row : 0) * dz.line;
#pragma unroll
        for (int i = 0; i < P::MT; ++i)
#pragma unroll
            for (int q = 0; q < 16; q += 8) {
                const uint32_t m = m0 + p.row() + i * 32 + p.block_row(q);   // and 8 rows on
                FVec<8> v;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float z = p.acc[i][j][q + t];
                    const float e = planes == 1 ? __builtin_amdgcn_exp2f(__builtin_fmaf(z, k, -from))
                                                : exp_of_minus(__builtin_elementwise_minimum(lse - z * a.sharp, 200.f));
                    v[t] = WHOLE || word0 + m + t % 4 + t / 4 * 8 < a.words ? e * f : 0.f;
                }
                const uint32_t at = m0 + p.row() + i * 32 + q * 2 + lane / 32 * 8;
                for (uint32_t plane = 0; plane < planes; ++plane) {
                    const Eight<E> part = __builtin_convertvector(v, Eight<E>);
                    const Eight<E> out8 = eight_rows<E>(__builtin_shufflevector(part, part, 0, 1, 2, 3),
                                                        __builtin_shufflevector(part, part, 4, 5, 6, 7));
                    if (on) *reinterpret_cast<Eight<E>*>(out + plane * dz.plane + at) = out8;
                    if (planes > 1) v -= __builtin_convertvector(part, FVec<8>);
                }
            }
    }
}

// One element of dz in all planes.
template <typename E>
__device__ __forceinline__ void put_dz(const Operand& dz, uint32_t planes, uint32_t row, uint32_t column, float v) {
    E* out = static_cast<E*>(const_cast<void*>(dz.p)) + uint64_t(row) * dz.line + column;
    for (uint32_t plane = 0; plane < planes; ++plane) {
        const E part = E(v);
        out[plane * dz.plane] = part;
        v -= float(part);
    }
}

// dz at the targets that are words of a tile, behind the tile's own stores: exp(z_t - lse) - 1 without the
// difference of two numbers near 1.
template <typename P>
__device__ __forceinline__ void put_targets(const LossArgs& a, uint32_t word0, uint32_t m0, uint32_t n0, const Operand& dz,
                                            uint32_t planes) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (uint32_t n = threadIdx.x; n < P::TN; n += P::THREADS) {
        const uint32_t row = n0 + n;
        if (row >= a.rows) continue;
        const int64_t id = a.ids[row];
        const float f = a.factor[row];
        if (is_word(id, a.words) && uint64_t(id) - word0 - m0 < P::TM && f != 0.f)
            put_dz<typename P::E>(dz, planes, row, uint32_t(id) - word0, expm1f(-a.loss[row]) * f);
    }
}

// A piece of the vocabulary from word0 on; w is its operand.
template <typename P, bool BACK>
__global__ __launch_bounds__(P::THREADS) void k_logits(LossArgs a, Operand w, uint32_t word0, uint32_t tiles_m,
                                                       uint32_t tiles_n, PlanePairs pairs, Operand dz, uint32_t planes,
                                                       uint32_t tile0) {
    extern __shared__ uint4 lds[];
    P p;
    const TilePlace t(blockIdx.x, tiles_m, tiles_n);
    const uint32_t m0 = t.m * P::TM, n0 = t.n * P::TN;
    p.run(w, a.x, m0, n0, 0, w.inner, pairs, reinterpret_cast<typename P::E*>(lds));
    const bool whole = word0 + m0 + P::TM <= a.words;
    if (BACK) {
        if (whole) leave_dz<true>(p, a, word0, m0, n0, dz, planes);
        else leave_dz<false>(p, a, word0, m0, n0, dz, planes);
        if (a.teacher == nullptr) put_targets<P>(a, word0, m0, n0, dz, planes);
    } else {
        float2* sums = reinterpret_cast<float2*>(lds);
        if (whole) leave_sums<true>(p, a, word0, m0, n0, tile0 + t.m, sums);
        else leave_sums<false>(p, a, word0, m0, n0, tile0 + t.m, sums);
    }
}

// z of one row at a word, by a wavefront.
template <typename T>
__device__ __forceinline__ float logit_at(const LossArgs& a, uint64_t row, int64_t id, uint32_t lane) {
    const T* x = static_cast<const T*>(a.hidden.p) + row * a.hidden.stride;
    const T* w = static_cast<const T*>(a.weight.p) + uint64_t(id) * a.weight.stride;
    constexpr int V = 16 / sizeof(T);
    float s = 0.f;
    uint32_t c = lane * V;
    for (; c + V <= a.width; c += 64 * V) {
        const FVec<V> u = to_float<V, T>(load_any<V>(x + c)), v = to_float<V, T>(load_any<V>(w + c));
#pragma unroll
        for (int k = 0; k < V; ++k) s = __builtin_fmaf(u[k], v[k], s);
    }
    for (; c < a.width; ++c) s = __builtin_fmaf(float(x[c]), float(w[c]), s);   // the one lane at the rows' end
    for (int m = 32; m > 0; m /= 2) s += __shfl_xor(s, m);
    return s * a.sharp;
}

// z at the picks: a wavefront a pick.
template <typename T>
__global__ __launch_bounds__(256) void k_picks(LossArgs a) {
    const uint64_t i = uint64_t(blockIdx.x) * 4 + threadIdx.x / 64;
    if (i >= uint64_t(a.rows) * a.picks) return;
    const uint32_t lane = threadIdx.x % 64;
    const int64_t id = a.ids[i];
    const float z = is_word(id, a.words) ? logit_at<T>(a, i / a.picks, id, lane) : 0.f;
    if (lane == 0) a.picked[i] = z;
}

// p of a row's picks by one wavefront: the largest teacher logit and the sum of exponentials.
struct Teacher {
    float most, sum;
    __device__ __forceinline__ Teacher(const LossArgs& a, uint32_t row, uint32_t lane) {
        most = -__builtin_inff();
        sum = 0.f;
        const uint64_t first = uint64_t(row) * a.picks;
        for (uint32_t k = lane; k < a.picks; k += 64)
            if (is_pick(a, first + k)) most = fmaxf(most, a.teacher[first + k]);
        for (int m = 32; m > 0; m /= 2) most = fmaxf(most, __shfl_xor(most, m));
        for (uint32_t k = lane; k < a.picks; k += 64)
            if (is_pick(a, first + k)) sum += expf((a.teacher[first + k] - most) * a.sharp);
        for (int m = 32; m > 0; m /= 2) sum += __shfl_xor(sum, m);
    }
    __device__ __forceinline__ float log_p(float logit, float sharp) const { return (logit - most) * sharp - logf(sum); }
};

// A wavefront a row: the tiles' sums joined, and the loss.
template <typename T>
__global__ __launch_bounds__(256) void k_loss(LossArgs a, uint32_t tiles) {
    const uint32_t row = blockIdx.x * 4 + threadIdx.x / 64, lane = threadIdx.x % 64;
    if (row >= a.rows) return;
    float target = 0.f;
    const bool scored = a.teacher == nullptr && is_word(a.ids[row], a.words);
    if (scored) target = logit_at<T>(a, row, a.ids[row], lane);
    float most = -__builtin_inff(), sum = 0.f;
    auto join = [&](float m, float s) {
        const float top = fmaxf(most, m), f0 = top == -__builtin_inff() ? 0.f : top;
        sum = sum * exp2f(most - f0) + s * exp2f(m - f0);
        most = top;
    };
    constexpr uint32_t U = 4;   // requested together
    for (uint32_t t = lane; t < tiles; t += 64 * U) {
        float2 s[U];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) s[u] = a.part[uint64_t(min(t + 64 * u, tiles - 1)) * a.rows + row];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u)
            if (t + 64 * u < tiles) join(s[u].x, s[u].y);
    }
    for (int m = 32; m > 0; m /= 2) join(__shfl_xor(most, m), __shfl_xor(sum, m));
    const float lse = __builtin_fmaf(most, kLn2, __builtin_fmaf(most, kLn2Low, logf(sum)));   // most in units of log 2
    if (lane == 0) a.lse[row] = lse;
    float loss = 0.f;
    if (a.teacher == nullptr) {
        if (scored) loss = lse - target;
    } else {
        const Teacher p(a, row, lane);
        for (uint32_t k = lane; k < a.picks; k += 64) {
            const uint64_t i = uint64_t(row) * a.picks + k;
            if (!is_pick(a, i)) continue;
            const float l = p.log_p(a.teacher[i], a.sharp);
            if (l != -__builtin_inff()) loss += expf(l) * (l + (lse - a.picked[i]));   // p log p is 0 at p = 0
        }
        for (int m = 32; m > 0; m /= 2) loss += __shfl_xor(loss, m);
    }
    if (lane == 0) a.loss[row] = loss;
}

// ---- backward ----

// dz at the picks of a piece, a wavefront a row.  A word that was picked twice has both its shares of p, from every
// one of its picks.
template <typename E>
__global__ __launch_bounds__(256) void k_pick_grad(LossArgs a, uint32_t word0, uint32_t words, Operand dz, uint32_t planes) {
    __shared__ int64_t ids[4][kLossMaxPicks];
    __shared__ float ps[4][kLossMaxPicks];
    const uint32_t row = blockIdx.x * 4 + threadIdx.x / 64, lane = threadIdx.x % 64, w = threadIdx.x / 64;
    const bool on = row < a.rows && a.factor[row < a.rows ? row : 0] != 0.f;
    if (on) {
        const Teacher p(a, row, lane);
        for (uint32_t k = lane; k < a.picks; k += 64) {
            const uint64_t i = uint64_t(row) * a.picks + k;
            ids[w][k] = a.ids[i];
            ps[w][k] = is_pick(a, i) ? expf(p.log_p(a.teacher[i], a.sharp)) : 0.f;
        }
    }
    __syncthreads();
    if (!on) return;
    for (uint32_t k = lane; k < a.picks; k += 64) {
        const int64_t id = ids[w][k];
        if (!is_word(id, a.words) || uint64_t(id) - word0 >= words) continue;
        float p = 0.f;
        for (uint32_t j = 0; j < a.picks; ++j) p += ids[w][j] == id ? ps[w][j] : 0.f;
        const float q = expf(a.picked[uint64_t(row) * a.picks + k] - a.lse[row]);
        put_dz<E>(dz, planes, row, uint32_t(id) - word0, (q - p) * a.factor[row]);
    }
}

// What becomes of a product's tile.
struct ProductOut {
    void* p;              // [n][m], of T, or float32 partial sums [share][n][m]
    uint64_t stride;
    uint32_t rows, cols;  // n and m that are there
    const float* scale;   // a factor of the result
    bool add;             // partial sums: to what is there
};

// N columns of a row from m on, as far as they are there.
template <typename T, int N>
__device__ __forceinline__ void put_columns(T* row, uint32_t m, uint32_t cols, bool on, typename Packed<T, N>::V v) {
    if (!on) return;
    if (m + N <= cols) {
        store_any<N>(row + m, v);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (m + k < cols) row[m + k] = v[k];
    }
}

// One product from dz: [n, m] = sum over k; shares of the inner axis where PARTIAL.
template <typename P, typename T, bool PARTIAL>
__global__ __launch_bounds__(P::THREADS) void k_product(Operand x, Operand y, uint32_t inner, PlanePairs pairs,
                                                        uint32_t tiles_m, uint32_t tiles_n, uint32_t shares, ProductOut out) {
    extern __shared__ uint4 lds[];
    P p;
    const uint32_t tiles = tiles_m * tiles_n, share = blockIdx.x / tiles;
    const TilePlace t(blockIdx.x % tiles, tiles_m, tiles_n);
    const uint32_t m0 = t.m * P::TM, n0 = t.n * P::TN;
    const uint32_t each = (inner + shares * kTileK - 1) / (shares * kTileK) * kTileK;
    const uint32_t begin = min(share * each, inner), end = min(begin + each, inner);
    p.run(x, y, m0, n0, begin, end, pairs, reinterpret_cast<typename P::E*>(lds));
    const float factor = PARTIAL ? 1.f : out.scale[0];
    const uint32_t lane = threadIdx.x % 64;
#pragma unroll
    for (int j = 0; j < P::NT; ++j) {
        const uint32_t n = n0 + p.column() + j * 32 + lane % 32;
        const bool on = n < out.rows;   // the lane 32 away has the same row
        T* row = static_cast<T*>(out.p) + (PARTIAL ? uint64_t(share) * out.rows * out.stride : 0) +
                 uint64_t(on ? n : 0) * out.stride;
#pragma unroll
        for (int i = 0; i < P::MT; ++i)
#pragma unroll
            for (int q = 0; q < 16; q += 8) {
                const uint32_t first = m0 + p.row() + i * 32 + q * 2;
                if constexpr (sizeof(T) == 2) {
                    FVec<8> v;
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = p.acc[i][j][q + k] * factor;
                    const Eight<T> part = __builtin_convertvector(v, Eight<T>);
                    const Eight<T> whole = eight_rows<T>(__builtin_shufflevector(part, part, 0, 1, 2, 3),
                                                         __builtin_shufflevector(part, part, 4, 5, 6, 7));
                    put_columns<T, 8>(row, first + lane / 32 * 8, out.cols, on, whole);
                } else {
#pragma unroll
                    for (int h = 0; h < 8; h += 4) {
                        const uint32_t m = first + h * 2 + lane / 32 * 4;
                        FVec<4> v;
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = p.acc[i][j][q + h + k] * factor;
                        if (PARTIAL && out.add && on && m < out.cols) v += load_any<4>(row + m);   // rows of whole 8 columns
                        put_columns<T, 4>(row, m, out.cols, on, v);
                    }
                }
            }
    }
}

// The shares' partial sums joined, scaled and rounded.
template <typename T>
__global__ __launch_bounds__(256) void k_join_shares(const float* part, uint32_t shares, uint64_t rows, uint32_t cols,
                                                     uint32_t line, const float* scale, T* out, uint64_t stride) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, per = line / 4, c = i % per * 4;
    const uint64_t row = i / per;
    if (row >= rows) return;
    FVec<4> v = 0.f;
#pragma unroll 8
    for (uint32_t s = 0; s < shares; ++s) v += load_any<4>(part + (s * rows + row) * line + c);
    v *= scale[0];
    T* to = out + row * stride + c;
    if (c + 4 <= cols) {
        store_any<4>(to, from_float<T, 4>(v));
    } else {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
            if (c + k < cols) to[k] = T(v[k]);
    }
}

// A gradient that nothing adds to.
template <typename T>
__global__ __launch_bounds__(256) void k_zero_rows(T* out, uint64_t stride, uint64_t rows, uint32_t cols) {
    for (uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * cols; i += uint64_t(gridDim.x) * 256)
        out[i / cols * stride + i % cols] = T(0.f);
}

}  // namespace adacomp
