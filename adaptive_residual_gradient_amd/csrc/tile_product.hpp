// Tiles of a matrix product on the matrix cores of gfx950: the sum over k of
// A[m, k] B[n, k] in float32, of bfloat16 or half operands.
//
// A workgroup of WM x WN wavefronts forms TM x TN results, a wavefront MT x NT
// blocks of 32 x 32 of them, in registers.  Steps of 64 of the inner axis lie in LDS
// buffers, one of which is read while the next steps' elements go straight
// from memory into the others.
//
// An operand is read in either order.  K inner (rows of the inner axis): its
// tile lies in LDS as rows of 64 elements, whose 16-byte pieces change places by
// the row, so that the 16 lanes of a cycle find 16 different bank groups.  K
// outer: the tile lies as 64 rows along m (or n), 64-byte pieces change places
// by the row, and the transposing LDS read hands each lane its 4 elements along k.
//
// Wide operands: a matrix is the sum of planes of 16 bits each.  Float32 matrices
// are split into three bfloat16 planes whose sum they are to 2^-24, and the
// product is the sum of the six products of planes that are not below that
// (kThreeByThree).  Or B alone has a second plane, of what the first leaves out
// (kOneByTwo).
//
// Where both operands are K inner, each part's elements are read during the products of the
// part before, across the steps' barrier too; the compiler's own order is a read, its
// wait and two products (8192 x 65536 x 2048 bf16 with the losses' sums 1780 us against 1967: the
// matrix cores busy 63% of the cycles against 52%, at a clock that goes down from 2.1 to
// 1.95 GHz).  Transposing reads, which have to wait in their own statement, leave the overlap
// to the other wavefront of the SIMD.  LDS does not show: its reads have no bank conflicts, and took the same
// time when half of their cycles were.
#pragma once

#include "elements.hpp"

namespace adacomp {

constexpr uint32_t kTileK = 64;      // the inner axis in LDS
// Pairs of planes of a product: how many, and the planes of A and B, 4 bits each, smallest products first.
struct PlanePairs {
    uint32_t count, a, b;
};
constexpr PlanePairs kOneByOne{1, 0x0, 0x0}, kOneByTwo{2, 0x00, 0x10}, kThreeByThree{6, 0x021010, 0x201100};

typedef float f32x16 __attribute__((ext_vector_type(16)));
template <typename E>
using Eight = E __attribute__((ext_vector_type(8)));
template <typename E>
using Four = E __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma(Eight<bf16> a, Eight<bf16> b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(Eight<f16> a, Eight<f16> b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
#define ADACOMP_LDS __attribute__((address_space(3)))
#define ADACOMP_GLOBAL __attribute__((address_space(1)))
// Transposing LDS reads of N blocks of 32 rows: two of each block, the second 4 lines behind the first, whose
// 4 + 4 elements along k are the lane's 8.  at: the blocks' LDS addresses; LOW: bytes from there to the lines.  The
// builtin waits for every copy into LDS that is still under way, also into the other buffer; these wait for
// themselves alone, in the same statement.
typedef short Half8 __attribute__((ext_vector_type(4)));
template <int LOW, int HIGH>
__device__ __forceinline__ void read_transposed(const uint32_t (&at)[1], Half8 (&v)[2]) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %2 offset:%3\n\tds_read_b64_tr_b16 %1, %2 offset:%4\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1])
        : "v"(at[0]), "n"(LOW), "n"(HIGH)
        : "memory");
}
template <int LOW, int HIGH>
__device__ __forceinline__ void read_transposed(const uint32_t (&at)[2], Half8 (&v)[4]) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4 offset:%6\n\tds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
        "ds_read_b64_tr_b16 %2, %5 offset:%6\n\tds_read_b64_tr_b16 %3, %5 offset:%7\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(at[0]), "v"(at[1]), "n"(LOW), "n"(HIGH)
        : "memory");
}
template <int LOW, int HIGH>
__device__ __forceinline__ void read_transposed(const uint32_t (&at)[4], Half8 (&v)[8]) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8 offset:%12\n\tds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
        "ds_read_b64_tr_b16 %2, %9 offset:%12\n\tds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
        "ds_read_b64_tr_b16 %4, %10 offset:%12\n\tds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
        "ds_read_b64_tr_b16 %6, %11 offset:%12\n\tds_read_b64_tr_b16 %7, %11 offset:%13\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(LOW), "n"(HIGH)
        : "memory");
}

// A matrix, 16-byte aligned, whose lines are 16-byte aligned too.
struct Operand {
    const void* p;
    uint64_t line;      // elements from one line to the next: along m, or along k where K is outer
    uint64_t plane;     // from one plane to the next
    uint32_t extent;    // of m, above 0; where K is outer a multiple of 8 within the line
    uint32_t inner;     // of k; where K is inner, zeros up to a multiple of 8
};

__device__ __constant__ const uint4 kTileZeros = {0u, 0u, 0u, 0u};

// One operand's tile on its way into LDS.
template <typename E, bool OUTER, int ROWS, int THREADS>
struct TileLoader {
    static constexpr int PIECES = ROWS * kTileK / 8;       // of 16 bytes
    static constexpr int N = PIECES / THREADS;
    static constexpr int LINE = (OUTER ? ROWS : kTileK) / 8;   // pieces of a line in LDS
    static_assert(PIECES % THREADS == 0, "whole turns");
    uint32_t offset[N];   // bytes from the tile's first element
    uint32_t k[N];        // the piece's place on the inner axis
    // Where piece c of a line lies.
    static __device__ __forceinline__ uint32_t place(uint32_t line, uint32_t c) {
        if (!OUTER) return c ^ (line >> 1 & 7u);   // 16 lines' pieces lie in the 64 banks once
        const uint32_t turn = ROWS >= 256 ? (line & 3u) | (line >> 1 & 4u) : ROWS >= 128 ? line & 3u : line >> 1 & 1u;
        return c ^ turn << 2;
    }
    __device__ __forceinline__ TileLoader(const Operand& x, uint32_t m0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t at = i * THREADS + threadIdx.x, line = at / LINE, c = place(line, at % LINE);   // its own inverse
            if (OUTER) {
                // past the last column an earlier one again: nobody looks at the results
                const uint32_t m = min(m0 + c * 8, x.extent - 8) - m0;
                offset[i] = (line * uint32_t(x.line) + m) * 2;
                k[i] = line;
            } else {
                const uint32_t m = min(m0 + line, x.extent - 1) - m0;
                offset[i] = (m * uint32_t(x.line) + c * 8) * 2;
                k[i] = c * 8;
            }
        }
    }
    // The tile's first element of a plane at k0, and the bytes from there to the next step's.
    static __device__ __forceinline__ const char* first(const Operand& x, uint32_t plane, uint32_t m0, uint32_t k0) {
        const E* p = static_cast<const E*>(x.p) + plane * x.plane;
        return reinterpret_cast<const char*>(p + (OUTER ? uint64_t(k0) * x.line + m0 : uint64_t(m0) * x.line + k0));
    }
    static __device__ __forceinline__ uint64_t advance(const Operand& x) { return (OUTER ? x.line : 1) * kTileK * 2; }
    // Step [k0, k0 + 64), whose first element is `base`; from `end` on zeros.
    __device__ __forceinline__ void request(const char* base, uint32_t k0, uint32_t end, E* tile) const {
        char* to = reinterpret_cast<char*>(tile) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64) * 1024;
        auto copy = [&](int i, const char* from) {
            __builtin_amdgcn_global_load_lds((ADACOMP_GLOBAL const void*)from, (ADACOMP_LDS void*)(to + i * THREADS * 16),
                                             16, 0, 0);
        };
        if (k0 + kTileK <= end) {
#pragma unroll
            for (int i = 0; i < N; ++i) copy(i, base + offset[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                copy(i, k0 + k[i] < end ? base + offset[i] : reinterpret_cast<const char*>(&kTileZeros));
        }
    }
    // A wavefront's BLOCKS of 32 rows from m on: where its lanes read them.
    template <int BLOCKS>
    struct Reader {
        uint32_t at[BLOCKS];   // LDS addresses in bytes, from the tile's first
        __device__ __forceinline__ explicit Reader(uint32_t m) {
            const uint32_t lane = threadIdx.x % 64;
#pragma unroll
            for (int i = 0; i < BLOCKS; ++i) {
                if (OUTER) {
                    // lanes 16 g .. 16 g + 15: the columns from 16 (g % 2) on and k from 8 (g / 2) on, in two halves.
                    // Lines 4 and 16 apart have their pieces in the same places.
                    const uint32_t g = lane / 16, column = m + i * 32 + 16 * (g % 2) + lane % 4 * 4;
                    const uint32_t line = 8 * (g / 2) + lane % 16 / 4;
                    at[i] = (line * ROWS + place(line, column / 8) * 8 + column % 8) * 2;
                } else {
                    at[i] = (m + i * 32 + lane % 32) * kTileK * 2;
                }
            }
        }
        // Elements K .. K + 15 of the step.
        template <int K>
        __device__ __forceinline__ void read(const E* tile, Eight<E> (&v)[BLOCKS]) const {
            if constexpr (OUTER) {
                const uint32_t base = uint32_t(uintptr_t((ADACOMP_LDS const E*)tile));
                uint32_t where[BLOCKS];
                Half8 half[2 * BLOCKS];
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i) where[i] = base + at[i];
                read_transposed<K * ROWS * 2, (K + 4) * ROWS * 2>(where, half);
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i)
                    v[i] = __builtin_bit_cast(Eight<E>, __builtin_shufflevector(half[2 * i], half[2 * i + 1], 0, 1, 2, 3, 4, 5,
                                                                                6, 7));
            } else {
                const uint32_t lane = threadIdx.x % 64;
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i) {
                    // rows 32 apart have their pieces in the same places
                    const char* p = reinterpret_cast<const char*>(tile) + at[i] + place(lane % 32, K / 8 + lane / 32) * 16;
                    v[i] = *reinterpret_cast<const Eight<E>*>(p);
                }
            }
        }
    };
};

// BUFFERS, a power of two: 2 of the large tiles; 4 of small ones, whose steps are over before the next one's
// elements arrive.
template <typename E_, int WM_, int WN_, int MT_, int NT_, int BUFFERS, bool AOUTER, bool BOUTER>
struct TileProduct {
    typedef E_ E;
    static constexpr int WM = WM_, WN = WN_, MT = MT_, NT = NT_;
    static constexpr int TM = WM * MT * 32, TN = WN * NT * 32, THREADS = WM * WN * 64;
    typedef TileLoader<E, AOUTER, TM, THREADS> LoadA;
    typedef TileLoader<E, BOUTER, TN, THREADS> LoadB;
    static constexpr uint32_t STEP = (TM + TN) * kTileK;   // elements of one buffer
    static constexpr uint32_t LDS_BYTES = BUFFERS * STEP * 2;
    // Whether parts are read ahead.
    static constexpr bool AHEAD = !AOUTER && !BOUTER && BUFFERS == 2;
    static constexpr int REQUESTS = LoadA::N + LoadB::N;   // a thread's, a step

    f32x16 acc[MT][NT];
    // the wavefront's first row and column of the tile
    __device__ static __forceinline__ uint32_t wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }
    __device__ static __forceinline__ uint32_t row() { return wave() % WM * (MT * 32); }
    __device__ static __forceinline__ uint32_t column() { return wave() / WM * (NT * 32); }
    // Row of register i of a block; the lane's column is lane % 32.
    __device__ static __forceinline__ uint32_t block_row(int i) {
        return 8 * (i / 4) + i % 4 + 4 * (threadIdx.x % 64 / 32);
    }

    // 16 elements of the inner axis.
    template <int K, typename RA, typename RB>
    __device__ __forceinline__ void part(const RA& ra, const RB& rb, const E* ta, const E* tb) {
        Eight<E> av[MT], bv[NT];
        ra.template read<K>(ta, av);
        rb.template read<K>(tb, bv);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = mfma(av[i], bv[j], acc[i][j]);
    }

    // The products of one part's elements, and the next part's read meanwhile: a read behind each product but the
    // first, which waits for the ones before.
    template <int K, typename RA, typename RB>
    __device__ __forceinline__ void part_ahead(const RA& ra, const RB& rb, const E* ta, const E* tb, Eight<E> (&av)[MT],
                                               Eight<E> (&bv)[NT]) {
        Eight<E> an[MT], bn[NT];
        ra.template read<K>(ta, an);
        rb.template read<K>(tb, bn);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = mfma(av[i], bv[j], acc[i][j]);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
        for (int i = 0; i < MT + NT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MT; ++i) av[i] = an[i];
#pragma unroll
        for (int i = 0; i < NT; ++i) bv[i] = bn[i];
    }

    // The sum over k in [kbegin, kend) of every pair of planes.
    __device__ __forceinline__ void run(const Operand& a, const Operand& b, uint32_t m0, uint32_t n0, uint32_t kbegin,
                                        uint32_t kend, PlanePairs pairs, E* lds) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = 0.f;
        const LoadA la(a, m0);
        const LoadB lb(b, n0);
        const uint32_t total = (kend - kbegin + kTileK - 1) / kTileK * pairs.count;
        uint32_t k = kbegin, left = 4 * (pairs.count - 1);
        const char *pa = LoadA::first(a, pairs.a >> left & 15u, m0, k), *pb = LoadB::first(b, pairs.b >> left & 15u, n0, k);
        const uint64_t sa = LoadA::advance(a), sb = LoadB::advance(b);
        const uint32_t enda = min(kend, a.inner), endb = min(kend, b.inner);
        auto request = [&](E* to) {
            la.request(pa, k, enda, to);
            lb.request(pb, k, endb, to + TM * kTileK);
            k += kTileK;
            pa += sa;
            pb += sb;
            if (k >= kend) {   // the next pair; after the last one nothing is requested
                k = kbegin;
                left = left >= 4 ? left - 4 : 0;
                pa = LoadA::first(a, pairs.a >> left & 15u, m0, k);
                pb = LoadB::first(b, pairs.b >> left & 15u, n0, k);
            }
        };
        for (uint32_t step = 0; step + 1 < BUFFERS && step < total; ++step) request(lds + step * STEP);
        const typename LoadA::template Reader<MT> ra(row());
        const typename LoadB::template Reader<NT> rb(column());
        if constexpr (AHEAD) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // step 0 is there
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (1 < total) request(lds + STEP);
            Eight<E> av[MT], bv[NT];
            ra.template read<0>(lds, av);
            rb.template read<0>(lds + TM * kTileK, bv);
            for (uint32_t step = 0; step < total; ++step) {
                const E* ta = lds + (step & 1) * STEP;
                const E* tb = ta + TM * kTileK;
                part_ahead<16>(ra, rb, ta, tb, av, bv);
                part_ahead<32>(ra, rb, ta, tb, av, bv);
                part_ahead<48>(ra, rb, ta, tb, av, bv);
                // The next step's elements are there, and this buffer has been read.
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                if (step + 2 < total) request(lds + (step & 1) * STEP);
                const E* na = lds + (~step & 1) * STEP;
                part_ahead<0>(ra, rb, na, na + TM * kTileK, av, bv);   // behind the last step read and not used
            }
            __syncthreads();   // the buffers are free
            return;
        }
        for (uint32_t step = 0; step < total; ++step) {
            // This step's elements are there: of the later requests, those of BUFFERS - 2 steps, none has to be.  And
            // the buffer before this one has been read, by every wavefront's own wait for its reads before the
            // barrier.  (A fence would wait for every request.)
            if (step + BUFFERS - 1 <= total)
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((BUFFERS - 2) * REQUESTS) : "memory");
            else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            const E* ta = lds + (step & (BUFFERS - 1)) * STEP;
            const E* tb = ta + TM * kTileK;
            if (step + BUFFERS - 1 < total) request(lds + ((step + BUFFERS - 1) & (BUFFERS - 1)) * STEP);
            part<0>(ra, rb, ta, tb);
            part<16>(ra, rb, ta, tb);
            part<32>(ra, rb, ta, tb);
            part<48>(ra, rb, ta, tb);
        }
        __syncthreads();   // the buffers are free
    }
};

// The tile of a workgroup.  Workgroups go to the 8 chiplets in turn: each chiplet takes a run of
// neighbouring tiles, 4 along m and then along n, whose operands its cache holds.
struct TilePlace {
    uint32_t m, n;
    __device__ __forceinline__ TilePlace(uint32_t i, uint32_t tiles_m, uint32_t tiles_n) {
        const uint32_t total = tiles_m * tiles_n, each = total / 8, rest = total % 8;
        const uint32_t xcd = i % 8;
        i = xcd * each + min(xcd, rest) + i / 8;
        constexpr uint32_t G = 4;
        const uint32_t group = i / (G * tiles_n), high = min(tiles_m - group * G, G), at = i - group * G * tiles_n;
        m = group * G + at % high;
        n = at / high;
    }
};

}  // namespace adacomp
