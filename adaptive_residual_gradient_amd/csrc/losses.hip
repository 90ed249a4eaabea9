// C ABI of the losses over a vocabulary (declared in include/adacomp.h):
// argument checking and stream-ordered kernel launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/adacomp.h"
#include "host_checks.hpp"
#include "vocabulary_loss.hpp"

using namespace adacomp;

namespace {

constexpr uint32_t kWord = 256;            // words of a tile of the vocabulary, at most
constexpr uint64_t kPieceBytes = 1u << 30;     // dz of a piece
constexpr uint32_t kPieceMost = 65536, kPieceLeast = 2048, kPackMost = 16384;   // words of a piece, backward and forward
constexpr uint32_t kCus = 256;

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }
uint32_t share_of(uint64_t n, uint32_t each) { return static_cast<uint32_t>((n + each - 1) / each); }
uint32_t blocks_of(uint64_t items) { return static_cast<uint32_t>((items + 255) / 256); }

// Tiles of the products, each by 8 wavefronts (small ones by fewer keep too few requests under way: 300 x 256
// float32 over 4999 words 106 us forward and backward, by 4 wavefronts 114, by 2 with 64 x 64 tiles 122, all before
// addresses went on from step to step, 92 since): 256 x 256
// where they give most CUs one; else 128 x 128; for few rows, or where these leave half of the CUs without one,
// 128 x 64.
enum { kBig, kMid, kSmall };
constexpr uint32_t kTileM[3] = {256, 128, 128};   // words, or columns of a gradient
uint64_t tiles(uint64_t m, uint64_t n, uint64_t side) { return (m + side - 1) / side * ((n + side - 1) / side); }
int tile_of(uint64_t m, uint64_t n, uint64_t shares = 1) {
    if (n <= 64) return kSmall;
    if (tiles(m, n, 256) * shares >= kCus * 3 / 4) return kBig;
    return tiles(m, n, 128) * shares >= kCus / 2 ? kMid : kSmall;
}
// Shares of the inner axis of a product into partial sums: for one tile a CU where 256 x 256 tiles are enough for a
// quarter of them, else for two of 128 x 128.
uint32_t shares_of(uint64_t m, uint64_t n, uint64_t k, uint32_t planes) {
    const uint64_t big = tiles(m, n, 256), small = std::max<uint64_t>(tiles(m, n, 128), 1);
    const uint64_t want = big >= kCus / 4 ? (kCus + big - 1) / big : (2 * kCus + small - 1) / small;
    const uint64_t most = (k + 255) / 256 * (planes == 3 ? 4 : planes);   // 256 of the inner axis, or as much work in planes
    return static_cast<uint32_t>(std::max<uint64_t>(std::min<uint64_t>({want, most, 64}), 1));
}

struct HeadLayout {
    uint32_t line, planes, dz_planes, piece, shares;   // line: a packed row's elements
    uint64_t x, w, part, factor, scale, counts, dz, dx, bytes;   // byte offsets
};

int check_head(const adacomp_head* h, uint32_t picks) {
    if (h == nullptr || type_size(h->type) == 0 || h->width == 0 || h->vocabulary == 0 || picks == 0)
        return ADACOMP_ERR_INVALID_ARGUMENT;
    constexpr uint64_t most = uint64_t(1) << 24;
    if (h->rows >= most || h->vocabulary >= most || h->width > 65536 || picks > ADACOMP_MAX_PICKS)
        return ADACOMP_ERR_TOO_LARGE;
    // Work-items of a launch: a wavefront a pick, 4 elements of the hidden rows, and a workgroup a tile of the logits.
    // (Smaller tiles than these are taken where there are few, and of 64 rows or fewer; the gradients' products have
    // a piece's words or a row's width in place of the vocabulary.)
    constexpr uint64_t items = uint64_t(1) << 32;
    if (h->rows * picks * 64 >= items || h->rows * (up(h->width, 8) / 4) >= items ||
        tiles(h->vocabulary, h->rows, 256) * 512 >= items)
        return ADACOMP_ERR_TOO_LARGE;
    return ADACOMP_OK;
}

HeadLayout head_layout(const adacomp_head& h, bool back) {
    HeadLayout l{};
    l.line = static_cast<uint32_t>(up(h.width, 8));
    const uint64_t R = h.rows, V = h.vocabulary;
    l.planes = h.type == ADACOMP_FLOAT ? 3 : 1;
    l.dz_planes = l.planes == 3 ? 3 : R <= kLossFewRows ? 2 : 1;
    if (back) {
        const uint64_t words = kPieceBytes / std::max<uint64_t>(2 * l.dz_planes * R, 1) / kWord * kWord;
        // The tiles of a piece's dweight are whole turns of the CUs, or all of the vocabulary's where their last turn
        // is half full; where it is not, the rest of the vocabulary is a piece of its own (8192 x 2048 over 49999
        // words: 49152 and 847).
        const uint64_t across = (h.width + 255) / 256, turn = up(kCus, across) / across * kWord, all = up(V, kWord);
        uint64_t piece = std::min<uint64_t>(std::max<uint64_t>(std::min<uint64_t>(words, kPieceMost), kPieceLeast), all);
        const uint64_t last = across * (all / kWord) % kCus;
        if (piece > turn && (piece < all || (last > 0 && last < kCus / 2))) piece = piece / turn * turn;
        l.piece = static_cast<uint32_t>(piece);
    } else {
        l.piece = static_cast<uint32_t>(std::min<uint64_t>(kPackMost, up(V, kWord)));
    }
    auto place = [&](uint64_t bytes) {
        const uint64_t at = l.bytes;
        l.bytes += up(bytes, 256);
        return at;
    };
    l.x = place(R * l.line * 2 * l.planes);
    l.w = place(uint64_t(l.piece) * l.line * 2 * l.planes);
    uint64_t parts = 0;   // whether the weight is taken as it lies, in one piece, or copied
    if (!back)
        for (const uint64_t piece : {V, uint64_t(l.piece)}) {
            const uint64_t side = kTileM[tile_of(piece, R)];
            parts = std::max(parts, V / piece * up(piece, side) / side + up(V % piece, side) / side);
        }
    l.part = place(R * parts * 8);
    if (back) {
        l.factor = place(R * 4);
        l.scale = place(4);
        l.counts = place(R * 4);
        l.dz = place(R * l.piece * 2 * l.dz_planes);
        l.shares = shares_of(h.width, R, l.piece, l.dz_planes);
        l.dx = place(uint64_t(l.shares) * R * l.line * 4);
    }
    return l;
}

// Pointers and strides of one call.
int check_matrix(const void* p, uint64_t stride, uint64_t rows, uint32_t width, uint64_t size) {
    if (rows == 0) return ADACOMP_OK;
    if (p == nullptr || stride < width) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (!aligned_to(p, size)) return ADACOMP_ERR_MISALIGNED;
    return stride >= (uint64_t(1) << 24) ? ADACOMP_ERR_TOO_LARGE : ADACOMP_OK;
}
Range matrix_range(const void* p, uint64_t stride, uint64_t rows, uint32_t width, uint64_t size) {
    return range_of(p, p && rows ? ((rows - 1) * stride + width) * size : 0);
}

struct LossCall {
    const adacomp_head* head;
    const int64_t* ids;
    const float* teacher;     // nullptr: cross entropy
    uint32_t picks;
    float temperature;
    float *loss, *lse, *picked;
    const float* dloss;       // backward
    void *dhidden, *dweight;
    uint64_t dhidden_stride, dweight_stride;
    void* ws;
    uint64_t ws_bytes;
    hipStream_t stream;
    bool back, distil;
};

template <typename T, typename E, int PLANES>
void pack(const void* from, uint64_t stride, uint64_t rows, const LossArgs& a, uint32_t line, void* to, hipStream_t s) {
    hipLaunchKernelGGL((k_pack<T, E, PLANES>), dim3(blocks_of(rows * (line / 8))), dim3(256), 0, s,
                       static_cast<const T*>(from), stride, uint32_t(rows), a.width, line, static_cast<E*>(to));
}

// An operand needs no copy where its rows are 16-byte aligned and end with a whole 16 bytes.
template <typename T>
bool direct(const void* p, uint64_t stride, uint32_t width) {
    return sizeof(T) == 2 && aligned16(p) && stride % 8 == 0 && width % 8 == 0 && stride < (1u << 22);
}

// T: the matrices' elements, E: the operands'.
template <typename T, typename E, int PLANES>
struct Loss {
    const LossCall& c;
    const HeadLayout& l;
    LossArgs a;
    char* ws;

    Operand operand(const void* p, uint64_t line, uint64_t rows) const {
        return Operand{p, line, rows * line, uint32_t(rows), l.line};
    }
    // Rows of the weight from word0 on, copied where they have to be.
    Operand weight(uint32_t word0, uint32_t words) const {
        const T* p = static_cast<const T*>(a.weight.p) + uint64_t(word0) * a.weight.stride;
        if (direct<T>(p, a.weight.stride, a.width)) return operand(p, a.weight.stride, words);
        pack<T, E, PLANES>(p, a.weight.stride, words, a, l.line, ws + l.w, c.stream);
        return operand(ws + l.w, l.line, words);
    }
    // Lines become the inner axis.
    static Operand turned(const Operand& x, uint32_t extent, uint32_t inner) {
        return Operand{x.p, x.line, x.plane, extent, inner};
    }

    template <typename P, bool BACK>
    void logits(const Operand& w, uint32_t word0, const Operand& dz, uint32_t tile0) const {
        const uint32_t tm = share_of(w.extent, P::TM), tn = share_of(a.rows, P::TN);
        hipLaunchKernelGGL((k_logits<P, BACK>), dim3(tm * tn), dim3(P::THREADS), P::LDS_BYTES, c.stream, a, w, word0, tm, tn,
                           PLANES == 3 ? kThreeByThree : kOneByOne, dz, l.dz_planes, tile0);
    }
    template <bool BACK>
    void logits(int tile, const Operand& w, uint32_t word0, const Operand& dz, uint32_t tile0) const {
        switch (tile) {
            case kBig: return logits<TileProduct<E, 2, 4, 4, 2, 2, false, false>, BACK>(w, word0, dz, tile0);
            case kMid: return logits<TileProduct<E, 4, 2, 1, 2, 2, false, false>, BACK>(w, word0, dz, tile0);
            default: return logits<TileProduct<E, 4, 2, 1, 1, 4, false, false>, BACK>(w, word0, dz, tile0);
        }
    }
    template <typename P, typename O, bool PARTIAL>
    void product(const Operand& x, const Operand& y, uint32_t inner, uint32_t shares, const ProductOut& out) const {
        const uint32_t tm = share_of(out.cols, P::TM), tn = share_of(out.rows, P::TN);
        hipLaunchKernelGGL((k_product<P, O, PARTIAL>), dim3(tm * tn * shares), dim3(P::THREADS), P::LDS_BYTES, c.stream, x,
                           y, inner, PLANES == 3 ? kThreeByThree : l.dz_planes == 2 ? kOneByTwo : kOneByOne, tm, tn, shares,
                           out);
    }
    template <typename O, bool PARTIAL, bool YOUTER>
    void product(int tile, const Operand& x, const Operand& y, uint32_t inner, uint32_t shares, const ProductOut& out) const {
        switch (tile) {
            case kBig: return product<TileProduct<E, 2, 4, 4, 2, 2, true, YOUTER>, O, PARTIAL>(x, y, inner, shares, out);
            case kMid: return product<TileProduct<E, 4, 2, 1, 2, 2, true, YOUTER>, O, PARTIAL>(x, y, inner, shares, out);
            default: return product<TileProduct<E, 4, 2, 1, 1, 4, true, YOUTER>, O, PARTIAL>(x, y, inner, shares, out);
        }
    }

    int forward() {
        if (direct<T>(a.hidden.p, a.hidden.stride, a.width)) {
            a.x = operand(a.hidden.p, a.hidden.stride, a.rows);
        } else {
            pack<T, E, PLANES>(a.hidden.p, a.hidden.stride, a.rows, a, l.line, ws + l.x, c.stream);
            a.x = operand(ws + l.x, l.line, a.rows);
        }
        const bool whole = direct<T>(a.weight.p, a.weight.stride, a.width);
        const uint32_t piece = whole ? a.words : l.piece;
        const int tile = tile_of(piece, a.rows);
        uint32_t tiles = 0;
        for (uint32_t word0 = 0; word0 < a.words; word0 += piece) {
            const Operand w = weight(word0, std::min(piece, a.words - word0));
            logits<false>(tile, w, word0, Operand{}, tiles);
            if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
            tiles += share_of(w.extent, kTileM[tile]);
        }
        if (c.distil) {
            hipLaunchKernelGGL(k_picks<T>, dim3(share_of(uint64_t(a.rows) * a.picks, 4)), dim3(256), 0, c.stream, a);
            if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
        }
        hipLaunchKernelGGL(k_loss<T>, dim3(share_of(a.rows, 4)), dim3(256), 0, c.stream, a, tiles);
        return launch_status();
    }

    int backward() {
        if (c.distil) {
            hipLaunchKernelGGL(k_row_counts, dim3(share_of(a.rows, 4)), dim3(256), 0, c.stream, a);
            if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
        }
        hipLaunchKernelGGL((k_loss_start<T, E, PLANES>), dim3(1 + share_of(uint64_t(a.rows) * (l.line / 8), 1024)), dim3(1024), 0,
                           c.stream, a, l.line, reinterpret_cast<E*>(ws + l.x));
        if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
        a.x = operand(ws + l.x, l.line, a.rows);
        for (uint32_t word0 = 0; word0 < a.words; word0 += l.piece) {
            const uint32_t words = std::min(l.piece, a.words - word0);
            const Operand w = weight(word0, words);
            const Operand dz{ws + l.dz, l.piece, uint64_t(a.rows) * l.piece, a.rows, words};
            logits<true>(tile_of(words, a.rows), w, word0, dz, 0);
            if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
            if (c.distil) {
                hipLaunchKernelGGL(k_pick_grad<E>, dim3(share_of(a.rows, 4)), dim3(256), 0, c.stream, a, word0, words, dz,
                                   l.dz_planes);
                if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
            }
            if (c.dhidden != nullptr) {
                const ProductOut out{ws + l.dx, l.line, a.rows, l.line, a.scale, word0 > 0};
                product<float, true, false>(tile_of(l.line, a.rows, l.shares), turned(w, l.line, words), dz, words, l.shares,
                                            out);
                if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
            }
            if (c.dweight != nullptr) {
                const ProductOut out{static_cast<T*>(c.dweight) + uint64_t(word0) * c.dweight_stride, c.dweight_stride, words,
                                     a.width, a.scale, false};
                product<T, false, true>(tile_of(a.width, words), turned(a.x, l.line, a.rows),
                                        turned(dz, uint32_t(up(words, 8)), a.rows), a.rows, 1, out);
                if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
            }
        }
        if (c.dhidden != nullptr)
            hipLaunchKernelGGL(k_join_shares<T>, dim3(blocks_of(uint64_t(a.rows) * (l.line / 4))), dim3(256), 0, c.stream,
                               reinterpret_cast<const float*>(ws + l.dx), l.shares, uint64_t(a.rows), a.width, l.line, a.scale,
                               static_cast<T*>(c.dhidden), c.dhidden_stride);
        return launch_status();
    }
};

template <typename T, typename E, int PLANES>
int launch_loss(const LossCall& c, const HeadLayout& l) {
    const adacomp_head& h = *c.head;
    char* ws = static_cast<char*>(c.ws);
    LossArgs a{};
    a.hidden = {h.hidden, h.hidden_stride};
    a.weight = {h.weight, h.weight_stride};
    a.ids = c.ids;
    a.teacher = c.teacher;
    a.loss = c.loss;
    a.lse = c.lse;
    a.picked = c.picked;
    a.dloss = c.dloss;
    a.factor = reinterpret_cast<float*>(ws + l.factor);
    a.scale = reinterpret_cast<float*>(ws + l.scale);
    a.counts = reinterpret_cast<uint32_t*>(ws + l.counts);
    a.part = reinterpret_cast<float2*>(ws + l.part);
    a.rows = uint32_t(h.rows);
    a.width = h.width;
    a.words = h.vocabulary;
    a.picks = c.picks;
    a.sharp = 1.f / c.temperature;
    Loss<T, E, PLANES> loss{c, l, a, ws};
    return c.back ? loss.backward() : loss.forward();
}

int run_loss(const LossCall& c) {
    int st = check_head(c.head, c.picks);
    if (st != ADACOMP_OK) return st;
    const adacomp_head& h = *c.head;
    const uint64_t size = type_size(h.type), R = h.rows;
    if (!(c.temperature > 0.f) || !std::isfinite(c.temperature) || !std::isfinite(1.f / c.temperature))
        return ADACOMP_ERR_INVALID_ARGUMENT;
    if ((st = check_matrix(h.hidden, h.hidden_stride, R, h.width, size)) != ADACOMP_OK) return st;
    if ((st = check_matrix(h.weight, h.weight_stride, h.vocabulary, h.width, size)) != ADACOMP_OK) return st;
    if (c.dhidden && (st = check_matrix(c.dhidden, c.dhidden_stride, R, h.width, size)) != ADACOMP_OK) return st;
    if (c.dweight && (st = check_matrix(c.dweight, c.dweight_stride, h.vocabulary, h.width, size)) != ADACOMP_OK) return st;
    const bool needs_loss = !c.back || !c.distil;   // the distillation's gradients go by picked
    if (R > 0 && (c.ids == nullptr || c.lse == nullptr || (needs_loss && c.loss == nullptr) ||
                  (c.distil && (c.teacher == nullptr || c.picked == nullptr)) || (c.back && c.dloss == nullptr)))
        return ADACOMP_ERR_INVALID_ARGUMENT;
    if (!aligned_to(c.ids, 8) || !aligned_to(c.teacher, 4) || !aligned_to(c.loss, 4) || !aligned_to(c.lse, 4) ||
        !aligned_to(c.picked, 4) || !aligned_to(c.dloss, 4) || !aligned16(c.ws))
        return ADACOMP_ERR_MISALIGNED;
    const HeadLayout l = head_layout(h, c.back);
    if (R > 0 && c.ws == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (R > 0 && c.ws_bytes < l.bytes) return ADACOMP_ERR_CAPACITY;
    const uint64_t rows4 = R * 4, picks4 = rows4 * c.picks;
    const Range r[12] = {range_of(c.back ? nullptr : c.loss, c.back || !c.loss ? 0 : rows4),
                         range_of(c.back ? nullptr : c.lse, c.back ? 0 : rows4),
                         range_of(c.back ? nullptr : c.picked, c.back || !c.picked ? 0 : picks4),
                         matrix_range(c.dhidden, c.dhidden_stride, R, h.width, size),
                         matrix_range(c.dweight, c.dweight_stride, h.vocabulary, h.width, size),
                         range_of(c.ws, R ? l.bytes : 0),
                         matrix_range(h.hidden, h.hidden_stride, R, h.width, size),
                         matrix_range(h.weight, h.weight_stride, h.vocabulary, h.width, size),
                         range_of(c.ids, 2 * picks4),
                         range_of(c.teacher, c.teacher ? picks4 : 0),
                         range_of(c.back ? c.loss : nullptr, c.back && c.loss ? rows4 : 0),
                         range_of(c.back ? c.lse : nullptr, c.back ? rows4 : 0)};
    if (outputs_clash(r, 6, 12)) return ADACOMP_ERR_INVALID_ARGUMENT;
    const Range in[2] = {range_of(c.back ? c.picked : nullptr, c.back && c.picked ? picks4 : 0),
                         range_of(c.dloss, c.dloss ? rows4 : 0)};
    for (int i = 0; i < 6; ++i)
        if (overlaps(r[i], in[0]) || overlaps(r[i], in[1])) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (R == 0) {
        if (c.dweight == nullptr) return ADACOMP_OK;
        const uint64_t V = h.vocabulary;
        const dim3 grid(blocks_of(std::min<uint64_t>(V * h.width, 1 << 24))), block(256);
        if (h.type == ADACOMP_FLOAT)
            hipLaunchKernelGGL(k_zero_rows<float>, grid, block, 0, c.stream, static_cast<float*>(c.dweight), c.dweight_stride, V,
                               h.width);
        else   // 0 has the same bits in both
            hipLaunchKernelGGL(k_zero_rows<f16>, grid, block, 0, c.stream, static_cast<f16*>(c.dweight), c.dweight_stride, V,
                               h.width);
        return launch_status();
    }
    if (h.type == ADACOMP_FLOAT) return launch_loss<float, bf16, 3>(c, l);
    if (h.type == ADACOMP_BFLOAT) return launch_loss<bf16, bf16, 1>(c, l);
    return launch_loss<f16, f16, 1>(c, l);
}

}  // namespace

extern "C" {

int adacomp_head_workspace_bytes(const adacomp_head* head, uint32_t picks, int backward, uint64_t* bytes) {
    if (bytes == nullptr || (backward != 0 && backward != 1)) return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = check_head(head, picks);
    if (st != ADACOMP_OK) return st;
    *bytes = head_layout(*head, false).bytes;
    if (backward) *bytes = std::max(*bytes, head_layout(*head, true).bytes);
    return ADACOMP_OK;
}

int adacomp_linear_cross_entropy(const adacomp_head* head, const int64_t* targets, float* loss, float* lse, void* ws,
                                 uint64_t ws_bytes, void* stream) {
    LossCall c{};
    c.head = head;
    c.ids = targets;
    c.picks = 1;
    c.temperature = 1.f;
    c.loss = loss;
    c.lse = lse;
    c.ws = ws;
    c.ws_bytes = ws_bytes;
    c.stream = static_cast<hipStream_t>(stream);
    return run_loss(c);
}

int adacomp_linear_cross_entropy_backward(const adacomp_head* head, const int64_t* targets, const float* loss,
                                          const float* lse, const float* dloss, void* dhidden, uint64_t dhidden_stride,
                                          void* dweight, uint64_t dweight_stride, void* ws, uint64_t ws_bytes,
                                          void* stream) {
    LossCall c{};
    c.head = head;
    c.ids = targets;
    c.picks = 1;
    c.temperature = 1.f;
    c.loss = const_cast<float*>(loss);
    c.lse = const_cast<float*>(lse);
    c.dloss = dloss;
    c.dhidden = dhidden;
    c.dhidden_stride = dhidden_stride;
    c.dweight = dweight;
    c.dweight_stride = dweight_stride;
    c.ws = ws;
    c.ws_bytes = ws_bytes;
    c.stream = static_cast<hipStream_t>(stream);
    c.back = true;
    return run_loss(c);
}

int adacomp_linear_distillation(const adacomp_head* head, const int64_t* ids, const float* teacher, uint32_t picks,
                                float temperature, float* loss, float* lse, float* picked, void* ws, uint64_t ws_bytes,
                                void* stream) {
    LossCall c{};
    c.head = head;
    c.ids = ids;
    c.teacher = teacher;
    c.picks = picks;
    c.temperature = temperature;
    c.loss = loss;
    c.lse = lse;
    c.picked = picked;
    c.ws = ws;
    c.ws_bytes = ws_bytes;
    c.stream = static_cast<hipStream_t>(stream);
    c.distil = true;
    return run_loss(c);
}

int adacomp_linear_distillation_backward(const adacomp_head* head, const int64_t* ids, const float* teacher, uint32_t picks,
                                         float temperature, const float* lse, const float* picked, const float* dloss,
                                         void* dhidden, uint64_t dhidden_stride, void* dweight, uint64_t dweight_stride,
                                         void* ws, uint64_t ws_bytes, void* stream) {
    LossCall c{};
    c.head = head;
    c.ids = ids;
    c.teacher = teacher;
    c.picks = picks;
    c.temperature = temperature;
    c.lse = const_cast<float*>(lse);
    c.picked = const_cast<float*>(picked);
    c.dloss = dloss;
    c.dhidden = dhidden;
    c.dhidden_stride = dhidden_stride;
    c.dweight = dweight;
    c.dweight_stride = dweight_stride;
    c.ws = ws;
    c.ws_bytes = ws_bytes;
    c.stream = static_cast<hipStream_t>(stream);
    c.back = true;
    c.distil = true;
    return run_loss(c);
}

}  // extern "C"
