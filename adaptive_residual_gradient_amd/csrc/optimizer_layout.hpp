// Host layout of an optimizer's tensor table: validation, moment blocks and
// the work tiles its kernels run on.  No HIP call.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "../../include/adacomp.h"

namespace adacomp {

// Elements of one work tile: 256 threads of one float4 each.  A multiple of the
// moment block, so tiles of one tensor hold whole blocks.  Small tiles keep the
// addresses in flight on the chip close together: a plain copy of 1.07 GB in
// workgroups of 4, 16 and 32 KB runs at 6.5, 6.3 and 4.4 TB/s.
constexpr uint32_t kOptThreads = 256;
constexpr uint32_t kOptTileElems = kOptThreads * 4;
static_assert(kOptTileElems % ADACOMP_MOMENT_BLOCK == 0, "tiles hold whole moment blocks");

// Most workgroups of the norm's first pass, each one float64 partial sum.
constexpr uint32_t kNormMaxBlocks = 2048;

// One work tile: consecutive elements of one tensor.
struct OptTile {
    uint64_t elem;    // first element in the flat buffers
    uint64_t block;   // its first moment block
    uint32_t count;   // elements, 1..kOptTileElems
    float weight_decay;
    float lr_scale;
    uint32_t pad;
};

struct OptLayout {
    std::vector<OptTile> tiles;
    adacomp_optimizer_info info{};
};

inline int build_optimizer(const adacomp_tensor* t, uint32_t n, bool with_tiles, OptLayout& L) {
    if (t == nullptr || n == 0) return ADACOMP_ERR_INVALID_ARGUMENT;
    std::vector<std::pair<uint64_t, uint64_t>> ends(n);
    uint64_t ntiles = 0;
    L.info.ntensors = n;
    for (uint32_t i = 0; i < n; ++i) {
        if (t[i].numel == 0 || !std::isfinite(t[i].weight_decay) || !std::isfinite(t[i].lr_scale))
            return ADACOMP_ERR_INVALID_ARGUMENT;
        if (t[i].offset % 4 != 0) return ADACOMP_ERR_MISALIGNED;
        if (t[i].numel >= (uint64_t(1) << 40) || t[i].offset >= (uint64_t(1) << 40))
            return ADACOMP_ERR_TOO_LARGE;
        ends[i] = {t[i].offset, t[i].offset + t[i].numel};
        ntiles += (t[i].numel + kOptTileElems - 1) / kOptTileElems;
        L.info.total_numel += t[i].numel;
        L.info.nblocks += (t[i].numel + ADACOMP_MOMENT_BLOCK - 1) / ADACOMP_MOMENT_BLOCK;
        L.info.span = std::max(L.info.span, (ends[i].second + 3) / 4 * 4);
    }
    std::sort(ends.begin(), ends.end());
    for (uint32_t i = 1; i < n; ++i)
        if (ends[i].first < ends[i - 1].second) return ADACOMP_ERR_OVERLAP;
    // work-items of one launch must fit in 32 bits
    if (ntiles * kOptThreads >= (uint64_t(1) << 32)) return ADACOMP_ERR_TOO_LARGE;
    L.info.norm_workspace_bytes = 8 * std::min<uint64_t>(ntiles, kNormMaxBlocks);
    if (!with_tiles) return ADACOMP_OK;
    L.tiles.reserve(ntiles);
    uint64_t block = 0;
    for (uint32_t i = 0; i < n; ++i) {
        for (uint64_t at = 0; at < t[i].numel; at += kOptTileElems) {
            const uint32_t count = static_cast<uint32_t>(std::min<uint64_t>(kOptTileElems, t[i].numel - at));
            L.tiles.push_back({t[i].offset + at, block, count, t[i].weight_decay, t[i].lr_scale, 0});
            block += (count + ADACOMP_MOMENT_BLOCK - 1) / ADACOMP_MOMENT_BLOCK;
        }
    }
    return ADACOMP_OK;
}

}  // namespace adacomp
