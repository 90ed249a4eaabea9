// Where the rows of a scan's [batch, length, channels] views lie, and whether
// two views share an element.  No HIP call.
#pragma once

#include <cstdint>

#include "../../include/adacomp.h"
#include "ranges.hpp"

namespace adacomp {

// The rows of a view as an outer and an inner axis whose rows do not meet: the
// outer stride is at least the reach of the inner rows.  Strides of axes of one
// place are never stepped and do not count.
struct RowGrid {
    uint64_t outer = 0, inner = 0;     // strides
    uint64_t nouter = 1, ninner = 1;   // places
};

// The rows' extent: sequences, steps, and the elements of a row.
struct RowSpace {
    uint64_t batch, length, width;
};

// False where rows meet (a batch stride of 0 of several sequences, say).  Needs length and batch > 0.
inline bool row_grid(const adacomp_view& v, const RowSpace& s, RowGrid& g) {
    const uint64_t B = s.batch, T = s.length, C = s.width, bs = v.batch_stride, ts = v.time_stride;
    g = RowGrid{};
    if (B == 1 || T == 1) {
        g.inner = B == 1 ? ts : bs;
        g.ninner = B == 1 ? T : B;
        return g.ninner == 1 || g.inner >= C;
    }
    if (ts >= C && bs >= (T - 1) * ts + C) g = {bs, ts, B, T};
    else if (bs >= C && ts >= (B - 1) * bs + C) g = {ts, bs, T, B};
    else return false;
    return true;
}

inline Range view_range(const adacomp_view& v, const RowSpace& s, uint64_t size) {
    return range_of(v.data, size * ((s.batch - 1) * v.batch_stride + (s.length - 1) * v.time_stride + s.width));
}

// Whether two views of the same batch and length may share an element; the
// answer is exact where both have the same strides: views side by side in the
// same rows (parts of one projection) do not, though their ranges cross.
inline bool views_clash(const adacomp_view& a, const RowSpace& sa, const adacomp_view& b, const RowSpace& sb,
                        uint64_t size) {
    if (!overlaps(view_range(a, sa, size), view_range(b, sb, size))) return false;
    RowGrid ga, gb;
    if (!row_grid(a, sa, ga) || !row_grid(b, sb, gb)) return true;
    if ((ga.nouter > 1 && (ga.outer != gb.outer || gb.nouter != ga.nouter)) ||
        (ga.ninner > 1 && (ga.inner != gb.inner || gb.ninner != ga.ninner)))
        return true;
    const int64_t d = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.data)) -
                       static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.data))) / static_cast<int64_t>(size);
    // rows i outer and j inner places apart share an element if b's begins less than a's width behind
    // a's or a's less than b's width behind b's, which leaves the two nearest i and, for each, the two
    // nearest j
    const auto near = [](int64_t x, uint64_t stride, uint64_t places, int64_t out[2]) {
        if (places == 1) {
            out[0] = out[1] = 0;
            return;
        }
        const int64_t t = static_cast<int64_t>(stride);
        out[0] = x / t - (x % t < 0);
        out[1] = out[0] + 1;
    };
    const auto within = [](int64_t i, uint64_t places) { return (i < 0 ? -i : i) < static_cast<int64_t>(places); };
    int64_t is[2], js[2];
    near(d, ga.outer, ga.nouter, is);
    for (const int64_t i : is) {
        if (!within(i, ga.nouter)) continue;
        const int64_t r = d - i * static_cast<int64_t>(ga.outer);
        near(r, ga.inner, ga.ninner, js);
        for (const int64_t j : js) {
            const int64_t gap = r - j * static_cast<int64_t>(ga.inner);
            if (within(j, ga.ninner) && gap < static_cast<int64_t>(sa.width) && -gap < static_cast<int64_t>(sb.width))
                return true;
        }
    }
    return false;
}

// The same of the gated scan's views, which have one shape.
inline RowSpace row_space(const adacomp_scan_shape& s) { return RowSpace{s.batch, s.length, s.channels}; }
inline bool row_grid(const adacomp_view& v, const adacomp_scan_shape& s, RowGrid& g) {
    return row_grid(v, row_space(s), g);
}
inline Range view_range(const adacomp_view& v, const adacomp_scan_shape& s, uint64_t size) {
    return view_range(v, row_space(s), size);
}
inline bool views_clash(const adacomp_view& a, const adacomp_view& b, const adacomp_scan_shape& s, uint64_t size) {
    return views_clash(a, row_space(s), b, row_space(s), size);
}

}  // namespace adacomp
