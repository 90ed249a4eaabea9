// views.hpp against the elements themselves: pairs of small views of every
// shape, with random, nested, interleaved and overlapping strides and offsets.
// Prints the number of pairs of each kind, or the first pair whose answer is
// wrong (exit status 1).
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>

#include "../../adaptive_residual_gradient_amd/csrc/views.hpp"

using namespace adacomp;

static std::vector<uint64_t> rows_of(const adacomp_view& v, const adacomp_scan_shape& s, uint64_t size) {
    std::vector<uint64_t> at;
    for (uint64_t b = 0; b < s.batch; ++b)
        for (uint64_t t = 0; t < s.length; ++t)
            at.push_back(reinterpret_cast<uintptr_t>(v.data) / size + b * v.batch_stride + t * v.time_stride);
    return at;
}

int main() {
    std::mt19937 rng(7);
    auto pick = [&](uint64_t lo, uint64_t hi) { return lo + rng() % (hi - lo + 1); };
    long apart = 0, shared = 0, crossing = 0, folded = 0;
    for (int trial = 0; trial < 200000; ++trial) {
        const uint64_t size = rng() % 2 ? 4 : 2;
        adacomp_scan_shape s{};
        s.batch = uint32_t(pick(1, 4));
        s.length = pick(1, 5);
        s.channels = uint32_t(pick(1, 4));
        adacomp_view a{}, b{};
        const uint64_t C = s.channels;
        switch (rng() % 3) {
            case 0:   // sequences one after the other
                a.time_stride = pick(C, 3 * C);
                a.batch_stride = s.length * a.time_stride + pick(0, 2);
                break;
            case 1:   // time first
                a.batch_stride = pick(C, 3 * C);
                a.time_stride = s.batch * a.batch_stride + pick(0, 2);
                break;
            default:
                a.time_stride = pick(C, 6 * C);
                a.batch_stride = pick(0, 6 * C);
        }
        // an axis of one place may have any stride
        if (s.length == 1) a.time_stride = pick(C, 20);
        if (s.batch == 1) a.batch_stride = pick(0, 20);
        b.time_stride = a.time_stride;
        b.batch_stride = a.batch_stride;
        if (s.length == 1 && rng() % 2) b.time_stride = pick(C, 20);
        if (s.batch == 1 && rng() % 2) b.batch_stride = pick(0, 20);
        const uint64_t base = 4096;
        a.data = reinterpret_cast<void*>((base + pick(0, 60)) * size);
        b.data = reinterpret_cast<void*>((base + pick(0, 60)) * size);

        const auto ra = rows_of(a, s, size), rb = rows_of(b, s, size);
        std::set<uint64_t> elements;
        bool meets = false;
        for (const uint64_t r : ra)
            for (uint64_t c = 0; c < C; ++c) meets |= !elements.insert(r + c).second;
        bool clash = false;
        for (const uint64_t r : rb)
            for (uint64_t c = 0; c < C; ++c) clash |= elements.count(r + c) > 0;
        RowGrid g;
        const bool grid = row_grid(a, s, g), said = views_clash(a, b, s, size);
        // rows that meet are always told, and nested rows are never said to meet; of rows that are
        // neither, nothing is promised
        const bool nested = s.batch == 1 || s.length == 1 || a.batch_stride >= (s.length - 1) * a.time_stride + C ||
                            (a.batch_stride >= C && a.time_stride >= (s.batch - 1) * a.batch_stride + C);
        const bool wrong = (meets && grid) || (nested && !meets && !grid) || (clash && !said) || (grid && !clash && said);
        if (wrong) {
            std::printf("FAIL size %d B %u T %d C %u bs %d ts %d offset %d: meets %d grid %d clash %d said %d\n", int(size),
                        s.batch, int(s.length), s.channels, int(a.batch_stride), int(a.time_stride),
                        int((reinterpret_cast<intptr_t>(b.data) - reinterpret_cast<intptr_t>(a.data)) / intptr_t(size)),
                        meets, grid, clash, said);
            return 1;
        }
        folded += !grid;
        shared += grid && clash;
        crossing += grid && !clash && overlaps(view_range(a, s, size), view_range(b, s, size));
        apart += grid && !clash;
    }
    std::printf("OK apart %ld (ranges crossing %ld) shared %ld folded %ld\n", apart, crossing, shared, folded);
    return crossing > 1000 && shared > 1000 && folded > 1000 ? 0 : 1;
}
