// C ABI of the causal convolution and the selective scan (declared in
// include/adacomp.h): argument checking and stream-ordered kernel launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/adacomp.h"
#include "causal_conv.hpp"
#include "host_checks.hpp"
#include "selective_scan.hpp"
#include "views.hpp"

using namespace adacomp;

namespace {

constexpr uint64_t kItems = uint64_t(1) << 32;   // work-items that one launch may not reach

// One view of a call: elements, or NULL where it is absent.
struct CallView {
    const adacomp_view* v;
    uint32_t width;
};

int check_sizes(uint64_t length, uint32_t batch, uint32_t channels) {
    if (channels == 0) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (length >= (uint64_t(1) << 31) || channels >= (1u << 24) || batch >= (1u << 24) ||
        uint64_t(batch) * channels >= (uint64_t(1) << 31))
        return ADACOMP_ERR_TOO_LARGE;
    return ADACOMP_OK;
}

// Views (outputs first) and plain ranges (outputs first) of one call: where each lies, and that no output
// shares an element with anything else.
template <int NV, int NR>
int check_buffers(uint64_t length, uint32_t batch, uint64_t size, const CallView (&views)[NV], int view_outputs,
                  const Range (&ranges)[NR], int range_outputs) {
    const bool steps = length > 0;   // without steps no view is touched
    const auto space = [&](const CallView& c) { return RowSpace{batch, length, c.width}; };
    for (int i = 0; i < NV && steps; ++i) {
        const adacomp_view* v = views[i].v;
        if (v == nullptr) continue;
        if (v->data == nullptr || v->time_stride < views[i].width) return ADACOMP_ERR_INVALID_ARGUMENT;
        if (!aligned_to(v->data, size)) return ADACOMP_ERR_MISALIGNED;
        if (v->time_stride >= (uint64_t(1) << 32) || v->batch_stride >= (uint64_t(1) << 40)) return ADACOMP_ERR_TOO_LARGE;
        RowGrid rows;   // an output's rows may not meet
        if (i < view_outputs && !row_grid(*v, space(views[i]), rows)) return ADACOMP_ERR_INVALID_ARGUMENT;
    }
    for (int i = 0; i < NV && steps; ++i) {
        if (views[i].v == nullptr) continue;
        for (int j = i + 1; j < NV; ++j)
            if (i < view_outputs && views[j].v != nullptr &&
                views_clash(*views[i].v, space(views[i]), *views[j].v, space(views[j]), size))
                return ADACOMP_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < NR; ++j)
            if ((i < view_outputs || j < range_outputs) && overlaps(view_range(*views[i].v, space(views[i]), size), ranges[j]))
                return ADACOMP_ERR_INVALID_ARGUMENT;
    }
    return outputs_clash(ranges, range_outputs, NR) ? ADACOMP_ERR_INVALID_ARGUMENT : ADACOMP_OK;
}

ScanView dev_view(const adacomp_view* v) {
    return v ? ScanView{v->data, v->batch_stride, v->time_stride} : ScanView{};
}

uint32_t blocks_of(uint64_t items) { return static_cast<uint32_t>((items + 255) / 256); }

// ---- causal convolution ----

int check_conv(const adacomp_conv_shape* s) {
    if (s == nullptr || type_size(s->type) == 0 || s->taps == 0 || s->taps > ADACOMP_CONV_MAX_TAPS ||
        (s->silu != 0 && s->silu != 1))
        return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = check_sizes(s->length, s->batch, s->channels);
    if (st != ADACOMP_OK) return st;
    const uint64_t vec = kConvBytes / type_size(s->type), lanes = (s->channels + vec - 1) / vec;
    if (s->batch * lanes * ((s->length + kConvRows[2] - 1) / kConvRows[2] + 1) >= kItems) return ADACOMP_ERR_TOO_LARGE;
    return ADACOMP_OK;
}

// Channels of a thread: a vector, or one where there are fewer channels than it has.
uint32_t conv_vec(const adacomp_conv_shape& s) {
    const uint32_t vec = kConvBytes / uint32_t(type_size(s.type));
    return s.channels < vec ? 1 : vec;
}

struct ConvBackLayout {
    uint32_t lanes, per, groups, rows, pieces, parts;
};
// Stretches: as many as workgroups of kConvMaxPartials partial rows hold, of 32 steps or more.
ConvBackLayout conv_back_layout(const adacomp_conv_shape& s) {
    ConvBackLayout l{};
    const uint32_t vec = conv_vec(s);
    l.lanes = (s.channels + vec - 1) / vec;
    l.groups = (l.lanes + kConvThreads - 1) / kConvThreads;
    l.per = (l.lanes + l.groups - 1) / l.groups;
    const uint64_t subs = kConvThreads / l.per, most = subs * kConvMaxPartials;
    const uint64_t each = std::max<uint64_t>(most / s.batch, 1);   // stretches of a sequence
    const uint64_t rows = std::max<uint64_t>((s.length + each - 1) / each, 32);
    l.rows = static_cast<uint32_t>(rows);
    l.pieces = static_cast<uint32_t>(std::max<uint64_t>((s.length + rows - 1) / rows, 1));
    l.parts = static_cast<uint32_t>((uint64_t(s.batch) * l.pieces + subs - 1) / subs);
    return l;
}

template <typename T, int VW, int KT>
void launch_conv(ConvArgs a, bool silu, hipStream_t s) {
    // at least 2 wavefronts a SIMD
    const auto threads = [&](uint32_t rows) { return a.batch * uint64_t(a.lanes) * ((a.length + rows - 1) / rows); };
    const int pick = threads(kConvRows[0]) >= 2 * 1024 * 64 ? 0 : threads(kConvRows[1]) >= 2 * 1024 * 64 ? 1 : 2;
    a.pieces = static_cast<uint32_t>(std::max<uint64_t>((a.length + kConvRows[pick] - 1) / kConvRows[pick], 1));
    const dim3 grid(blocks_of(uint64_t(a.batch) * a.lanes * a.pieces)), block(kConvThreads);
    if (pick == 0) hipLaunchKernelGGL((k_conv<T, VW, KT, kConvRows[0]>), grid, block, 0, s, a, silu);
    else if (pick == 1) hipLaunchKernelGGL((k_conv<T, VW, KT, kConvRows[1]>), grid, block, 0, s, a, silu);
    else hipLaunchKernelGGL((k_conv<T, VW, KT, kConvRows[2]>), grid, block, 0, s, a, silu);
}

template <typename T, int VW>
void launch_conv_taps(const ConvArgs& a, bool silu, hipStream_t s) {
    switch (conv_kernel_taps(a.taps)) {
        case 2: return launch_conv<T, VW, 2>(a, silu, s);
        case 3: return launch_conv<T, VW, 3>(a, silu, s);
        case 4: return launch_conv<T, VW, 4>(a, silu, s);
        default: return launch_conv<T, VW, 8>(a, silu, s);
    }
}

template <typename T>
void launch_conv_back(const ConvArgs& a, const ConvBackLayout& l, uint32_t vec, bool silu, hipStream_t s) {
    constexpr int V = kConvBytes / sizeof(T);
    const dim3 grid(l.parts * l.groups), block(kConvThreads);
#define ADACOMP_CONV_BACK(VW, KT)                                                        \
    do {                                                                                 \
        if (vec == 1) hipLaunchKernelGGL((k_conv_backward<T, 1, KT>), grid, block, 0, s, a, silu); \
        else hipLaunchKernelGGL((k_conv_backward<T, VW, KT>), grid, block, 0, s, a, silu);         \
    } while (0)
    switch (conv_kernel_taps(a.taps)) {
        case 2: ADACOMP_CONV_BACK(V, 2); break;
        case 3: ADACOMP_CONV_BACK(V, 3); break;
        case 4: ADACOMP_CONV_BACK(V, 4); break;
        default: ADACOMP_CONV_BACK(V, 8);
    }
#undef ADACOMP_CONV_BACK
}

// ---- selective scan ----

struct SsmLayout {
    uint32_t padded, nb, groups, chunks, steps;   // nb: states of a forward wavefront
    uint64_t rows, ends, sums, steps_of, part_rows, part_a, bytes;   // byte offsets
};

SsmLayout ssm_layout(const adacomp_ssm_shape& s, bool back) {
    SsmLayout l{};
    l.nb = s.states <= 8 ? 8 : kSsmBlock;
    l.padded = (s.states + l.nb - 1) / l.nb * l.nb;
    l.groups = (s.channels + 63) / 64;
    // Chunks: for 4 wavefronts a SIMD, of 32 steps or more; where these leave less than 2, for 2, of 16 or more; where
    // these leave less than 1, for 1, of 8 or more (forward of 1 x 2048 x 2048: 77 us, of 64 steps or more 105, of 16 83;
    // of 2 x 300 x 1024: 37 us, of 32 or more 53).
    const uint64_t waves = std::max<uint64_t>(uint64_t(s.batch) * l.groups * (l.padded / l.nb), 1);
    uint64_t chunks = 1;
    for (const uint64_t least : {32, 16, 8}) {
        const uint64_t want = 128 * least;   // 4, 2 and 1 a SIMD
        chunks = std::max<uint64_t>(std::min<uint64_t>((want + waves - 1) / waves, (s.length + least - 1) / least), chunks);
        if (chunks * waves >= want / 2) break;
    }
    const uint64_t steps = ((s.length + chunks - 1) / chunks + kSsmKeep - 1) / kSsmKeep * kSsmKeep;
    l.steps = static_cast<uint32_t>(std::max<uint64_t>(steps, kSsmKeep));
    l.chunks = static_cast<uint32_t>(std::max<uint64_t>((s.length + l.steps - 1) / l.steps, 1));
    auto place = [&](uint64_t floats) {
        const uint64_t at = l.bytes;
        l.bytes += (floats * 4 + 255) / 256 * 256;
        return at;
    };
    const uint64_t B = s.batch, C = s.channels, rows = B * s.length * 2 * l.padded;
    l.rows = place(rows);
    l.ends = place(l.chunks > 1 ? B * l.chunks * l.padded * C : 0);
    l.sums = place(l.chunks > 1 ? B * l.chunks * C : 0);
    l.steps_of = place(!back && l.chunks > 1 ? B * s.length * C : 0);
    if (back) {
        l.part_rows = place(rows * l.groups);
        l.part_a = place(B * l.chunks * (l.padded + 2) * C);
    }
    return l;
}
uint64_t ssm_kept_bytes(const adacomp_ssm_shape& s) {
    return 4 * uint64_t(s.batch) * ((s.length + kSsmKeep - 1) / kSsmKeep) * ssm_layout(s, false).padded * s.channels;
}

// The launches' grids fit in 32 bits of work-items.
bool ssm_fits(const adacomp_ssm_shape& s, const SsmLayout& l) {
    const uint64_t B = s.batch, blocks = l.padded / l.nb, per = std::max<uint64_t>(4 / blocks, 1);   // as SsmGrid's
    const uint64_t waves = std::max((l.groups + per - 1) / per * per * blocks, uint64_t(l.groups) * (l.padded / kSsmBackBlock));
    return B * s.length * 2 * l.padded < kItems && B * l.padded * s.channels < kItems && B * l.chunks * waves * 64 < kItems &&
           B * s.channels * 16 < kItems;
}

int check_ssm(const adacomp_ssm_shape* s) {
    if (s == nullptr || type_size(s->type) == 0 || s->states == 0 || (s->softplus != 0 && s->softplus != 1))
        return ADACOMP_ERR_INVALID_ARGUMENT;
    if (s->states > ADACOMP_SCAN_MAX_STATES) return ADACOMP_ERR_TOO_LARGE;
    const int st = check_sizes(s->length, s->batch, s->channels);
    if (st != ADACOMP_OK) return st;
    return ssm_fits(*s, ssm_layout(*s, false)) ? ADACOMP_OK : ADACOMP_ERR_TOO_LARGE;
}

void ssm_args(SsmArgs& a, const adacomp_ssm_shape& s, const adacomp_ssm_inputs& in, const SsmLayout& l, void* ws) {
    a.x = dev_view(&in.x);
    a.dt = dev_view(&in.dt);
    a.z = dev_view(&in.z);
    a.b = dev_view(&in.b);
    a.c = dev_view(&in.c);
    a.a = in.a;
    a.d = in.d;
    a.dt_bias = in.dt_bias;
    a.lengths = in.lengths;
    a.length = s.length;
    a.batch = s.batch;
    a.channels = s.channels;
    a.states = s.states;
    a.padded = l.padded;
    a.chunks = l.chunks;
    a.steps = l.steps;
    a.groups = l.groups;
    a.softplus = s.softplus != 0;
    char* p = static_cast<char*>(ws);
    a.rows = reinterpret_cast<float*>(p + l.rows);
    a.ends = reinterpret_cast<float*>(p + l.ends);
    a.sums = reinterpret_cast<float*>(p + l.sums);
    a.steps_of = reinterpret_cast<float*>(p + l.steps_of);
}

// Workgroups of 4 wavefronts or so: the blocks of one group of channels, of as many groups as fit.
struct SsmGrid {
    dim3 grid, block;
    SsmGrid(const SsmArgs& a) {
        const uint32_t per = std::max(4 / a.blocks, 1u);
        grid = dim3((a.groups + per - 1) / per * a.chunks * a.batch);
        block = dim3(64 * per * a.blocks);
    }
};

template <typename T, int NB>
int launch_ssm(SsmArgs a, hipStream_t s) {
    hipLaunchKernelGGL(k_ssm_rows<T>, dim3(blocks_of(uint64_t(a.batch) * a.length * 2 * a.padded)), dim3(256), 0, s, a);
    if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
    a.blocks = a.padded / NB;
    const SsmGrid g(a);
    const uint32_t lds = a.blocks > 1 ? 2 * g.block.x * kSsmKeep * 4 : 0;
#define ADACOMP_SSM(MODE)                                                                                          \
    do {                                                                                                           \
        if (a.z.p != nullptr) hipLaunchKernelGGL((k_ssm_forward<T, NB, MODE, true>), g.grid, g.block, lds, s, a);  \
        else hipLaunchKernelGGL((k_ssm_forward<T, NB, MODE, false>), g.grid, g.block, lds, s, a);                  \
    } while (0)
    if (a.chunks == 1) {
        ADACOMP_SSM(kSsmWhole);
        return launch_status();
    }
    hipLaunchKernelGGL((k_ssm_forward<T, NB, kSsmEnds, false>), g.grid, g.block, 0, s, a);
    if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
    hipLaunchKernelGGL(k_ssm_join<false>, dim3(blocks_of(uint64_t(a.batch) * a.padded * a.channels)), dim3(256), 0, s, a);
    if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
    ADACOMP_SSM(kSsmChunks);
#undef ADACOMP_SSM
    return launch_status();
}

template <typename T>
int launch_ssm(const SsmArgs& a, uint32_t nb, hipStream_t s) {
    if (a.kept == nullptr && a.length <= kSsmShort) {
        uint32_t quads = 1;
        while (quads * 4 < a.states) quads *= 2;
        hipLaunchKernelGGL(k_ssm_short<T>, dim3(blocks_of(uint64_t(a.batch) * a.channels * quads)), dim3(256), 0, s, a,
                           quads);
        return launch_status();
    }
    return nb == 8 ? launch_ssm<T, 8>(a, s) : launch_ssm<T, 16>(a, s);
}

template <typename T, bool GATED>
int launch_ssm_back(SsmArgs a, uint32_t nb, hipStream_t s) {
    if (a.chunks > 1) {
        a.blocks = a.padded / nb;
        const SsmGrid g(a);
        if (nb == 8) hipLaunchKernelGGL((k_ssm_back_ends<T, 8, GATED>), g.grid, g.block, 0, s, a);
        else hipLaunchKernelGGL((k_ssm_back_ends<T, 16, GATED>), g.grid, g.block, 0, s, a);
        if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
        hipLaunchKernelGGL(k_ssm_join<true>, dim3(blocks_of(uint64_t(a.batch) * a.padded * a.channels)), dim3(256), 0, s, a);
        if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
    }
    a.blocks = a.padded / kSsmBackBlock;   // 2, 4, 8, 12 or 16
    const dim3 grid(a.groups * a.chunks * a.batch), block(64 * a.blocks);
    const uint32_t lds = (3 + a.blocks * (GATED ? 3 : 2)) * kSsmKeep * 64 * 4;
    if (a.blocks == 2) hipLaunchKernelGGL((k_ssm_backward<T, 4, GATED>), grid, block, lds, s, a);
    else if (a.blocks == 4) hipLaunchKernelGGL((k_ssm_backward<T, 2, GATED>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((k_ssm_backward<T, 1, GATED>), grid, block, lds, s, a);
    return launch_status();
}

template <typename T>
int launch_ssm_back(const SsmArgs& a, uint32_t nb, const adacomp_ssm_gradients& out, hipStream_t s) {
    const uint64_t rows = uint64_t(a.batch) * a.length * 2 * a.padded;
    if (rows > 0) {
        hipLaunchKernelGGL(k_ssm_rows<T>, dim3(blocks_of(rows)), dim3(256), 0, s, a);
        if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
    }
    const int st = a.z.p != nullptr ? launch_ssm_back<T, true>(a, nb, s) : launch_ssm_back<T, false>(a, nb, s);
    if (st != ADACOMP_OK) return st;
    if (rows > 0) {
        hipLaunchKernelGGL(k_ssm_row_grad<T>, dim3(blocks_of(rows)), dim3(256), 0, s, a);
        if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
    }
    hipLaunchKernelGGL(k_ssm_channel_grad, dim3((a.channels + 15) / 16, a.padded + 2), dim3(256), 0, s, a.part_a,
                       a.batch * a.chunks, a.padded, a.states, a.channels, out.da, out.dd, out.ddt_bias);
    return launch_status();
}

int check_ssm_inputs(const adacomp_ssm_shape* s, const adacomp_ssm_inputs* in) {
    const int st = check_ssm(s);
    if (st != ADACOMP_OK) return st;
    if (in == nullptr || in->a == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (!aligned_to(in->a, 4) || !aligned_to(in->d, 4) || !aligned_to(in->dt_bias, 4) || !aligned_to(in->lengths, 4))
        return ADACOMP_ERR_MISALIGNED;
    return ADACOMP_OK;
}

}  // namespace

extern "C" {

int adacomp_causal_conv(const adacomp_conv_shape* shape, const adacomp_view* x, const float* weight, const float* bias,
                        const adacomp_view* y, const void* state, void* state_out, const int32_t* lengths,
                        void* stream) {
    int st = check_conv(shape);
    if (st != ADACOMP_OK) return st;
    const adacomp_conv_shape& s = *shape;
    if (weight == nullptr || (s.length > 0 && (x == nullptr || y == nullptr))) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (s.batch == 0) return ADACOMP_OK;
    const uint64_t size = type_size(s.type), kept = uint64_t(s.batch) * (s.taps - 1) * s.channels * size, C = s.channels;
    if (!aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(state, size) || !aligned_to(state_out, size) ||
        !aligned_to(lengths, 4))
        return ADACOMP_ERR_MISALIGNED;
    const CallView views[2] = {{y, s.channels}, {x, s.channels}};
    const Range ranges[5] = {range_of(state_out, state_out ? kept : 0), range_of(state, state ? kept : 0),
                             range_of(weight, 4 * C * s.taps), range_of(bias, bias ? 4 * C : 0),
                             range_of(lengths, lengths ? 4 * uint64_t(s.batch) : 0)};
    if ((st = check_buffers(s.length, s.batch, size, views, 1, ranges, 1)) != ADACOMP_OK) return st;
    ConvArgs a{};
    a.x = dev_view(x);
    a.y = dev_view(y);
    a.weight = weight;
    a.bias = bias;
    a.state = state;
    a.state_out = state_out;
    a.lengths = lengths;
    a.length = s.length;
    a.batch = s.batch;
    a.channels = s.channels;
    a.taps = s.taps;
    a.past = s.batch * s.length * s.channels * size > kKeepBytes;
    const uint32_t vec = conv_vec(s);
    a.lanes = (s.channels + vec - 1) / vec;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    const bool silu = s.silu != 0;
    if (s.type == ADACOMP_FLOAT) vec == 1 ? launch_conv_taps<float, 1>(a, silu, hs) : launch_conv_taps<float, 2>(a, silu, hs);
    else if (s.type == ADACOMP_BFLOAT) vec == 1 ? launch_conv_taps<bf16, 1>(a, silu, hs) : launch_conv_taps<bf16, 4>(a, silu, hs);
    else vec == 1 ? launch_conv_taps<f16, 1>(a, silu, hs) : launch_conv_taps<f16, 4>(a, silu, hs);
    return launch_status();
}

int adacomp_causal_conv_workspace_bytes(const adacomp_conv_shape* shape, uint64_t* bytes) {
    if (bytes == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = check_conv(shape);
    if (st != ADACOMP_OK) return st;
    *bytes = shape->batch ? uint64_t(conv_back_layout(*shape).parts) * (shape->taps + 1) * shape->channels * 4 : 0;
    return ADACOMP_OK;
}

int adacomp_causal_conv_backward(const adacomp_conv_shape* shape, const adacomp_view* dy, const adacomp_view* x,
                                 const float* weight, const float* bias, const adacomp_view* dx, float* dweight,
                                 float* dbias, const void* state, void* dstate, const int32_t* lengths, void* ws,
                                 uint64_t ws_bytes, void* stream) {
    int st = check_conv(shape);
    if (st != ADACOMP_OK) return st;
    const adacomp_conv_shape& s = *shape;
    if (weight == nullptr || dweight == nullptr ||
        (s.batch > 0 && s.length > 0 && (x == nullptr || dy == nullptr || dx == nullptr)))
        return ADACOMP_ERR_INVALID_ARGUMENT;
    const uint64_t size = type_size(s.type), C = s.channels, kept = uint64_t(s.batch) * (s.taps - 1) * C * size;
    if (!aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4) ||
        !aligned_to(state, size) || !aligned_to(dstate, size) || !aligned_to(lengths, 4) || !aligned16(ws))
        return ADACOMP_ERR_MISALIGNED;
    ConvBackLayout l{};
    if (s.batch > 0) l = conv_back_layout(s);
    const uint64_t need = uint64_t(l.parts) * (s.taps + 1) * C * 4;
    if (need > 0 && ws == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (ws_bytes < need) return ADACOMP_ERR_CAPACITY;
    const CallView views[3] = {{dx, s.channels}, {dy, s.channels}, {x, s.channels}};
    const Range ranges[8] = {range_of(dweight, 4 * C * s.taps), range_of(dbias, dbias ? 4 * C : 0),
                             range_of(dstate, dstate ? kept : 0), range_of(ws, need), range_of(state, state ? kept : 0),
                             range_of(weight, 4 * C * s.taps), range_of(bias, bias ? 4 * C : 0),
                             range_of(lengths, lengths ? 4 * uint64_t(s.batch) : 0)};
    if ((st = check_buffers(s.batch ? s.length : 0, s.batch, size, views, 1, ranges, 4)) != ADACOMP_OK) return st;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    ConvArgs a{};
    a.x = dev_view(x);
    a.dy = dev_view(dy);
    a.dx = dev_view(dx);
    a.weight = weight;
    a.bias = bias;
    a.state = state;
    a.dstate = dstate;
    a.lengths = lengths;
    a.partial = static_cast<float*>(ws);
    a.length = s.length;
    a.batch = s.batch;
    a.channels = s.channels;
    a.taps = s.taps;
    a.past = s.batch * s.length * s.channels * size > kKeepBytes;
    a.lanes = l.lanes;
    a.per = l.per;
    a.pieces = l.pieces;
    a.rows = l.rows;
    if (s.batch > 0) {
        const uint32_t vec = conv_vec(s);
        if (s.type == ADACOMP_FLOAT) launch_conv_back<float>(a, l, vec, s.silu != 0, hs);
        else if (s.type == ADACOMP_BFLOAT) launch_conv_back<bf16>(a, l, vec, s.silu != 0, hs);
        else launch_conv_back<f16>(a, l, vec, s.silu != 0, hs);
        if ((st = launch_status()) != ADACOMP_OK) return st;
    }
    hipLaunchKernelGGL(k_conv_weight_grad, dim3((s.channels + 15) / 16, s.taps + 1), dim3(1024), 0, hs, a.partial, l.parts,
                       s.taps, s.channels, dweight, dbias);
    return launch_status();
}

int adacomp_selective_scan_workspace_bytes(const adacomp_ssm_shape* shape, int backward, uint64_t* bytes) {
    if (bytes == nullptr || (backward != 0 && backward != 1)) return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = check_ssm(shape);
    if (st != ADACOMP_OK) return st;
    // a workspace of the backward call serves the forward call too
    *bytes = ssm_layout(*shape, false).bytes;
    if (backward) *bytes = std::max(*bytes, ssm_layout(*shape, true).bytes);
    return ADACOMP_OK;
}

int adacomp_selective_scan_kept_bytes(const adacomp_ssm_shape* shape, uint64_t* bytes) {
    if (bytes == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = check_ssm(shape);
    if (st != ADACOMP_OK) return st;
    *bytes = ssm_kept_bytes(*shape);
    return ADACOMP_OK;
}

int adacomp_selective_scan(const adacomp_ssm_shape* shape, const adacomp_ssm_inputs* inputs, const adacomp_view* y,
                           const float* h0, float* h_last, float* kept, void* ws, uint64_t ws_bytes, void* stream) {
    int st = check_ssm_inputs(shape, inputs);
    if (st != ADACOMP_OK) return st;
    const adacomp_ssm_shape& s = *shape;
    const adacomp_ssm_inputs& in = *inputs;
    if (s.batch == 0) return ADACOMP_OK;
    if (s.length > 0 && y == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (!aligned_to(h0, 4) || !aligned_to(h_last, 4) || !aligned16(kept) || !aligned16(ws)) return ADACOMP_ERR_MISALIGNED;
    const SsmLayout l = ssm_layout(s, false);
    if (l.bytes > 0 && ws == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (ws_bytes < l.bytes) return ADACOMP_ERR_CAPACITY;
    const uint64_t size = type_size(s.type), C = s.channels, state = 4 * uint64_t(s.batch) * C * s.states;
    const CallView views[6] = {{y, s.channels}, {&in.x, s.channels}, {&in.dt, s.channels}, {&in.b, s.states},
                               {&in.c, s.states}, {in.z.data ? &in.z : nullptr, s.channels}};
    const Range ranges[8] = {range_of(h_last, h_last ? state : 0), range_of(kept, kept ? ssm_kept_bytes(s) : 0),
                             range_of(ws, l.bytes), range_of(h0, h0 ? state : 0), range_of(in.a, 4 * C * s.states),
                             range_of(in.d, in.d ? 4 * C : 0), range_of(in.dt_bias, in.dt_bias ? 4 * C : 0),
                             range_of(in.lengths, in.lengths ? 4 * uint64_t(s.batch) : 0)};
    if ((st = check_buffers(s.length, s.batch, size, views, 1, ranges, 3)) != ADACOMP_OK) return st;
    SsmArgs a{};
    ssm_args(a, s, in, l, ws);
    a.y = dev_view(y);
    a.h0 = h0;
    a.last = h_last;
    a.kept = kept;
    if (s.length == 0) a.kept = nullptr;   // the short kernel carries the states over
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (s.type == ADACOMP_FLOAT) return launch_ssm<float>(a, l.nb, hs);
    if (s.type == ADACOMP_BFLOAT) return launch_ssm<bf16>(a, l.nb, hs);
    return launch_ssm<f16>(a, l.nb, hs);
}

int adacomp_selective_scan_backward(const adacomp_ssm_shape* shape, const adacomp_ssm_inputs* inputs,
                                    const adacomp_view* dy, const float* kept, const float* dh_last,
                                    const adacomp_ssm_gradients* gradients, void* ws, uint64_t ws_bytes,
                                    void* stream) {
    int st = check_ssm_inputs(shape, inputs);
    if (st != ADACOMP_OK) return st;
    const adacomp_ssm_shape& s = *shape;
    const adacomp_ssm_inputs& in = *inputs;
    if (gradients == nullptr || gradients->da == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    const adacomp_ssm_gradients& g = *gradients;
    const uint64_t steps = s.batch ? s.length : 0;
    if (steps > 0 && (dy == nullptr || kept == nullptr || (in.z.data != nullptr) != (g.dz.data != nullptr)))
        return ADACOMP_ERR_INVALID_ARGUMENT;
    if (!aligned16(kept) || !aligned16(ws) || !aligned_to(dh_last, 4) || !aligned_to(g.da, 4) || !aligned_to(g.dd, 4) ||
        !aligned_to(g.ddt_bias, 4) || !aligned_to(g.dh0, 4))
        return ADACOMP_ERR_MISALIGNED;
    SsmLayout l = ssm_layout(s, true);
    if (s.batch == 0) {
        l = SsmLayout{};
        l.padded = (s.states + 7) / 8 * 8;
    }
    if (l.bytes > 0 && ws == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (ws_bytes < l.bytes) return ADACOMP_ERR_CAPACITY;
    const uint64_t size = type_size(s.type), C = s.channels, state = 4 * uint64_t(s.batch) * C * s.states;
    const bool gated = in.z.data != nullptr;
    const CallView views[11] = {{&g.dx, s.channels}, {&g.ddt, s.channels}, {&g.db, s.states}, {&g.dc, s.states},
                                {gated ? &g.dz : nullptr, s.channels}, {dy, s.channels}, {&in.x, s.channels},
                                {&in.dt, s.channels}, {&in.b, s.states}, {&in.c, s.states},
                                {gated ? &in.z : nullptr, s.channels}};
    const Range ranges[11] = {range_of(g.da, 4 * C * s.states), range_of(g.dd, g.dd ? 4 * C : 0),
                              range_of(g.ddt_bias, g.ddt_bias ? 4 * C : 0), range_of(g.dh0, g.dh0 ? state : 0),
                              range_of(ws, l.bytes), range_of(dh_last, dh_last ? state : 0),
                              range_of(kept, steps ? ssm_kept_bytes(s) : 0), range_of(in.a, 4 * C * s.states),
                              range_of(in.d, in.d ? 4 * C : 0), range_of(in.dt_bias, in.dt_bias ? 4 * C : 0),
                              range_of(in.lengths, in.lengths ? 4 * uint64_t(s.batch) : 0)};
    if ((st = check_buffers(steps, s.batch, size, views, 5, ranges, 5)) != ADACOMP_OK) return st;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (s.batch == 0) {   // the sums over nothing
        hipLaunchKernelGGL(k_ssm_channel_grad, dim3((s.channels + 15) / 16, l.padded + 2), dim3(256), 0, hs, nullptr, 0u,
                           l.padded, s.states, s.channels, g.da, g.dd, g.ddt_bias);
        return launch_status();
    }
    SsmArgs a{};
    ssm_args(a, s, in, l, ws);
    if (!gated) a.z = ScanView{};
    a.dy = dev_view(dy);
    a.dx = dev_view(&g.dx);
    a.ddt = dev_view(&g.ddt);
    a.dz = dev_view(&g.dz);
    a.db = dev_view(&g.db);
    a.dc = dev_view(&g.dc);
    a.kept = const_cast<float*>(kept);
    a.h0 = dh_last;
    a.last = g.dh0;
    a.part_rows = reinterpret_cast<float*>(static_cast<char*>(ws) + l.part_rows);
    a.part_a = reinterpret_cast<float*>(static_cast<char*>(ws) + l.part_a);
    if (s.type == ADACOMP_FLOAT) return launch_ssm_back<float>(a, l.nb, g, hs);
    if (s.type == ADACOMP_BFLOAT) return launch_ssm_back<bf16>(a, l.nb, g, hs);
    return launch_ssm_back<f16>(a, l.nb, g, hs);
}

}  // extern "C"
