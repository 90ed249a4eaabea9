// C ABI of the training-step operators (declared in include/adacomp.h):
// optimizer tables, argument checking and stream-ordered kernel launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "../../include/adacomp.h"
#include "adamw.hpp"
#include "gated_scan.hpp"
#include "host_checks.hpp"
#include "layer_norm.hpp"
#include "optimizer_layout.hpp"
#include "views.hpp"

using adacomp::aligned16;
using adacomp::launch_status;
using adacomp::overlaps;
using adacomp::Range;
using adacomp::range_of;
using adacomp::view_range;
using adacomp::views_clash;

struct adacomp_optimizer {
    adacomp_optimizer_info info{};
    uint32_t ntiles = 0;
    int device = -1;
    adacomp::OptTile* tiles = nullptr;
};

namespace {

uint64_t type_size(int type) {
    return type == ADACOMP_FLOAT ? 4 : type == ADACOMP_BFLOAT || type == ADACOMP_HALF ? 2 : 0;
}
bool aligned_to(const void* p, uint64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// No output may share a byte with any other buffer; the first `nout` ranges are outputs.
bool outputs_clash(const Range* r, int nout, int n) {
    for (int i = 0; i < nout; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlaps(r[i], r[j])) return true;
    return false;
}

int check_device(const adacomp_optimizer* o) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return ADACOMP_ERR_HIP;
    return dev == o->device ? ADACOMP_OK : ADACOMP_ERR_INVALID_ARGUMENT;
}

// float32 or 8-bit moments share every check but the moments' element size.
int adamw_impl(const adacomp_optimizer* o, float* weights, const void* grad, int grad_type, void* m, void* v,
               void* scales, bool packed, void* weights_bf16, uint64_t n_elems, const adacomp_adamw* p,
               uint32_t seed, const float* clip, void* stream_) {
    if (o == nullptr || weights == nullptr || grad == nullptr || m == nullptr || v == nullptr || p == nullptr ||
        (packed && scales == nullptr) || type_size(grad_type) == 0 || p->step == 0)
        return ADACOMP_ERR_INVALID_ARGUMENT;
    if (!aligned16(weights) || !aligned16(grad) || !aligned16(m) || !aligned16(v) || !aligned16(scales) ||
        !aligned16(weights_bf16) || !aligned_to(clip, 8))
        return ADACOMP_ERR_MISALIGNED;
    if (n_elems < o->info.span) return ADACOMP_ERR_CAPACITY;
    const uint64_t n = o->info.span, state = packed ? 1 : 4;
    const Range r[7] = {range_of(weights, 4 * n),
                        range_of(m, state * n),
                        range_of(v, state * n),
                        range_of(weights_bf16, weights_bf16 ? 2 * n : 0),
                        range_of(scales, packed ? 2 * o->info.nblocks : 0),
                        range_of(grad, type_size(grad_type) * n),
                        range_of(clip, clip ? 8 : 0)};
    if (outputs_clash(r, 5, 7)) return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = check_device(o);
    if (st != ADACOMP_OK) return st;
    adacomp::AdamwArgs a{};
    a.tiles = o->tiles;
    a.w = weights;
    a.grad = grad;
    a.m = m;
    a.v = v;
    a.scales = static_cast<uint8_t*>(scales);
    a.w16 = static_cast<adacomp::bf16*>(weights_bf16);
    a.clip = clip;
    a.lr = p->lr;
    a.beta1 = p->beta1;
    a.beta2 = p->beta2;
    a.omb1 = 1.0 - a.beta1;
    a.omb2 = 1.0 - a.beta2;
    a.inv_bc1 = 1.0 / (1.0 - std::pow(a.beta1, double(p->step)));
    a.rbc2 = float(1.0 / std::sqrt(1.0 - std::pow(a.beta2, double(p->step))));
    a.eps = p->eps;
    a.scale = p->scale;
    a.key = adacomp::fmix32(seed) ^ p->step;
    hipStream_t stream = static_cast<hipStream_t>(stream_);
    const dim3 grid(o->ntiles), block(adacomp::kOptThreads);
#define ADACOMP_ADAMW(G)                                                              \
    do {                                                                              \
        if (packed) hipLaunchKernelGGL(adacomp::k_adamw_packed<G>, grid, block, 0, stream, a); \
        else hipLaunchKernelGGL(adacomp::k_adamw<G>, grid, block, 0, stream, a);      \
    } while (0)
    if (grad_type == ADACOMP_FLOAT) ADACOMP_ADAMW(float);
    else if (grad_type == ADACOMP_BFLOAT) ADACOMP_ADAMW(adacomp::bf16);
    else ADACOMP_ADAMW(adacomp::f16);
#undef ADACOMP_ADAMW
    return launch_status();
}

}  // namespace

extern "C" {

int adacomp_optimizer_query(const adacomp_tensor* tensors, uint32_t ntensors, adacomp_optimizer_info* info) {
    if (info == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    try {
        adacomp::OptLayout L;
        const int st = adacomp::build_optimizer(tensors, ntensors, false, L);
        if (st == ADACOMP_OK) *info = L.info;
        return st;
    } catch (...) {
        return ADACOMP_ERR_INVALID_ARGUMENT;
    }
}

int adacomp_optimizer_create(const adacomp_tensor* tensors, uint32_t ntensors, adacomp_optimizer** out) {
    if (out == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    *out = nullptr;
    adacomp_optimizer* o = nullptr;
    try {
        adacomp::OptLayout L;
        int st = adacomp::build_optimizer(tensors, ntensors, true, L);
        if (st != ADACOMP_OK) return st;
        o = new adacomp_optimizer();
        o->info = L.info;
        o->ntiles = static_cast<uint32_t>(L.tiles.size());
        const uint64_t bytes = sizeof(adacomp::OptTile) * L.tiles.size();
        void* mem = nullptr;
        if (hipGetDevice(&o->device) != hipSuccess || hipMalloc(&mem, bytes) != hipSuccess) {
            delete o;
            return ADACOMP_ERR_HIP;
        }
        o->tiles = static_cast<adacomp::OptTile*>(mem);
        if (hipMemcpy(mem, L.tiles.data(), bytes, hipMemcpyHostToDevice) != hipSuccess) {
            (void)hipFree(mem);
            delete o;
            return ADACOMP_ERR_HIP;
        }
        *out = o;
        return ADACOMP_OK;
    } catch (...) {
        if (o && o->tiles) (void)hipFree(o->tiles);
        delete o;
        return ADACOMP_ERR_INVALID_ARGUMENT;
    }
}

int adacomp_optimizer_destroy(adacomp_optimizer* o) {
    if (o == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = hipFree(o->tiles) == hipSuccess ? ADACOMP_OK : ADACOMP_ERR_HIP;
    delete o;
    return st;
}

int adacomp_optimizer_get_info(const adacomp_optimizer* o, adacomp_optimizer_info* info) {
    if (o == nullptr || info == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    *info = o->info;
    return ADACOMP_OK;
}

int adacomp_grad_norm(const adacomp_optimizer* o, const void* grad, int grad_type, uint64_t n_elems, float max_norm,
                      float scale, float* clip, void* ws, uint64_t ws_bytes, void* stream_) {
    if (o == nullptr || grad == nullptr || clip == nullptr || ws == nullptr || type_size(grad_type) == 0 ||
        !(max_norm >= 0.f))
        return ADACOMP_ERR_INVALID_ARGUMENT;
    if (!aligned16(grad) || !aligned16(ws) || !aligned_to(clip, 8)) return ADACOMP_ERR_MISALIGNED;
    if (n_elems < o->info.span || ws_bytes < o->info.norm_workspace_bytes) return ADACOMP_ERR_CAPACITY;
    const Range r[3] = {range_of(clip, 8), range_of(ws, o->info.norm_workspace_bytes),
                        range_of(grad, type_size(grad_type) * o->info.span)};
    if (outputs_clash(r, 2, 3)) return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = check_device(o);
    if (st != ADACOMP_OK) return st;
    hipStream_t stream = static_cast<hipStream_t>(stream_);
    double* partial = static_cast<double*>(ws);
    const uint32_t blocks = std::min(o->ntiles, adacomp::kNormMaxBlocks);
#define ADACOMP_NORM(G) \
    hipLaunchKernelGGL(adacomp::k_grad_norm<G>, dim3(blocks), dim3(256), 0, stream, o->tiles, o->ntiles, grad, partial)
    if (grad_type == ADACOMP_FLOAT) ADACOMP_NORM(float);
    else if (grad_type == ADACOMP_BFLOAT) ADACOMP_NORM(adacomp::bf16);
    else ADACOMP_NORM(adacomp::f16);
#undef ADACOMP_NORM
    if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
    hipLaunchKernelGGL(adacomp::k_grad_norm_finish, dim3(1), dim3(256), 0, stream, partial, blocks, double(max_norm),
                       double(scale), clip);
    return launch_status();
}

int adacomp_adamw_step(const adacomp_optimizer* o, float* weights, const void* grad, int grad_type, float* m, float* v,
                       void* weights_bf16, uint64_t n_elems, const adacomp_adamw* adamw, const float* clip,
                       void* stream) {
    return adamw_impl(o, weights, grad, grad_type, m, v, nullptr, false, weights_bf16, n_elems, adamw, 0, clip, stream);
}

int adacomp_adamw_packed_step(const adacomp_optimizer* o, float* weights, const void* grad, int grad_type,
                              void* m_codes, void* v_codes, void* scales, void* weights_bf16, uint64_t n_elems,
                              const adacomp_adamw* adamw, uint32_t seed, const float* clip, void* stream) {
    return adamw_impl(o, weights, grad, grad_type, m_codes, v_codes, scales, true, weights_bf16, n_elems, adamw, seed,
                      clip, stream);
}

}  // extern "C"

// ---- layer norm ----

namespace {

uint64_t rows_bytes(uint64_t rows, uint64_t stride, uint32_t cols, uint64_t size) {
    return rows ? ((rows - 1) * stride + cols) * size : 0;
}

// Checks of one matrix argument.
int check_rows(const void* p, uint64_t stride, uint64_t rows, uint32_t cols, int type) {
    if (p == nullptr || stride < cols) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (!aligned_to(p, type_size(type))) return ADACOMP_ERR_MISALIGNED;
    if (rows > 1 && stride > (uint64_t(1) << 40) / rows) return ADACOMP_ERR_TOO_LARGE;
    return ADACOMP_OK;
}

// Rows that a workgroup each takes are as many as work-items of one launch fit in 32 bits; the kernels of
// shorter rows step over them with a bounded grid.
int check_norm_shape(uint64_t rows, uint32_t cols, int type, bool back) {
    if (type_size(type) == 0 || cols == 0) return ADACOMP_ERR_INVALID_ARGUMENT;
    const bool wide = cols > (back ? adacomp::kNormBackRegCols : adacomp::kNormRegCols);
    const uint64_t items = (uint64_t(1) << 32) - 1;
    if (cols > ADACOMP_NORM_MAX_COLS || rows > (wide ? items / adacomp::kNormWideThreads : items))
        return ADACOMP_ERR_TOO_LARGE;
    return ADACOMP_OK;
}

// Partial rows of the weight gradients: one per workgroup.
uint32_t norm_partials(uint64_t rows) {
    return static_cast<uint32_t>(std::min<uint64_t>(std::max<uint64_t>(rows, 1), adacomp::kNormMaxPartials));
}

// Lanes of one wavefront's team: the fewest whose vectors cover the row.
int team_lanes(uint32_t cols, uint32_t vec) {
    int lanes = 4;
    while (lanes < 64 && lanes * vec < cols) lanes *= 2;
    return lanes;
}

// Workgroups for `need` shares of rows: at most `most`, each with as many shares as the others
// but for one.
uint32_t norm_blocks(uint64_t need, uint32_t most) {
    const uint64_t turns = (need + most - 1) / most;
    return static_cast<uint32_t>((need + turns - 1) / turns);
}

// The kernel of one row length: rows shorter than a vector by single elements, up to one
// wavefront's columns by teams of its lanes, longer ones by whole workgroups.
#define ADACOMP_NORM_TEAMS(LAUNCH)                                   \
    do {                                                             \
        if (a.cols < VEC) LAUNCH(1, 1, 8);                           \
        else if (a.cols > 64 * VEC * 2) LAUNCH(VEC, NVMAX, 64);      \
        else if (a.cols > 64 * VEC) LAUNCH(VEC, 2, 64);              \
        else switch (team_lanes(a.cols, VEC)) {                      \
            case 4: LAUNCH(VEC, 1, 4); break;                        \
            case 8: LAUNCH(VEC, 1, 8); break;                        \
            case 16: LAUNCH(VEC, 1, 16); break;                      \
            case 32: LAUNCH(VEC, 1, 32); break;                      \
            default: LAUNCH(VEC, 1, 64); break;                      \
        }                                                            \
    } while (0)

template <typename T, int KEEP>
void launch_norm(const adacomp::NormArgs& a, hipStream_t s) {
    using namespace adacomp;
    constexpr int VEC = norm_vec<T>(), NVMAX = kNormElems / VEC;
    const uint64_t rows = a.rows;
    if (a.cols > kNormRegCols) {
        hipLaunchKernelGGL(k_layer_norm_wide<T>, dim3(uint32_t(rows)), dim3(kNormWideThreads), 0, s, a);
    } else if (a.cols > kNormWaveCols) {
        const uint32_t waves = (a.cols + kNormWaveCols - 1) / kNormWaveCols;
        hipLaunchKernelGGL((k_layer_norm<T, VEC, NVMAX, 64, true, KEEP>), dim3(norm_blocks(rows, kNormMaxWaves / waves)),
                           dim3(64 * waves), 0, s, a);
    } else {
#define ADACOMP_LN(V, NV, LANES)                                                              \
    hipLaunchKernelGGL((k_layer_norm<T, V, NV, LANES, false, KEEP>),                                \
                       dim3(norm_blocks((rows + 256 / LANES - 1) / (256 / LANES), kNormMaxWaves / 4)), dim3(256), 0, \
                       s, a)
        ADACOMP_NORM_TEAMS(ADACOMP_LN);
#undef ADACOMP_LN
    }
}

// Returns the number of partial rows written.
template <typename T, int KEEP>
uint32_t launch_norm_backward(const adacomp::NormArgs& a, hipStream_t s) {
    using namespace adacomp;
    constexpr int VEC = norm_vec<T>(), NVMAX = kNormElems / VEC;
    const uint64_t rows = a.rows;
    const uint32_t most = norm_partials(rows);
    if (a.cols > kNormBackRegCols) {
        hipLaunchKernelGGL(k_layer_norm_backward_wide<T>, dim3(uint32_t(rows)), dim3(kNormWideThreads), 0, s, a);
        if (a.partial == nullptr || hipPeekAtLastError() != hipSuccess) return 0;   // the caller reports it
        const uint32_t n = std::min(most, 64u);
        hipLaunchKernelGGL(k_norm_partial_wide<T>, dim3((a.cols + 255) / 256, n), dim3(256), 0, s, a);
        return n;
    }
    // Teams a workgroup: half of the most that fit where the rows need no more workgroups than may be
    // (100 x 777 bf16 8.3 us against 9.6 with all, 32768 x 1024 41.9 against 42.9).
    auto teams_of = [&](uint32_t limit) { return limit > 1 && rows <= uint64_t(limit / 2) * most ? limit / 2 : limit; };
    if (a.cols > kNormWaveCols) {
        const uint32_t waves = (a.cols + kNormWaveCols - 1) / kNormWaveCols;
        const uint32_t teams = teams_of(kNormBackThreads / 64 / waves);
        const uint32_t n = norm_blocks((rows + teams - 1) / teams, most);
        hipLaunchKernelGGL((k_layer_norm_backward<T, VEC, NVMAX, 64, true, KEEP>), dim3(n), dim3(64 * waves * teams),
                           2 * 4 * kNormWaveCols * waves * teams, s, a);
        return n;
    }
    uint32_t n = 0;
#define ADACOMP_LNB(V, NV, LANES)                                                               \
    do {                                                                                        \
        const uint32_t teams = teams_of(kNormBackThreads / LANES);                              \
        n = norm_blocks((rows + teams - 1) / teams, most);                                      \
        hipLaunchKernelGGL((k_layer_norm_backward<T, V, NV, LANES, false, KEEP>), dim3(n),            \
                           dim3(teams * LANES), 2 * 4 * teams * LANES * NV * V, s, a);          \
    } while (0)
    ADACOMP_NORM_TEAMS(ADACOMP_LNB);
#undef ADACOMP_LNB
    return n;
}
#undef ADACOMP_NORM_TEAMS

int norm_keep(uint64_t read, uint64_t written) {
    return read <= adacomp::kKeepBytes ? adacomp::kNormKeepIn
                                           : written <= adacomp::kKeepBytes ? adacomp::kNormKeepOut
                                                                                : adacomp::kNormKeepNone;
}
template <typename T>
void launch_norm(const adacomp::NormArgs& a, hipStream_t s) {
    const uint64_t bytes = a.rows * a.cols * sizeof(T);
    switch (norm_keep(bytes, bytes)) {
        case adacomp::kNormKeepIn: return launch_norm<T, adacomp::kNormKeepIn>(a, s);
        default: return launch_norm<T, adacomp::kNormKeepNone>(a, s);   // the output is as large as the input
    }
}
template <typename T>
uint32_t launch_norm_backward(const adacomp::NormArgs& a, hipStream_t s) {
    const uint64_t bytes = a.rows * a.cols * sizeof(T);
    switch (norm_keep(2 * bytes, bytes)) {
        case adacomp::kNormKeepIn: return launch_norm_backward<T, adacomp::kNormKeepIn>(a, s);
        case adacomp::kNormKeepOut: return launch_norm_backward<T, adacomp::kNormKeepOut>(a, s);
        default: return launch_norm_backward<T, adacomp::kNormKeepNone>(a, s);
    }
}

}  // namespace

extern "C" {

int adacomp_layer_norm(const void* x, uint64_t x_stride, const float* weight, const float* bias, void* y,
                       uint64_t y_stride, float* mean, float* rstd, uint64_t rows, uint32_t cols, int type, float eps,
                       void* stream_) {
    int st = check_norm_shape(rows, cols, type, false);
    if (st != ADACOMP_OK) return st;
    if (!(eps >= 0.f) || std::isinf(eps)) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (rows == 0) return ADACOMP_OK;
    if ((st = check_rows(x, x_stride, rows, cols, type)) != ADACOMP_OK) return st;
    if ((st = check_rows(y, y_stride, rows, cols, type)) != ADACOMP_OK) return st;
    if (!aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return ADACOMP_ERR_MISALIGNED;
    const uint64_t size = type_size(type);
    const Range r[6] = {range_of(y, rows_bytes(rows, y_stride, cols, size)),
                        range_of(mean, mean ? 4 * rows : 0),
                        range_of(rstd, rstd ? 4 * rows : 0),
                        range_of(x, rows_bytes(rows, x_stride, cols, size)),
                        range_of(weight, weight ? 4 * uint64_t(cols) : 0),
                        range_of(bias, bias ? 4 * uint64_t(cols) : 0)};
    if (outputs_clash(r, 3, 6)) return ADACOMP_ERR_INVALID_ARGUMENT;
    adacomp::NormArgs a{};
    a.x = x;
    a.out = y;
    a.weight = weight;
    a.bias = bias;
    a.mean = mean;
    a.rstd = rstd;
    a.x_stride = x_stride;
    a.out_stride = y_stride;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.inv_cols = 1.0f / float(cols);
    hipStream_t s = static_cast<hipStream_t>(stream_);
    if (type == ADACOMP_FLOAT) launch_norm<float>(a, s);
    else if (type == ADACOMP_BFLOAT) launch_norm<adacomp::bf16>(a, s);
    else launch_norm<adacomp::f16>(a, s);
    return launch_status();
}

int adacomp_layer_norm_workspace_bytes(uint64_t rows, uint32_t cols, uint64_t* bytes) {
    if (bytes == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = check_norm_shape(rows, cols, ADACOMP_FLOAT, true);
    if (st != ADACOMP_OK) return st;
    *bytes = uint64_t(norm_partials(rows)) * 2 * cols * 4;
    return ADACOMP_OK;
}

int adacomp_layer_norm_backward(const void* dy, uint64_t dy_stride, const void* x, uint64_t x_stride,
                                const float* weight, const float* mean, const float* rstd, void* dx,
                                uint64_t dx_stride, float* dweight, float* dbias, uint64_t rows, uint32_t cols,
                                int type, void* ws, uint64_t ws_bytes, void* stream_) {
    int st = check_norm_shape(rows, cols, type, true);
    if (st != ADACOMP_OK) return st;
    const bool sums = dweight != nullptr;
    if ((dbias != nullptr) != sums) return ADACOMP_ERR_INVALID_ARGUMENT;
    const uint64_t size = type_size(type), need = uint64_t(norm_partials(rows)) * 2 * cols * 4;
    if (rows > 0) {
        if ((st = check_rows(dy, dy_stride, rows, cols, type)) != ADACOMP_OK) return st;
        if ((st = check_rows(x, x_stride, rows, cols, type)) != ADACOMP_OK) return st;
        if ((st = check_rows(dx, dx_stride, rows, cols, type)) != ADACOMP_OK) return st;
        if (mean == nullptr || rstd == nullptr || (sums && ws == nullptr)) return ADACOMP_ERR_INVALID_ARGUMENT;
    } else if (!sums) {
        return ADACOMP_OK;
    }
    if (!aligned_to(weight, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dweight, 4) ||
        !aligned_to(dbias, 4) || (sums && !aligned16(ws)))
        return ADACOMP_ERR_MISALIGNED;
    if (rows > 0 && sums && ws_bytes < need) return ADACOMP_ERR_CAPACITY;
    const Range r[9] = {range_of(dx, rows_bytes(rows, dx_stride, cols, size)),
                        range_of(dweight, sums ? 4 * uint64_t(cols) : 0),
                        range_of(dbias, sums ? 4 * uint64_t(cols) : 0),
                        range_of(ws, sums && rows ? need : 0),
                        range_of(dy, rows_bytes(rows, dy_stride, cols, size)),
                        range_of(x, rows_bytes(rows, x_stride, cols, size)),
                        range_of(weight, weight ? 4 * uint64_t(cols) : 0),
                        range_of(mean, 4 * rows),
                        range_of(rstd, 4 * rows)};
    if (outputs_clash(r, 4, 9)) return ADACOMP_ERR_INVALID_ARGUMENT;
    adacomp::NormArgs a{};
    a.x = x;
    a.dy = dy;
    a.out = dx;
    a.weight = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.partial = sums ? static_cast<float*>(ws) : nullptr;
    a.x_stride = x_stride;
    a.dy_stride = dy_stride;
    a.out_stride = dx_stride;
    a.rows = rows;
    a.cols = cols;
    a.inv_cols = 1.0f / float(cols);
    hipStream_t s = static_cast<hipStream_t>(stream_);
    uint32_t n = 0;
    if (rows > 0) {
        if (type == ADACOMP_FLOAT) n = launch_norm_backward<float>(a, s);
        else if (type == ADACOMP_BFLOAT) n = launch_norm_backward<adacomp::bf16>(a, s);
        else n = launch_norm_backward<adacomp::f16>(a, s);
        if ((st = launch_status()) != ADACOMP_OK) return st;
    }
    if (sums) {
        hipLaunchKernelGGL(adacomp::k_norm_weight_grad, dim3((cols + 15) / 16, 2), dim3(1024), 0, s, a.partial, n,
                           cols, dweight, dbias);
        st = launch_status();
    }
    return st;
}

}  // extern "C"

// ---- gated scan ----

namespace {

struct ScanLayout {
    uint32_t lanes, groups, threads, steps, tiles, span, spans, most;
    bool chain;
    uint64_t ws;
};

int check_shape(const adacomp_scan_shape* s) {
    if (s == nullptr || type_size(s->type) == 0 || s->channels == 0 || (s->sigmoid != 0 && s->sigmoid != 1))
        return ADACOMP_ERR_INVALID_ARGUMENT;
    if (s->length >= (uint64_t(1) << 31) || s->channels >= (1u << 24) || s->batch >= (1u << 24) ||
        uint64_t(s->batch) * s->channels >= (uint64_t(1) << 31))
        return ADACOMP_ERR_TOO_LARGE;
    return ADACOMP_OK;
}

// Tiles of one shape for vectors of vw channels.
ScanLayout scan_layout(const adacomp_scan_shape& s, uint32_t vw, bool back) {
    const uint32_t per = adacomp::scan_thread_steps(s.sigmoid != 0, back);
    using namespace adacomp;
    ScanLayout l{};
    if (s.length <= kScanShort) {   // one thread per vector
        l.lanes = (s.channels + vw - 1) / vw;
        return l;
    }
    l.lanes = 4;
    while (l.lanes < 64 && l.lanes * vw < s.channels) l.lanes *= 2;
    l.groups = (s.channels + l.lanes * vw - 1) / (l.lanes * vw);
    uint32_t subs = std::max(64 / l.lanes, 2u);
    while (subs * l.lanes < kScanThreads && uint64_t(subs) * per < s.length) subs *= 2;
    l.threads = subs * l.lanes;
    l.steps = subs * per;
    l.tiles = static_cast<uint32_t>((s.length + l.steps - 1) / l.steps);
    const uint64_t chains = uint64_t(s.batch) * l.groups;
    // At 64 chains and more the hop from tile to tile hides behind the other chains' tiles, and looking
    // further back only adds to the traffic.
    l.chain = chains >= 64;
    const uint32_t looks = l.threads / (l.lanes * vw);   // threads a slot; 4 and more where there are several tiles
    l.span = std::max(looks * kScanWindow / 2, 1u);
    l.most = looks * kScanWindow;
    l.spans = (l.tiles + l.span - 1) / l.span;
    // a word of every slot of a tile, and of a group of tiles
    if (l.tiles > 1) l.ws = kScanCountBytes + chains * (l.tiles + l.spans) * l.lanes * vw * 8;
    return l;
}
// Channels of one thread: 4 bytes.
uint32_t scan_vector(const adacomp_scan_shape& s) { return s.type == ADACOMP_FLOAT || s.channels < 2 ? 1 : 2; }
// What either direction and any type of this shape needs.
uint64_t scan_workspace(adacomp_scan_shape s) {
    uint64_t most = 0;
    for (s.sigmoid = 0; s.sigmoid < 2; ++s.sigmoid)
        for (const bool back : {false, true})
            for (uint32_t vw = 1; vw <= std::min(s.channels, 2u); ++vw)
                most = std::max(most, scan_layout(s, vw, back).ws);
    return most;
}

int check_view(const adacomp_view* v, const adacomp_scan_shape& s) {
    if (v == nullptr || v->data == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (v->time_stride < s.channels) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (!aligned_to(v->data, type_size(s.type))) return ADACOMP_ERR_MISALIGNED;
    if (v->time_stride >= (uint64_t(1) << 32) || v->batch_stride >= (uint64_t(1) << 40)) return ADACOMP_ERR_TOO_LARGE;
    return ADACOMP_OK;
}

adacomp::ScanView dev_view(const adacomp_view* v) {
    return v ? adacomp::ScanView{v->data, v->batch_stride, v->time_stride} : adacomp::ScanView{};
}

struct ScanCall {
    const adacomp_scan_shape* shape;
    const adacomp_view* in[4];
    int nin;
    const adacomp_view* out[2];
    int nout;
    const float* states_in[2];   // nullable [batch, channels]
    float* state_out;            // nullable
    const int32_t* lengths;
    void* ws;
    uint64_t ws_bytes;
};

int check_scan(const ScanCall& c) {
    const adacomp_scan_shape& s = *c.shape;
    int st;
    const bool steps = s.length > 0;   // without steps no view is touched
    for (int i = 0; i < c.nin && steps; ++i)
        if ((st = check_view(c.in[i], s)) != ADACOMP_OK) return st;
    for (int i = 0; i < c.nout && steps; ++i) {
        if ((st = check_view(c.out[i], s)) != ADACOMP_OK) return st;
        adacomp::RowGrid rows;   // an output's rows may not meet
        if (!adacomp::row_grid(*c.out[i], s, rows)) return ADACOMP_ERR_INVALID_ARGUMENT;
    }
    if (!aligned_to(c.states_in[0], 4) || !aligned_to(c.states_in[1], 4) || !aligned_to(c.state_out, 4) ||
        !aligned_to(c.lengths, 4) || !aligned16(c.ws))
        return ADACOMP_ERR_MISALIGNED;
    const uint64_t need = scan_workspace(s);
    if (need > 0 && c.ws == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    if (c.ws_bytes < need) return ADACOMP_ERR_CAPACITY;
    const uint64_t state = 4 * uint64_t(s.batch) * s.channels, size = type_size(s.type);
    Range r[11] = {range_of(c.state_out, c.state_out ? state : 0), range_of(c.ws, need)};
    int n = 2;
    for (int i = 0; i < c.nout && steps; ++i) r[n++] = view_range(*c.out[i], s, size);
    const int nout = n, nview = steps ? n + c.nin : n;
    for (int i = 0; i < c.nin && steps; ++i) r[n++] = view_range(*c.in[i], s, size);
    for (int i = 0; i < 2; ++i) r[n++] = range_of(c.states_in[i], c.states_in[i] ? state : 0);
    r[n++] = range_of(c.lengths, c.lengths ? 4 * uint64_t(s.batch) : 0);
    for (int i = 0; i < nout; ++i)
        for (int j = i + 1; j < n; ++j) {
            if (!overlaps(r[i], r[j])) continue;
            if (i >= 2 && j < nview) {   // two views
                const adacomp_view* b = j < nout ? c.out[j - 2] : c.in[j - nout];
                if (!views_clash(*c.out[i - 2], *b, s, size)) continue;
            }
            return ADACOMP_ERR_INVALID_ARGUMENT;
        }
    return ADACOMP_OK;
}

// How a call's views are accessed.  Where a step of one does not start on a cache line, the lines at a
// tile's edges serve the neighbouring channels' tiles as well, which run on the same chiplet, and have
// to stay in its cache.
int scan_access(const adacomp::ScanArgs& a, uint64_t size, uint64_t inputs) {
    for (const adacomp::ScanView* v : {&a.gate, &a.x, &a.h, &a.dh, &a.dgate, &a.dx})
        if (v->p && (!aligned_to(v->p, 128) || v->ts * size % 128 != 0 || v->bs * size % 128 != 0))
            return adacomp::kScanCached;
    return inputs * size * a.batch * a.length * a.channels <= adacomp::kKeepBytes ? adacomp::kScanKeepIn
                                                                                  : adacomp::kScanStream;
}

template <typename T, int VW, bool SIG, bool BACK, int ACCESS>
int launch_scan(adacomp::ScanArgs& a, const ScanLayout& l, void* ws, hipStream_t s) {
    using namespace adacomp;
    const uint64_t chains = uint64_t(a.batch) * l.groups, n = chains * l.tiles;
    a.queues = static_cast<uint32_t>(std::min<uint64_t>(chains, kScanQueues));
    const uint64_t blocks = l.tiles == 1 ? n : (chains + a.queues - 1) / a.queues * a.queues * l.tiles;
    if (blocks * l.threads >= (uint64_t(1) << 32)) return ADACOMP_ERR_TOO_LARGE;   // work-items of one launch
    const dim3 block(l.threads);
    if (l.tiles == 1) {
        hipLaunchKernelGGL((k_scan_tile<T, VW, SIG, BACK, kScanAlone, ACCESS>), dim3(uint32_t(blocks)), block, 0, s, a);
        return launch_status();
    }
    const uint64_t slots = l.lanes * VW, words = l.chain ? n * slots * 4 : (n + chains * l.spans) * slots * 8;
    const uint64_t vecs = (kScanCountBytes + words + 15) / 16;
    a.tickets = static_cast<uint32_t*>(ws);
    a.words = a.tickets + kScanCountBytes / 4;
    a.group_words = static_cast<uint64_t*>(a.words) + n * slots;
    hipLaunchKernelGGL(k_scan_clear, dim3(uint32_t((vecs + 255) / 256)), dim3(256), 0, s, static_cast<uint4*>(ws),
                       vecs);
    if (launch_status() != ADACOMP_OK) return ADACOMP_ERR_HIP;
    const dim3 grid(static_cast<uint32_t>(blocks));
    if (l.chain) hipLaunchKernelGGL((k_scan_tile<T, VW, SIG, BACK, kScanChain, ACCESS>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_scan_tile<T, VW, SIG, BACK, kScanBack, ACCESS>), grid, block, 0, s, a);
    return launch_status();
}

template <typename T, int VW, bool SIG, bool BACK>
int launch_scan(adacomp::ScanArgs& a, const ScanLayout& l, void* ws, hipStream_t s) {
    using namespace adacomp;
    if (l.tiles == 0) {
        const uint64_t blocks = (uint64_t(a.batch) * l.lanes + 255) / 256;
        hipLaunchKernelGGL((k_scan_short<T, VW, SIG, BACK>), dim3(uint32_t(blocks)), dim3(256), 0, s, a);
        return launch_status();
    }
    switch (scan_access(a, sizeof(T), BACK ? (SIG ? 4 : 3) : 2)) {
        case kScanStream: return launch_scan<T, VW, SIG, BACK, kScanStream>(a, l, ws, s);
        case kScanKeepIn: return launch_scan<T, VW, SIG, BACK, kScanKeepIn>(a, l, ws, s);
        default: return launch_scan<T, VW, SIG, BACK, kScanCached>(a, l, ws, s);
    }
}

template <typename T, int VW>
int launch_scan_as(adacomp::ScanArgs& a, bool sigmoid, bool back, const ScanLayout& l, void* ws, hipStream_t s) {
    if (sigmoid)
        return back ? launch_scan<T, VW, true, true>(a, l, ws, s) : launch_scan<T, VW, true, false>(a, l, ws, s);
    return back ? launch_scan<T, VW, false, true>(a, l, ws, s) : launch_scan<T, VW, false, false>(a, l, ws, s);
}

int run_scan(const ScanCall& c, adacomp::ScanArgs& a, bool back, void* stream) {
    const adacomp_scan_shape& s = *c.shape;
    const uint32_t vw = scan_vector(s);
    const ScanLayout l = scan_layout(s, vw, back);
    a.lengths = c.lengths;
    a.last = c.state_out;
    a.length = s.length;
    a.batch = s.batch;
    a.channels = s.channels;
    a.lanes = l.lanes;
    a.groups = l.groups;
    a.tiles = l.tiles;
    a.steps = l.steps;
    a.span = l.span;
    a.spans = l.spans;
    a.most = l.most;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    const bool sig = s.sigmoid != 0;
    if (s.type == ADACOMP_FLOAT) return launch_scan_as<float, 1>(a, sig, back, l, c.ws, hs);
    if (s.type == ADACOMP_BFLOAT)
        return vw == 1 ? launch_scan_as<adacomp::bf16, 1>(a, sig, back, l, c.ws, hs)
                       : launch_scan_as<adacomp::bf16, 2>(a, sig, back, l, c.ws, hs);
    return vw == 1 ? launch_scan_as<adacomp::f16, 1>(a, sig, back, l, c.ws, hs)
                   : launch_scan_as<adacomp::f16, 2>(a, sig, back, l, c.ws, hs);
}

}  // namespace

extern "C" {

int adacomp_gated_scan_workspace_bytes(const adacomp_scan_shape* shape, uint64_t* bytes) {
    if (bytes == nullptr) return ADACOMP_ERR_INVALID_ARGUMENT;
    const int st = check_shape(shape);
    if (st == ADACOMP_OK) *bytes = scan_workspace(*shape);
    return st;
}

int adacomp_gated_scan(const adacomp_scan_shape* shape, const adacomp_view* gate, const adacomp_view* x,
                       const adacomp_view* h, const float* h0, float* h_last, const int32_t* lengths, void* ws,
                       uint64_t ws_bytes, void* stream) {
    int st = check_shape(shape);
    if (st != ADACOMP_OK) return st;
    if (shape->batch == 0) return ADACOMP_OK;
    const ScanCall c{shape, {gate, x, nullptr, nullptr}, 2, {h, nullptr}, 1, {h0, nullptr}, h_last, lengths,
                     ws,    ws_bytes};
    if ((st = check_scan(c)) != ADACOMP_OK) return st;
    adacomp::ScanArgs a{};
    a.gate = dev_view(gate);
    a.x = dev_view(x);
    a.h = dev_view(h);
    a.h0 = h0;
    return run_scan(c, a, false, stream);
}

int adacomp_gated_scan_backward(const adacomp_scan_shape* shape, const adacomp_view* gate, const adacomp_view* x,
                                const adacomp_view* h, const adacomp_view* dh, const adacomp_view* dgate,
                                const adacomp_view* dx, const float* h0, const float* dh_last, float* dh0,
                                const int32_t* lengths, void* ws, uint64_t ws_bytes, void* stream) {
    int st = check_shape(shape);
    if (st != ADACOMP_OK) return st;
    if (shape->batch == 0) return ADACOMP_OK;
    const bool sig = shape->sigmoid != 0;
    const ScanCall c{shape, {gate, h, dh, sig ? x : nullptr}, sig ? 4 : 3, {dgate, dx}, 2, {h0, dh_last}, dh0,
                     lengths, ws, ws_bytes};
    if ((st = check_scan(c)) != ADACOMP_OK) return st;
    adacomp::ScanArgs a{};
    a.gate = dev_view(gate);
    if (sig) a.x = dev_view(x);
    a.h = dev_view(h);
    a.dh = dev_view(dh);
    a.dgate = dev_view(dgate);
    a.dx = dev_view(dx);
    a.h0 = h0;
    a.dh_last = dh_last;
    return run_scan(c, a, true, stream);
}

}  // extern "C"
