// api_routing.cu — the C ABI of routing: choosing experts, sorting rows by
// them, and moving rows to the experts and back.  As in api.cu, every argument
// is validated before any CUDA call.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>

#include "swiglu_mlp.h"
#include "host.h"
#include "routing.h"

namespace {

// The kernels number tokens, slots, rows and columns in 32 bits, and CTAs too.
constexpr int64_t kMaxDim = 0x80000000ll - 1024;
constexpr int64_t kMaxStride = 0x7fffffff;

bool aligned(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }

bool type_bytes(int type, int &bytes)
{
    switch (type) {
    case SWG_TYPE_F16: case SWG_TYPE_BF16: bytes = 2; return true;
    case SWG_TYPE_F32: bytes = 4; return true;
    default: return false;
    }
}

bool aligned4(std::initializer_list<const void *> all)
{
    for (const void *p : all)
        if (!aligned(p, 4)) return false;
    return true;
}

// Rules on tokens and slots shared by every entry point.
int check_slots(int64_t T, int64_t top)
{
    if (T < 0 || top < 1) return SWG_ERR_INVALID_ARG;
    if (top > SWG_MAX_TOP || T > kMaxDim || T * top > kMaxDim) return SWG_ERR_UNSUPPORTED;
    return SWG_OK;
}

int check_experts(int64_t E, int64_t top)
{
    if (E < 1 || top > E) return SWG_ERR_INVALID_ARG;
    return E > SWG_MAX_EXPERTS ? SWG_ERR_UNSUPPORTED : SWG_OK;
}

// Logits, or their gradient: rows of E elements, of any alignment of the type.
int check_logits(const void *x, int64_t ld, int64_t E, int bytes)
{
    if (x == nullptr || ld < E) return SWG_ERR_INVALID_ARG;
    if (ld > kMaxStride) return SWG_ERR_UNSUPPORTED;
    return aligned(x, bytes) ? SWG_OK : SWG_ERR_MISALIGNED;
}

// Rows of D elements in 16-byte pieces.
int check_rows(const void *x, int64_t ld, int64_t D, int bytes)
{
    if (x == nullptr || ld < D) return SWG_ERR_INVALID_ARG;
    if (ld > kMaxStride) return SWG_ERR_UNSUPPORTED;
    return aligned(x, 16) && ld * bytes % 16 == 0 ? SWG_OK : SWG_ERR_MISALIGNED;
}

// The device, and a workspace for more than one chunk's counts.
int plan_workspace(int chunks, int64_t E, cudaStream_t s, int32_t *&counts, std::unique_lock<std::mutex> &held)
{
    counts = nullptr;
    if (chunks <= 1) return SWG_OK;
    float *ws = nullptr;
    if (int rc = swg::stream_workspace(s, sizeof(int32_t) * (size_t)chunks * (size_t)E, ws, held)) return rc;
    counts = reinterpret_cast<int32_t *>(ws);
    return SWG_OK;
}

}  // namespace

extern "C" {

int expert_route(int score, int64_t T, int64_t E, int64_t top, const void *logits, int64_t ldl, int type,
                 const float *bias, int64_t groups, int64_t top_groups, int group_sum, int normalise,
                 float scale, int32_t *experts, float *weights, int32_t *offsets, int32_t *source,
                 int32_t *position, void *stream)
{
    int bytes;
    if (!type_bytes(type, bytes)) return SWG_ERR_UNSUPPORTED;
    if (score != SWG_SOFTMAX && score != SWG_SIGMOID) return SWG_ERR_UNSUPPORTED;
    if (int rc = check_slots(T, top)) return rc;
    if (int rc = check_experts(E, top)) return rc;
    if (groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups || top > E / groups * top_groups)
        return SWG_ERR_INVALID_ARG;
    if (group_sum != 1 && group_sum != 2) return SWG_ERR_INVALID_ARG;
    if (groups > SWG_MAX_EXPERT_GROUPS) return SWG_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return SWG_ERR_INVALID_ARG;
    const bool planned = offsets != nullptr;
    // (of no tokens there are no slots: tensors of none have no address)
    if (T > 0 && (planned != (source != nullptr) || planned != (position != nullptr)))
        return SWG_ERR_INVALID_ARG;
    if (!aligned4({bias, experts, weights, offsets, source, position})) return SWG_ERR_MISALIGNED;
    if (T > 0) {
        if (experts == nullptr || weights == nullptr) return SWG_ERR_INVALID_ARG;
        if (int rc = check_logits(logits, ldl, E, bytes)) return rc;
    } else if (!planned) {
        return SWG_OK;
    }
    swg::RouteArgs p{};
    p.logits = logits;
    p.ld = ldl;
    p.type = type;
    p.bias = bias;
    p.T = (int)T;
    p.E = (int)E;
    p.top = (int)top;
    p.score = score;
    // all groups: no choice
    p.groups = top_groups == groups ? 1 : (int)groups;
    p.top_groups = (int)top_groups;
    p.group_sum = group_sum;
    p.normalise = normalise != 0;
    p.scale = scale;
    p.experts = experts;
    p.weights = weights;
    p.plan = {offsets, source, position};
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int chunks = planned ? swg::plan_chunks(p.T, p.top, true, d.sms) : 0;
    int32_t *counts = nullptr;
    std::unique_lock<std::mutex> held;               // until the counts' reader is queued
    if (int rc = plan_workspace(chunks, E, s, counts, held)) return rc;
    if (int rc = swg::count_launch(swg::launch_route(p, chunks, counts, s))) return rc;
    if (chunks <= 1) return SWG_OK;
    return swg::count_launch(
        swg::launch_sort(p.T, p.E, p.top, experts, p.plan, chunks, counts, nullptr, s));
}

int expert_sort(int64_t T, int64_t E, int64_t top, const int32_t *experts, int32_t *offsets, int32_t *source,
                int32_t *position, void *stream)
{
    if (int rc = check_slots(T, top)) return rc;
    if (E < 1) return SWG_ERR_INVALID_ARG;
    if (E > SWG_MAX_EXPERTS) return SWG_ERR_UNSUPPORTED;
    if (offsets == nullptr || (T > 0 && (experts == nullptr || source == nullptr || position == nullptr)))
        return SWG_ERR_INVALID_ARG;
    if (!aligned4({experts, offsets, source, position})) return SWG_ERR_MISALIGNED;
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const swg::Plan plan{offsets, source, position};
    const int chunks = swg::plan_chunks((int)T, (int)top, false, d.sms);
    int32_t *counts = nullptr;
    std::unique_lock<std::mutex> held;
    if (int rc = plan_workspace(chunks, E, s, counts, held)) return rc;
    if (chunks > 1)
        if (int rc = swg::count_launch(
                swg::launch_count((int)T, (int)E, (int)top, experts, chunks, counts, s)))
            return rc;
    return swg::count_launch(
        swg::launch_sort((int)T, (int)E, (int)top, experts, plan, chunks, counts, d.err, s));
}

int expert_route_grad(int score, int64_t T, int64_t E, int64_t top, const void *logits, int64_t ldl, int type,
                      const int32_t *experts, int normalise, float scale, const float *d_weights,
                      void *d_logits, int64_t ldd, void *stream)
{
    int bytes;
    if (!type_bytes(type, bytes)) return SWG_ERR_UNSUPPORTED;
    if (score != SWG_SOFTMAX && score != SWG_SIGMOID) return SWG_ERR_UNSUPPORTED;
    if (int rc = check_slots(T, top)) return rc;
    if (int rc = check_experts(E, top)) return rc;
    if (!std::isfinite(scale)) return SWG_ERR_INVALID_ARG;
    if (T == 0) return SWG_OK;
    if (experts == nullptr || d_weights == nullptr) return SWG_ERR_INVALID_ARG;
    if (!aligned4({experts, d_weights})) return SWG_ERR_MISALIGNED;
    if (int rc = check_logits(logits, ldl, E, bytes)) return rc;
    if (int rc = check_logits(d_logits, ldd, E, bytes)) return rc;
    swg::RouteGradArgs p{};
    p.logits = logits;
    p.ld = ldl;
    p.type = type;
    p.T = (int)T;
    p.E = (int)E;
    p.top = (int)top;
    p.score = score;
    p.normalise = normalise != 0;
    p.scale = scale;
    p.experts = experts;
    p.d_weights = d_weights;
    p.d_logits = d_logits;
    p.ldd = ldd;
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    return swg::count_launch(swg::launch_route_grad(p, d.err, static_cast<cudaStream_t>(stream)));
}

// Rules and arguments that moving rows has in common.
static int rows_args(int64_t T, int64_t R, int64_t D, int64_t top, int type, const int32_t *position,
                     const float *weights, int &bytes, swg::RowsArgs &p)
{
    if (!type_bytes(type, bytes)) return SWG_ERR_UNSUPPORTED;
    if (int rc = check_slots(T, top)) return rc;
    if (R < 0 || D < 0) return SWG_ERR_INVALID_ARG;
    // (a warp has at least 128 columns, a CTA 8 warps: their number fits 32 bits)
    if (R > kMaxDim || D > kMaxDim || (T > 0 && D / 128 + 1 > 8 * kMaxDim / T)) return SWG_ERR_UNSUPPORTED;
    if (T > 0 && position == nullptr) return SWG_ERR_INVALID_ARG;
    if (!aligned4({position, weights})) return SWG_ERR_MISALIGNED;
    p.T = (int)T;
    p.R = (int)R;
    p.D = (int)D;
    p.top = (int)top;
    p.type = type;
    p.position = position;
    p.weights = weights;
    return SWG_OK;
}

int expert_dispatch(int64_t T, int64_t R, int64_t D, int64_t top, const void *X, int64_t ldx, int type,
                    const int32_t *position, void *rows, int64_t ldr, void *stream)
{
    int bytes;
    swg::RowsArgs p{};
    if (int rc = rows_args(T, R, D, top, type, position, nullptr, bytes, p)) return rc;
    if (T == 0) return SWG_OK;
    if (R == 0) p.D = 0;                             // only positions to look at
    if (p.D > 0) {
        if (int rc = check_rows(X, ldx, D, bytes)) return rc;
        if (int rc = check_rows(rows, ldr, D, bytes)) return rc;
    }
    p.X = X;
    p.ldx = ldx;
    p.rows = rows;
    p.ldr = ldr;
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    return swg::count_launch(swg::launch_dispatch(p, d.sms, d.err, static_cast<cudaStream_t>(stream)));
}

int expert_combine(int64_t T, int64_t R, int64_t D, int64_t top, const void *rows, int64_t ldr, int type,
                   const int32_t *position, const float *weights, float beta, void *out, int64_t ldo,
                   int otype, void *stream)
{
    int bytes, obytes;
    swg::RowsArgs p{};
    if (!type_bytes(otype, obytes) || (otype != type && type != SWG_TYPE_F32)) return SWG_ERR_UNSUPPORTED;
    if (int rc = rows_args(T, R, D, top, type, position, weights, bytes, p)) return rc;
    if (T == 0) return SWG_OK;
    if (D > 0) {
        if (R > 0)
            if (int rc = check_rows(rows, ldr, D, bytes)) return rc;
        if (int rc = check_rows(out, ldo, D, obytes)) return rc;
    }
    p.rows = const_cast<void *>(rows);
    p.ldr = ldr;
    p.out = out;
    p.ldo = ldo;
    p.beta = beta;
    p.out_type = otype;
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    return swg::count_launch(swg::launch_combine(p, d.sms, d.err, static_cast<cudaStream_t>(stream)));
}

int expert_combine_grad(int64_t T, int64_t R, int64_t D, int64_t top, const void *d_out, int64_t ldd,
                        const void *rows, int64_t ldr, int type, const int32_t *position,
                        const float *weights, void *d_rows, int64_t lddr, float *d_weights, void *stream)
{
    int bytes;
    swg::RowsArgs p{};
    if (int rc = rows_args(T, R, D, top, type, position, weights, bytes, p)) return rc;
    if (T == 0) return SWG_OK;
    if (!aligned4({d_weights})) return SWG_ERR_MISALIGNED;
    if (D > 0) {
        if (int rc = check_rows(d_out, ldd, D, bytes)) return rc;
        if (R > 0 && d_weights != nullptr)
            if (int rc = check_rows(rows, ldr, D, bytes)) return rc;
        if (R > 0)
            if (int rc = check_rows(d_rows, lddr, D, bytes)) return rc;
    }
    p.X = d_out;
    p.ldx = ldd;
    p.rows = const_cast<void *>(rows);
    p.ldr = ldr;
    p.out = d_rows;
    p.ldo = lddr;
    p.d_weights = d_weights;
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    return swg::count_launch(swg::launch_combine_grad(p, d.err, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
