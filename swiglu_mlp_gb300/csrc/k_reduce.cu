// k_reduce.cu — the second half of a split contraction of the expert
// operators: sums the FP32 partials of the K ranges in their order, so results
// do not depend on which range was done first, and applies the epilogue.  One
// row, 4096 x 4096 in 4 ranges: 11.6 us with the product, of 17.2 in one range.
#include <algorithm>

#include "experts_launch.h"
#include "tc_gemm.cuh"

namespace swg {
namespace {

constexpr int THREADS = 256;
constexpr int COLS = 8;              // accumulator columns per thread

// It streams 4 bytes per partial and accumulator once, a few MB that the
// products before it left in L2, so its time is a launch; that overlaps the
// product's end (programmatic dependent launch).
template <int EPI>
__global__ void __launch_bounds__(THREADS) reduce_kernel(const ReduceArgs p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int begin = 0, end = p.rows;
    if (p.groups.offsets != nullptr) {
        // the rows of the groups as the products clamp them (groups.cuh): from
        // the first offset to the largest
        int top = 0;
        for (int i = threadIdx.x & 31; i <= p.groups.G; i += 32) top = max(top, p.groups.offsets[i]);
        begin = max(p.groups.offsets[0], 0);
        end = min(__reduce_max_sync(0xffffffffu, top), p.groups.M);
    }
    const int per_row = (p.N + COLS - 1) / COLS;
    const long long total = (long long)p.rows * per_row;
    for (long long i = blockIdx.x * (long long)THREADS + threadIdx.x; i < total;
         i += (long long)gridDim.x * THREADS) {
        const int row = (int)(i / per_row), n = (int)(i - (long long)row * per_row) * COLS;
        if (row < begin || row >= end) continue;
        float v[COLS] = {};
        const float *src = p.ws + row * p.ld + n;
        for (int s = 0; s < p.splits; ++s) {
            const float4 a = reinterpret_cast<const float4 *>(src + s * p.stride)[0];
            const float4 b = reinterpret_cast<const float4 *>(src + s * p.stride)[1];
            v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
            v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
        }
        if (EPI == GRP_STORE) {
            const int g = p.per_group > 0 ? row / p.per_group : 0;
            const long long o = g * p.strideC + (row - g * (long long)p.per_group) * p.ldc + n;
#pragma unroll
            for (int j = 0; j < COLS; ++j) {
                v[j] *= p.alpha;
                if (p.beta != 0.0f && n + j < p.N) v[j] += p.beta * load_out(p.C, o + j, p.out_kind);
            }
            if (n + COLS <= p.N && p.out_kind != OUT_F32) {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.C) + o) =
                    make_uint4(pack2(v[0], v[1], p.out_kind), pack2(v[2], v[3], p.out_kind),
                               pack2(v[4], v[5], p.out_kind), pack2(v[6], v[7], p.out_kind));
            } else {
#pragma unroll
                for (int j = 0; j < COLS; ++j)
                    if (n + j < p.N) store_out(p.C, o + j, v[j], p.out_kind);
            }
            continue;
        }
        // (N is a multiple of 16 here)
        const long long half = row * (long long)(p.N / 2) + n / 2;
        float y[COLS / 2];
#pragma unroll
        for (int j = 0; j < COLS / 2; ++j) {
            const float g = p.alpha * v[2 * j], u = p.alpha * v[2 * j + 1];
            if (EPI == GRP_SWIGLU) {
                y[j] = silu_f32(g) * u;
            } else {
                const float s = __fdividef(1.0f, 1.0f + __expf(-g));
                const float d = load_out(p.dY, half + j, OUT_BF16);
                const float gs = g * s;
                y[j] = gs * u;
                v[2 * j] = d * u * (s + gs * (1.0f - s));
                v[2 * j + 1] = d * gs;
            }
        }
        const uint2 yy = make_uint2(pack2(y[0], y[1], OUT_BF16), pack2(y[2], y[3], OUT_BF16));
        if (EPI == GRP_SWIGLU) {
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.C) + row * p.ldc + n / 2) = yy;
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.C) + row * p.ldc + n) =
                make_uint4(pack2(v[0], v[1], OUT_BF16), pack2(v[2], v[3], OUT_BF16),
                           pack2(v[4], v[5], OUT_BF16), pack2(v[6], v[7], OUT_BF16));
            if (p.Y) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.Y) + half) = yy;
        }
    }
}

}  // namespace

cudaError_t launch_reduce(const ReduceArgs &p, GrpEpi epi, int sms, cudaStream_t s)
{
    const long long work = (long long)p.rows * ((p.N + COLS - 1) / COLS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long long>((work + THREADS - 1) / THREADS, sms * 8LL));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return epi == GRP_STORE    ? cudaLaunchKernelEx(&cfg, reduce_kernel<GRP_STORE>, p)
           : epi == GRP_SWIGLU ? cudaLaunchKernelEx(&cfg, reduce_kernel<GRP_SWIGLU>, p)
                               : cudaLaunchKernelEx(&cfg, reduce_kernel<GRP_DSWIGLU>, p);
}

}  // namespace swg
