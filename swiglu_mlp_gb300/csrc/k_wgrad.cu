// k_wgrad.cu — weight gradients grouped by expert.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts_launch.h"
#include "groups.cuh"
#include "tc_gemm.cuh"

namespace swg {
namespace {

constexpr int T = 64, TK = 16, THREADS = 256;

struct Loader {
    const void *p;
    const uint8_t *s;
    int kind;
    __device__ float get(long long row, long long ld, int k, long long srow, int tiles_k) const
    {
        if (kind == GRP_F16) return __half2float(static_cast<const __half *>(p)[row * ld + k]);
        if (kind == GRP_BF16)
            return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[row * ld + k]);
        const bool nv = kind == GRP_NVFP4;
        const int b = k / (nv ? 16 : 32);
        const uint32_t q = static_cast<const uint8_t *>(p)[row * ld + k / 2] >> (4 * (k & 1));
        const uint32_t c = s[((srow >> 7) * tiles_k + (b >> 2)) * 512 + 16 * (srow & 31) +
                             4 * ((srow & 127) >> 5) + (b & 3)];
        return e2m1_value(q & 15) * mx4_scale_value(nv, c);
    }
};

__global__ void __launch_bounds__(THREADS) simple_wgrad_kernel(WgradArgs p, int *err)
{
    extern __shared__ int table[];
    int *start = table, *first = table + p.groups.G + 1;
    __shared__ float sa[TK][T], sb[TK][T];
    if (threadIdx.x < 32)
        group_table(p.groups, start, first, err, [](int) { return 1; });
    __syncthreads();
    const int g = blockIdx.z;
    const int k0 = blockIdx.y * T, n0 = blockIdx.x * T;
    const Loader la{p.A, nullptr, p.in_bf16 ? GRP_BF16 : GRP_F16};
    const Loader ld{p.D, nullptr, p.in_bf16 ? GRP_BF16 : GRP_F16};
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int r0 = start[g]; r0 < start[g + 1]; r0 += TK) {
        for (int u = threadIdx.x; u < T * TK; u += THREADS) {
            const int c = u % T, r = u / T;
            const bool in = r0 + r < start[g + 1];
            sa[r][c] = in && k0 + c < p.K ? la.get(r0 + r, p.lda, k0 + c, 0, 0) : 0.0f;
            sb[r][c] = in && n0 + c < p.N ? ld.get(r0 + r, p.ldd, n0 + c, 0, 0) : 0.0f;
        }
        __syncthreads();
        for (int r = 0; r < TK; ++r)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[r][ty * 4 + i] * sb[r][tx * 4 + j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (k >= p.K || n >= p.N) continue;
            const long long o = (long long)g * p.strideC + (long long)k * p.ldc + n;
            float v = p.alpha * acc[i][j];
            if (p.beta != 0.0f) v += p.beta * load_out(p.C, o, p.out_kind);
            store_out(p.C, o, v, p.out_kind);
        }
}

}  // namespace

cudaError_t launch_wgrad(const WgradArgs &p, int, int *err, cudaStream_t s)
{
    const dim3 grid((p.N + T - 1) / T, (p.K + T - 1) / T, p.groups.G);
    simple_wgrad_kernel<<<grid, THREADS, 2 * sizeof(int) * (p.groups.G + 1), s>>>(p, err);
    return cudaGetLastError();
}

}  // namespace swg
