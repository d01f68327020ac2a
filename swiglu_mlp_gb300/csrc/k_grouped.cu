// k_grouped.cu — products grouped by expert.
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

__device__ __forceinline__ float sigmoid_f32(float x) { return 1.0f / (1.0f + __expf(-x)); }

template <int EPI>
__global__ void __launch_bounds__(THREADS) simple_kernel(GrpArgs p, int kind, int *err)
{
    extern __shared__ int table[];
    int *start = table, *first = table + p.groups.G + 1;
    __shared__ float sa[TK][T], sb[TK][T];
    if (threadIdx.x < 32)
        group_table(p.groups, start, first, err, [](int rows) { return ceil_div(rows, T); });
    __syncthreads();
    const int t = blockIdx.y;
    if (t >= first[p.groups.G]) return;
    const int g = group_of(first, p.groups.G, t);
    const int local = (t - first[g]) * T;
    const int row0 = start[g] + local, end = start[g + 1];
    const int n0 = blockIdx.x * T;
    const bool nv = kind == GRP_NVFP4;
    const int tiles_k = ceil_div(p.K, nv ? 64 : 128);
    int blocks = 0;                      // rows of scale tiles before this group
    for (int i = 0; i < g; ++i) blocks += ceil_div(start[i + 1] - start[i], 128);
    const Loader la{p.A, p.SA, kind};
    const Loader lb{p.B, p.SB, kind};
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += TK) {
        for (int u = threadIdx.x; u < T * TK; u += THREADS) {
            const int k = u % TK, r = u / TK;
            sa[k][r] = row0 + r < end && k0 + k < p.K
                           ? la.get(row0 + r, p.lda, k0 + k, (long long)blocks * 128 + local + r, tiles_k)
                           : 0.0f;
            float b = 0.0f;
            if (n0 + r < p.N && k0 + k < p.K) {
                const long long rows_b = p.b_kn ? k0 + k : n0 + r;
                const int cols_b = p.b_kn ? n0 + r : k0 + k;
                Loader lg = lb;
                const long long off = (long long)g * p.strideB;
                if (kind >= GRP_MXFP4)
                    lg.p = static_cast<const uint8_t *>(p.B) + off;
                else
                    lg.p = static_cast<const uint16_t *>(p.B) + off;
                b = lg.get(rows_b, p.ldb, cols_b, (long long)g * ceil_div(p.N, 128) * 128 + n0 + r, tiles_k);
            }
            sb[k][r] = b;
        }
        __syncthreads();
        for (int k = 0; k < TK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty * 4 + i] * sb[k][tx * 4 + j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const long long row = row0 + ty * 4 + i;
        if (row >= end) continue;
        if (EPI == GRP_STORE) {
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                if (n >= p.N) continue;
                float v = p.alpha * acc[i][j];
                if (p.beta != 0.0f) v += p.beta * load_out(p.C, row * p.ldc + n, p.out_kind);
                store_out(p.C, row * p.ldc + n, v, p.out_kind);
            }
            continue;
        }
        for (int j = 0; j < 4; j += 2) {
            const int n = n0 + tx * 4 + j;
            if (n >= p.N) continue;
            const float gate = p.alpha * acc[i][j], up = p.alpha * acc[i][j + 1];
            const float s = sigmoid_f32(gate), y = gate * s * up;
            if (EPI == GRP_SWIGLU) {
                store_out(p.C, row * p.ldc + n / 2, y, OUT_BF16);
            } else {
                const float d = load_out(p.dY, row * (p.N / 2) + n / 2, OUT_BF16);
                store_out(p.C, row * p.ldc + n, d * up * s * (1.0f + gate * (1.0f - s)), OUT_BF16);
                store_out(p.C, row * p.ldc + n + 1, d * gate * s, OUT_BF16);
                if (p.Y) store_out(p.Y, row * (p.N / 2) + n / 2, y, OUT_BF16);
            }
        }
    }
}

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

cudaError_t launch_grouped(const GrpArgs &p, GrpKind kind, GrpEpi epi, int, int *err,
                           cudaStream_t s)
{
    const dim3 grid((p.N + T - 1) / T, (p.groups.M + T - 1) / T + p.groups.G);
    const size_t smem = 2 * sizeof(int) * (p.groups.G + 1);
    if (epi == GRP_STORE)
        simple_kernel<GRP_STORE><<<grid, THREADS, smem, s>>>(p, kind, err);
    else if (epi == GRP_SWIGLU)
        simple_kernel<GRP_SWIGLU><<<grid, THREADS, smem, s>>>(p, kind, err);
    else
        simple_kernel<GRP_DSWIGLU><<<grid, THREADS, smem, s>>>(p, kind, err);
    return cudaGetLastError();
}

cudaError_t launch_wgrad(const WgradArgs &p, int, int *err, cudaStream_t s)
{
    const dim3 grid((p.N + T - 1) / T, (p.K + T - 1) / T, p.groups.G);
    simple_wgrad_kernel<<<grid, THREADS, 2 * sizeof(int) * (p.groups.G + 1), s>>>(p, err);
    return cudaGetLastError();
}

}  // namespace swg
