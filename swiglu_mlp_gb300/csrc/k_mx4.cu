// k_mx4.cu — microscaled 4-bit floating point: to 4 bits and back.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "experts_launch.h"
#include "groups.cuh"
#include "tc_gemm.cuh"

namespace swg {
namespace {

constexpr int TILE_ROWS = 128;       // rows of a scale tile
constexpr int THREADS = 256;

__device__ __forceinline__ float load_f32(const void *x, long long i, int type)
{
    if (type == 2) return static_cast<const float *>(x)[i];
    if (type == 1) return __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i]);
    return __half2float(static_cast<const __half *>(x)[i]);
}

__device__ __forceinline__ void store_f32(void *x, long long i, float v, int type)
{
    if (type == 2)
        static_cast<float *>(x)[i] = v;
    else if (type == 1)
        static_cast<__nv_bfloat16 *>(x)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(x)[i] = __float2half_rn(v);
}

// The scale of a block whose largest magnitude is `top`: its byte and value.
__device__ __forceinline__ uint32_t block_scale(bool nv, float top, float &scale)
{
    if (nv) {
        if (!(top <= 3.402823466e38f)) {                 // NaN or infinity
            scale = __int_as_float(0x7fffffff);
            return 0x7fu;
        }
        const float s = fminf(__fdiv_rn(top, 6.0f), 448.0f);
        uint32_t code = __nv_cvt_float_to_fp8(s, __NV_SATFINITE, __NV_E4M3);
        if (code == 0) code = 1;                         // at least 2^-9
        scale = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
        return code;
    }
    const int e = (__float_as_int(top) >> 23) & 0xff;    // exponent field of |x|
    if (e == 255) {
        scale = __int_as_float(0x7fffffff);
        return 0xffu;
    }
    const uint32_t code = e > 2 ? e - 2 : 0;             // 2^(floor(log2 top) - 2)
    scale = __int_as_float(code > 0 ? code << 23 : 1 << 22);
    return code;
}

// One thread per block of one row.
__global__ void __launch_bounds__(THREADS)
    quantize_kernel(Mx4Args p, int *err)
{
    extern __shared__ int table[];
    int *start = table, *first = table + p.groups.G + 1;
    const bool nv = p.format == 1;
    const int B = nv ? 16 : 32;
    const int tiles_k = ceil_div(p.K, 4 * B);
    if (threadIdx.x < 32)
        group_table(p.groups, start, first, err,
                    [](int rows) { return ceil_div(rows, TILE_ROWS); });
    __syncthreads();
    const int t = blockIdx.y;
    if (t >= first[p.groups.G]) return;
    const int g = group_of(first, p.groups.G, t);
    const int row0 = start[g] + (t - first[g]) * TILE_ROWS;
    for (int u = threadIdx.x; u < TILE_ROWS * 4; u += THREADS) {
        const int r = u >> 2, b = u & 3;
        const int row = row0 + r;
        const int k0 = (blockIdx.x * 4 + b) * B;
        uint32_t code = 0;
        if (row < start[g + 1] && k0 < p.K) {
            float top = 0.0f, scale;
            bool nan = false;
            for (int i = 0; i < B && k0 + i < p.K; ++i) {
                const float v = fabsf(p.scale * load_f32(p.X, (long long)row * p.ldx + k0 + i, p.type));
                nan = nan || v != v;
                top = fmaxf(top, v);
            }
            if (nan) top = __int_as_float(0x7fffffff);
            code = block_scale(nv, top, scale);
            uint8_t *q = p.Q + (long long)row * p.ldq + k0 / 2;
            for (int i = 0; i < B; i += 2) {
                float v[2];
                for (int j = 0; j < 2; ++j)
                    v[j] = k0 + i + j < p.K
                               ? __fdiv_rn(p.scale * load_f32(p.X, (long long)row * p.ldx + k0 + i + j, p.type), scale)
                               : 0.0f;
                q[i / 2] = __nv_cvt_float2_to_fp4x2(make_float2(v[0], v[1]), __NV_E2M1, cudaRoundNearest);
            }
            // NVFP4: the codes up to a multiple of 32 columns are zero too
            if (nv && k0 + 16 >= p.K && (k0 & 31) == 0)
                for (int i = 8; i < 16; ++i) q[i] = 0;
        }
        p.S[((long long)t * tiles_k + blockIdx.x) * 512 + 16 * (r & 31) + 4 * (r >> 5) + b] =
            (uint8_t)code;
    }
}

__global__ void __launch_bounds__(THREADS)
    dequantize_kernel(Mx4Args p, int *err)
{
    extern __shared__ int table[];
    int *start = table, *first = table + p.groups.G + 1;
    const bool nv = p.format == 1;
    const int B = nv ? 16 : 32;
    const int tiles_k = ceil_div(p.K, 4 * B);
    if (threadIdx.x < 32)
        group_table(p.groups, start, first, err,
                    [](int rows) { return ceil_div(rows, TILE_ROWS); });
    __syncthreads();
    const int t = blockIdx.y;
    if (t >= first[p.groups.G]) return;
    const int g = group_of(first, p.groups.G, t);
    const int row0 = start[g] + (t - first[g]) * TILE_ROWS;
    for (int u = threadIdx.x; u < TILE_ROWS * 4; u += THREADS) {
        const int r = u >> 2, b = u & 3;
        const int row = row0 + r;
        const int k0 = (blockIdx.x * 4 + b) * B;
        if (row >= start[g + 1] || k0 >= p.K) continue;
        const uint32_t code =
            p.S[((long long)t * tiles_k + blockIdx.x) * 512 + 16 * (r & 31) + 4 * (r >> 5) + b];
        const float s = mx4_scale_value(nv, code);
        for (int i = 0; i < B && k0 + i < p.K; ++i) {
            const uint32_t q = p.Q[(long long)row * p.ldq + (k0 + i) / 2] >> (4 * (i & 1));
            store_f32(p.X, (long long)row * p.ldx + k0 + i, p.scale * (e2m1_value(q & 15) * s), p.type);
        }
    }
}

}  // namespace

cudaError_t launch_mx4(const Mx4Args &p, bool back, int tile_rows, int *err, cudaStream_t s)
{
    const int B = p.format == 1 ? 16 : 32;
    const dim3 grid((p.K + 4 * B - 1) / (4 * B), tile_rows);
    const size_t smem = 2 * sizeof(int) * (p.groups.G + 1);
    if (back)
        dequantize_kernel<<<grid, THREADS, smem, s>>>(p, err);
    else
        quantize_kernel<<<grid, THREADS, smem, s>>>(p, err);
    return cudaGetLastError();
}

}  // namespace swg
