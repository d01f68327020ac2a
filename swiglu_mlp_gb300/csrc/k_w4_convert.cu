// k_w4_convert.cu — weights to 4 bits with group scales, and back.
//
// Both directions stream: 2 bytes (16-bit x) and half a byte per element. A lane
// has eight columns, a word of codes; a warp 256 columns of four rows; a CTA 32
// rows, whose scales (which lie side by side for the rows of a group of columns)
// pass through shared memory, so that they are stored 64 bytes at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.h"
#include "w4.h"

namespace swg {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int THREADS = 256;
constexpr int ROWS = 4;              // per warp
constexpr int CTA_ROWS = 32;
constexpr int COLS = 256;            // per CTA
constexpr int BLOCKS = COLS / 32;    // most groups of columns in them

__device__ __forceinline__ float half_value(uint16_t b, bool bf16)
{
    return bf16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

// Eight columns in FP32, those from cnt on zero and not read.
template <int TYPE>
__device__ __forceinline__ void load8(const void *x, long long i, int cnt, float (&v)[8])
{
    if (TYPE == 2) {
        const float *src = static_cast<const float *>(x) + i;
        if (cnt == 8) {
            const float4 a = reinterpret_cast<const float4 *>(src)[0], b = reinterpret_cast<const float4 *>(src)[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j < cnt ? src[j] : 0.0f;
        }
        return;
    }
    const uint16_t *src = static_cast<const uint16_t *>(x) + i;
    uint32_t u[4] = {};
    if (cnt == 8) {
        const uint4 w = *reinterpret_cast<const uint4 *>(src);
        u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cnt) u[j / 2] |= (uint32_t)src[j] << (16 * (j & 1));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = half_value((uint16_t)(u[j / 2] >> (16 * (j & 1))), TYPE == 1);
}

template <int TYPE>
__device__ __forceinline__ void store8(void *x, long long i, int cnt, const float (&v)[8])
{
    if (TYPE == 2) {
        float *dst = static_cast<float *>(x) + i;
        if (cnt == 8) {
            reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < cnt) dst[j] = v[j];
        }
        return;
    }
    constexpr int kind = TYPE == 1 ? OUT_BF16 : OUT_F16;
    uint16_t *dst = static_cast<uint16_t *>(x) + i;
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = pack2(v[2 * j], v[2 * j + 1], kind);
    if (cnt == 8) {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cnt) dst[j] = (uint16_t)(u[j / 2] >> (16 * (j & 1)));
    }
}

// Bit of column j's code in its word of eight: columns 0, 2, 4, 6 in the lower
// half, 1, 3, 5, 7 in the upper, so that one mask takes a pair of neighbours.
__device__ __forceinline__ constexpr int code_bit(int j) { return 16 * (j & 1) + 4 * (j >> 1); }

// A scale in FP32 to its type: to nearest even; beyond the type's largest value
// that value.
__device__ __forceinline__ uint16_t scale_bits(float s, bool bf16)
{
    if (bf16) {
        const uint16_t b = __bfloat16_as_ushort(__float2bfloat16_rn(s));
        return b == 0x7f80 ? 0x7f7f : b;
    }
    return __half_as_ushort(__float2half_rn(fminf(s, 65504.0f)));
}

template <int TYPE, bool ZERO>
__global__ void __launch_bounds__(THREADS) w4_quantize_kernel(const W4Convert p, int row_tiles)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ uint16_t scales[BLOCKS][CTA_ROWS];
    __shared__ uint8_t zeros[BLOCKS][CTA_ROWS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = blockIdx.x / row_tiles, n0 = (blockIdx.x - g * row_tiles) * CTA_ROWS;
    const int k0 = blockIdx.y * COLS, k = k0 + lane * 8;
    const int cnt = min(max(p.w.K - k, 0), 8), lanes = p.w.group / 8;   // lanes per group of columns
    const bool bf16 = p.stype == 1;
    float v[ROWS][8];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int n = n0 + warp * ROWS + r;
        load8<TYPE>(p.X, ((long long)g * p.w.N + n) * p.ldx + k, n < p.w.N ? cnt : 0, v[r]);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int row = warp * ROWS + r, n = n0 + row;
        float lo = 0.0f, hi = 0.0f;
        bool finite = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            lo = fminf(lo, v[r][j]);
            hi = fmaxf(hi, v[r][j]);
            finite = finite && fabsf(v[r][j]) < __int_as_float(0x7f800000);
        }
        if (!finite) hi = __int_as_float(0x7f800000);    // (a NaN may not show in either)
        for (int d = 1; d < lanes; d <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(ALL, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(ALL, hi, d));
        }
        const bool bad = !(hi < __int_as_float(0x7f800000) && lo > -__int_as_float(0x7f800000));
        const uint16_t bits = scale_bits(ZERO ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f, bf16);
        const float s = half_value(bits, bf16);
        const float inverse = s > 0.0f ? 1.0f / s : 0.0f;
        // x / s with one residual correction (Markstein's), which rounds as the
        // division does where that decides: a tie between two codes times the
        // scale has at most 16 bits, so that an x next to it has a quotient more
        // than half of a float's unit from the tie.  (The inverse of a very small
        // scale may have no FP32 value: divided.)
        const bool plain = s < 0x1p-100f;
        auto quotient = [&](float x) {
            if (plain) return s > 0.0f ? x / s : 0.0f;
            const float q = x * inverse;
            return fmaf(fmaf(-q, s, x), inverse, q);
        };
        const float z = ZERO ? fminf(fmaxf(rintf(quotient(-lo)), 0.0f), 15.0f) : 8.0f;
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = fminf(fmaxf(rintf(quotient(v[r][j])) + z, 0.0f), 15.0f);
            word |= (uint32_t)(j < cnt ? (int)q : 0) << code_bit(j);
        }
        if (bad) word = 0;
        if (n < p.w.N && k < (p.w.K + 31) / 32 * 32)
            *reinterpret_cast<uint32_t *>(const_cast<uint8_t *>(p.w.Q) +
                                          ((long long)g * p.w.N + n) * p.w.row_bytes() + k / 2) = word;
        if (lane % lanes == 0) {
            scales[lane / lanes][row] = bad ? 0x7fff : bits;
            if (ZERO) zeros[lane / lanes][row] = bad ? 0 : (uint8_t)z;
        }
    }
    __syncthreads();
    const int blocks = p.w.blocks(), first = k0 / p.w.group;
    for (int i = threadIdx.x; i < COLS / p.w.group * CTA_ROWS; i += THREADS) {
        const int b = i / CTA_ROWS, row = i % CTA_ROWS;
        if (first + b >= blocks || n0 + row >= p.w.N) continue;
        const long long o = ((long long)g * blocks + first + b) * p.w.lds + n0 + row;
        static_cast<uint16_t *>(const_cast<void *>(p.w.S))[o] = scales[b][row];
        if (ZERO) const_cast<uint8_t *>(p.w.Z)[o] = zeros[b][row];
    }
}

template <int TYPE, bool ZERO>
__global__ void __launch_bounds__(THREADS) w4_dequantize_kernel(const W4Convert p, int row_tiles)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = blockIdx.x / row_tiles, n0 = (blockIdx.x - g * row_tiles) * CTA_ROWS + warp * ROWS;
    const int k = blockIdx.y * COLS + lane * 8;
    const int cnt = min(max(p.w.K - k, 0), 8);
    if (cnt == 0) return;
    const long long at = ((long long)g * p.w.blocks() + k / p.w.group) * p.w.lds + n0;
    uint32_t word[ROWS];
    float s[ROWS], z[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (n0 + r >= p.w.N) continue;
        word[r] = *reinterpret_cast<const uint32_t *>(
            p.w.Q + ((long long)g * p.w.N + n0 + r) * p.w.row_bytes() + k / 2);
        s[r] = half_value(static_cast<const uint16_t *>(p.w.S)[at + r], p.stype == 1);
        z[r] = ZERO ? (float)(p.w.Z[at + r] & 15) : 8.0f;
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (n0 + r >= p.w.N) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = s[r] * ((float)((word[r] >> code_bit(j)) & 15u) - z[r]);
        store8<TYPE>(p.X, ((long long)g * p.w.N + n0 + r) * p.ldx + k, cnt, v);
    }
}

template <int TYPE, bool ZERO>
cudaError_t launch(const W4Convert &p, bool back, cudaStream_t s)
{
    const int row_tiles = (p.w.N + CTA_ROWS - 1) / CTA_ROWS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)p.G * row_tiles), (unsigned)((p.w.K + COLS - 1) / COLS));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return back ? cudaLaunchKernelEx(&cfg, w4_dequantize_kernel<TYPE, ZERO>, p, row_tiles)
                : cudaLaunchKernelEx(&cfg, w4_quantize_kernel<TYPE, ZERO>, p, row_tiles);
}

}  // namespace

cudaError_t launch_w4_convert(const W4Convert &p, bool back, cudaStream_t s)
{
    const bool zero = p.w.Z != nullptr;
    if (p.type == 0) return zero ? launch<0, true>(p, back, s) : launch<0, false>(p, back, s);
    if (p.type == 1) return zero ? launch<1, true>(p, back, s) : launch<1, false>(p, back, s);
    return zero ? launch<2, true>(p, back, s) : launch<2, false>(p, back, s);
}

}  // namespace swg
