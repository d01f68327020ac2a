// k_w4_convert.cu — weights to 4 bits with group scales, and back.
//
// Both directions stream: 2 bytes (16-bit x) and half a byte per element, which
// leaves about ten instructions per element and lane; so a code costs a product with
// two corrections, two bounds, an addition that rounds and one that packs.  A lane
// has eight columns, a word of codes; a warp 256 columns of four rows; a CTA 32
// rows, whose scales (which lie side by side for the rows of a group of columns)
// pass through shared memory, so that they are stored 64 bytes at a time.
//
// 14336 x 4096 bfloat16, groups of 128: 43 us there and 24.5 back, 3.4 and 6.0 TB/s.  On the
// way there instructions bound it (the range, the quotient and its correction); FP32 pairs in
// one instruction and ranges in 16 bits took it from 62.
#include <type_traits>

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
constexpr int ROWS_BACK = 8;         // ... of the way back, to have as much to read on the way
constexpr int CTA_ROWS_BACK = 64;
constexpr int COLS = 256;            // per CTA
constexpr int BLOCKS = COLS / 32;    // most groups of columns in them

__device__ __forceinline__ float half_value(uint16_t b, bool bf16)
{
    return bf16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

// The larger, or smaller, of two; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Eight columns as they are stored; those from cnt on are zero and not read.
template <int TYPE> struct Raw8 {
    uint32_t u[TYPE == 2 ? 8 : 4];
};

template <int TYPE>
__device__ __forceinline__ Raw8<TYPE> load8(const void *x, long long i, int cnt)
{
    Raw8<TYPE> r;
    if (TYPE == 2) {
        const float *src = static_cast<const float *>(x) + i;
        if (cnt == 8) {
            const uint4 a = reinterpret_cast<const uint4 *>(src)[0], b = reinterpret_cast<const uint4 *>(src)[1];
            r.u[0] = a.x, r.u[1] = a.y, r.u[2] = a.z, r.u[3] = a.w;
            r.u[TYPE == 2 ? 4 : 0] = b.x, r.u[TYPE == 2 ? 5 : 0] = b.y, r.u[TYPE == 2 ? 6 : 0] = b.z, r.u[TYPE == 2 ? 7 : 0] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r.u[j % (TYPE == 2 ? 8 : 4)] = j < cnt ? __float_as_uint(src[j]) : 0u;
        }
        return r;
    }
    const uint16_t *src = static_cast<const uint16_t *>(x) + i;
    if (cnt == 8) {
        const uint4 w = *reinterpret_cast<const uint4 *>(src);
        r.u[0] = w.x, r.u[1] = w.y, r.u[2] = w.z, r.u[3] = w.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) r.u[j] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cnt) r.u[j / 2] |= (uint32_t)src[j] << (16 * (j & 1));
    }
    return r;
}

// Columns 2 j and 2 j + 1 in FP32.
template <int TYPE>
__device__ __forceinline__ float2 pair(const Raw8<TYPE> &r, int j)
{
    if (TYPE == 2) return make_float2(__uint_as_float(r.u[(2 * j) % (TYPE == 2 ? 8 : 4)]), __uint_as_float(r.u[(2 * j + 1) % (TYPE == 2 ? 8 : 4)]));
    if (TYPE == 1) return make_float2(__uint_as_float(r.u[j] << 16), __uint_as_float(r.u[j] & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&r.u[j]));
}

// The range of the eight columns and 0 (not ZERO: hi the largest magnitude), NaN where
// there is one; of 16-bit columns two at a time.
template <int TYPE, bool ZERO>
__device__ __forceinline__ void range8(const Raw8<TYPE> &r, float &lo, float &hi)
{
    lo = hi = 0.0f;
    if constexpr (TYPE == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = __uint_as_float(r.u[j]);
            if (ZERO) lo = min_nan(lo, v);
            hi = max_nan(hi, ZERO ? v : fabsf(v));
        }
    } else {
        using T2 = std::conditional_t<TYPE == 1, __nv_bfloat162, __half2>;
        auto two = [](uint32_t u) { return *reinterpret_cast<const T2 *>(&u); };
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = ZERO ? r.u[j] : r.u[j] & 0x7fff7fffu;
        const T2 top = __hmax2_nan(__hmax2_nan(two(u[0]), two(u[1])), __hmax2_nan(two(u[2]), two(u[3])));
        Raw8<TYPE> f;
        f.u[0] = *reinterpret_cast<const uint32_t *>(&top);
        const float2 t = pair<TYPE>(f, 0);
        hi = max_nan(hi, max_nan(t.x, t.y));
        if (ZERO) {
            const T2 low = __hmin2_nan(__hmin2_nan(two(u[0]), two(u[1])), __hmin2_nan(two(u[2]), two(u[3])));
            f.u[0] = *reinterpret_cast<const uint32_t *>(&low);
            const float2 b = pair<TYPE>(f, 0);
            lo = min_nan(lo, min_nan(b.x, b.y));
        }
    }
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

// x / s from the product with the inverse and one residual correction
// (Markstein's), which rounds as the division does where that decides: a tie
// between two codes times the scale has at most 16 bits, so that an x next to it has
// a quotient more than half of a float's unit from the tie.  Scales below TINY, and
// what they divide, are made LARGER first, or the inverse might have no FP32 value.
constexpr float TINY = 0x1p-100f, LARGER = 0x1p100f;
__device__ __forceinline__ float quotient(float x, float s, float inverse)
{
    const float q = x * inverse;
    return fmaf(fmaf(-q, s, x), inverse, q);
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
    Raw8<TYPE> raw[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int n = n0 + warp * ROWS + r;
        raw[r] = load8<TYPE>(p.X, ((long long)g * p.w.N + n) * p.ldx + k, n < p.w.N ? cnt : 0);
    }
    // where this lane's codes end (those of columns that do not exist are 0)
    uint32_t keep = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < cnt) keep |= 15u << code_bit(j);
    // The ranges of the rows' groups of columns.  (max.NaN: a NaN anywhere shows.)
    float lo[ROWS], hi[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        range8<TYPE, ZERO>(raw[r], lo[r], hi[r]);
        for (int d = 1; d < lanes; d <<= 1) {
            hi[r] = max_nan(hi[r], __shfl_xor_sync(ALL, hi[r], d));
            if (ZERO) lo[r] = min_nan(lo[r], __shfl_xor_sync(ALL, lo[r], d));
        }
    }
    // Four lanes of a group of columns compute a row's scale each: its bits (0x7fff, a
    // NaN, where the group holds a NaN or an infinity), inverse and zero point.
    static_assert(ROWS == 4, "a row for each of a group's four first lanes");
    uint32_t my_bits;
    float my_inverse, my_zero = 8.0f;
    {
        const int r = lane & 3;
        const float h = r == 0 ? hi[0] : r == 1 ? hi[1] : r == 2 ? hi[2] : hi[3];
        const float l = !ZERO ? 0.0f : r == 0 ? lo[0] : r == 1 ? lo[1] : r == 2 ? lo[2] : lo[3];
        const float inf = __int_as_float(0x7f800000);
        my_bits = scale_bits(ZERO ? (h - l) / 15.0f : h / 7.0f, bf16);
        const float s = half_value((uint16_t)my_bits, bf16);
        // (the inverse of a very small scale may have no FP32 value: see below)
        my_inverse = s > 0.0f ? 1.0f / (s < TINY ? s * LARGER : s) : 0.0f;
        if (ZERO) {
            const float larger = s < TINY ? LARGER : 1.0f;
            my_zero = fminf(fmaxf(rintf(quotient(-l * larger, s * larger, my_inverse)), 0.0f), 15.0f);
        }
        if (!(h < inf) || !(l > -inf)) {
            my_bits = 0x7fff;
            my_zero = 0.0f;
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int row = warp * ROWS + r, n = n0 + row;
        const int from = (lane & ~3) + r;
        const uint32_t bits = __shfl_sync(ALL, my_bits, from);
        const float inverse = __shfl_sync(ALL, my_inverse, from);
        const float z = ZERO ? __shfl_sync(ALL, my_zero, from) : 8.0f;
        const bool bad = bits == 0x7fffu;
        const float s = half_value((uint16_t)bits, bf16);
        const bool tiny = s < TINY;
        // 2^23 + 2^22 takes the units' place: the sum is rounded to a whole number,
        // ties to even, and its lowest bits are that number's.
        constexpr float UNITS = 12582912.0f;
        uint32_t word = 0;
        // Without a zero point a quotient is at most 7 and a scale's rounding, which needs no
        // bound, unless the scale's type has no digits left or the scale was too large.
        const bool plain = !ZERO && s >= (bf16 ? TINY : 0x1p-14f) && s < (bf16 ? 0x1p126f : 65504.0f);
        if (__all_sync(ALL, plain || bad)) {
            const float2 inv = make_float2(inverse, inverse), less = make_float2(-s, -s), units = make_float2(UNITS, UNITS);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = pair<TYPE>(raw[r], j), q = __fmul2_rn(x, inv);
                const float2 u = __fadd2_rn(__ffma2_rn(__ffma2_rn(q, less, x), inv, q), units);
                word += __float_as_uint(u.x) << code_bit(2 * j);
                word += __float_as_uint(u.y) << code_bit(2 * j + 1);
            }
        } else {
            const float larger = tiny ? LARGER : 1.0f, scale = s * larger;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 x = pair<TYPE>(raw[r], j / 2);
                const float q = quotient((j & 1 ? x.y : x.x) * larger, scale, inverse);
                word += __float_as_uint(fminf(fmaxf(q, -z), 15.0f - z) + UNITS) << code_bit(j);
            }
        }
        // less the units, plus the zero point, in every code's place
        uint32_t places = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) places += 1u << code_bit(j);
        word += places * ((uint32_t)(int)z - __float_as_uint(UNITS));
        word = bad ? 0 : word & keep;
        if (n < p.w.N && k < (p.w.K + 31) / 32 * 32)
            *reinterpret_cast<uint32_t *>(const_cast<uint8_t *>(p.w.Q) +
                                          ((long long)g * p.w.N + n) * p.w.row_bytes() + k / 2) = word;
        if (lane % lanes == 0) {
            scales[lane / lanes][row] = (uint16_t)bits;
            if (ZERO) zeros[lane / lanes][row] = (uint8_t)z;
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
    const int g = blockIdx.x / row_tiles, n0 = (blockIdx.x - g * row_tiles) * CTA_ROWS_BACK + warp * ROWS_BACK;
    const int k = blockIdx.y * COLS + lane * 8;
    const int cnt = min(max(p.w.K - k, 0), 8);
    if (cnt == 0) return;
    const long long at = ((long long)g * p.w.blocks() + k / p.w.group) * p.w.lds + n0;
    if (TYPE == p.stype && cnt == 8) {
        // To the scales' own type two at a time: a code less its zero point is exact
        // there, and its product with the scale is rounded once.
        using T2 = std::conditional_t<TYPE == 1, __nv_bfloat162, __half2>;
        constexpr uint32_t UNITS = TYPE == 1 ? 0x43004300u : 0x64006400u;    // 128 or 1024: a code in the units' place
        uint32_t codes[ROWS_BACK], scale[ROWS_BACK], zero[ROWS_BACK];
#pragma unroll
        for (int r = 0; r < ROWS_BACK; ++r) {
            const int n = min(n0 + r, p.w.N - 1) - n0;           // (n0 may be behind the last row)
            codes[r] = *reinterpret_cast<const uint32_t *>(p.w.Q + ((long long)g * p.w.N + n0 + n) * p.w.row_bytes() + k / 2);
            scale[r] = static_cast<const uint16_t *>(p.w.S)[at + n];
            zero[r] = ZERO ? p.w.Z[at + n] & 15u : 8u;
        }
#pragma unroll
        for (int r = 0; r < ROWS_BACK; ++r) {
            if (n0 + r >= p.w.N) continue;
            const uint32_t w = codes[r], zz = UNITS + zero[r] * 0x00010001u, ss = scale[r] * 0x00010001u;
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t q = ((w >> (4 * i)) & 0x000f000fu) | UNITS;
                const T2 d = __hmul2(__hsub2(*reinterpret_cast<const T2 *>(&q), *reinterpret_cast<const T2 *>(&zz)),
                                     *reinterpret_cast<const T2 *>(&ss));
                u[i] = *reinterpret_cast<const uint32_t *>(&d);
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.X) + ((long long)g * p.w.N + n0 + r) * p.ldx + k) =
                make_uint4(u[0], u[1], u[2], u[3]);
        }
        return;
    }
    uint32_t word[ROWS_BACK];
    float s[ROWS_BACK], z[ROWS_BACK];
#pragma unroll
    for (int r = 0; r < ROWS_BACK; ++r) {
        if (n0 + r >= p.w.N) continue;
        word[r] = *reinterpret_cast<const uint32_t *>(
            p.w.Q + ((long long)g * p.w.N + n0 + r) * p.w.row_bytes() + k / 2);
        s[r] = half_value(static_cast<const uint16_t *>(p.w.S)[at + r], p.stype == 1);
        z[r] = ZERO ? (float)(p.w.Z[at + r] & 15) : 8.0f;
    }
#pragma unroll
    for (int r = 0; r < ROWS_BACK; ++r) {
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
    const int rows = back ? CTA_ROWS_BACK : CTA_ROWS, row_tiles = (p.w.N + rows - 1) / rows;
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
