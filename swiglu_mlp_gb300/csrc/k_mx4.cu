// k_mx4.cu — microscaled 4-bit floating point: to 4 bits and back.
//
// Both directions stream: 2 bytes (16-bit x) and 1/2 + 1/32 or 1/16 bytes per
// element, each once, so memory bounds them.  A CTA takes 256 columns of 32 of
// the 128 rows of a row of scale tiles: those with r mod 32 in one eighth, in
// fours r, r + 32, r + 64, r + 96 a warp, whose scales lie side by side in
// memory.  A lane has 8 columns of each of its warp's four rows: one 16-byte
// access of x and 4 bytes of codes per row.  A block's largest magnitude meets
// across its 4 (MXFP4) or 2 (NVFP4) lanes, and four lanes swap their blocks'
// scale bytes so that each stores 4 bytes of a tile.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "experts_launch.h"
#include "groups.cuh"
#include "launch.h"
#include "tc_gemm.cuh"

namespace swg {
namespace {

constexpr int TILE_ROWS = 128;       // rows of a scale tile
constexpr int TILE_COLS = 256;       // columns per CTA: 2 (MXFP4) or 4 (NVFP4) scale tiles
constexpr int THREADS = 256;
constexpr int STRIPS = 4;            // CTAs per row of scale tiles
constexpr int ROWS = 4;              // rows per warp, 32 apart

template <int TYPE> struct Elem;
template <> struct Elem<0> { using T = __half; };
template <> struct Elem<1> { using T = __nv_bfloat16; };
template <> struct Elem<2> { using T = float; };

// 8 columns of a row as they are stored; those from `cnt` on are zero and not
// read.
template <int TYPE> struct Raw8 {
    uint4 w[TYPE == 2 ? 2 : 1];
};

template <int TYPE>
__device__ __forceinline__ Raw8<TYPE> load8(const void *x, long long i, int cnt)
{
    using T = typename Elem<TYPE>::T;
    const T *src = static_cast<const T *>(x) + i;
    Raw8<TYPE> r;
    if (cnt == 8) {
        r.w[0] = reinterpret_cast<const uint4 *>(src)[0];
        if (TYPE == 2) r.w[TYPE == 2] = reinterpret_cast<const uint4 *>(src)[1];
    } else {
        uint32_t u[TYPE == 2 ? 8 : 4] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= cnt) continue;
            if (TYPE == 2)
                u[j % (TYPE == 2 ? 8 : 4)] = reinterpret_cast<const uint32_t *>(src)[j];
            else
                u[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(src)[j] << (16 * (j & 1));
        }
#pragma unroll
        for (int h = 0; h < (TYPE == 2 ? 2 : 1); ++h)
            r.w[h] = make_uint4(u[4 * h], u[4 * h + 1], u[4 * h + 2], u[4 * h + 3]);
    }
    return r;
}

template <int TYPE>
__device__ __forceinline__ void to_floats(const Raw8<TYPE> &r, float (&v)[8])
{
#pragma unroll
    for (int h = 0; h < (TYPE == 2 ? 2 : 1); ++h) {
        const uint32_t u[4] = {r.w[h].x, r.w[h].y, r.w[h].z, r.w[h].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (TYPE == 2) {
                v[4 * h + j] = __uint_as_float(u[j]);
            } else {
                const float2 f = TYPE == 1
                                     ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[j]))
                                     : __half22float2(*reinterpret_cast<const __half2 *>(&u[j]));
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        }
    }
}

template <int TYPE>
__device__ __forceinline__ void store8(void *x, long long i, int cnt, const float (&v)[8])
{
    using T = typename Elem<TYPE>::T;
    T *dst = static_cast<T *>(x) + i;
    if (cnt == 8 && TYPE == 2) {
        reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if (cnt == 8) {
        constexpr int kind = TYPE == 1 ? OUT_BF16 : OUT_F16;
        *reinterpret_cast<uint4 *>(dst) =
            make_uint4(pack2(v[0], v[1], kind), pack2(v[2], v[3], kind), pack2(v[4], v[5], kind),
                       pack2(v[6], v[7], kind));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cnt) dst[j] = T(v[j]);
    }
}

// The larger of two magnitudes; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The scale of a block whose largest magnitude is `top` (NaN if the block has
// one): its byte; `scale` its value and `inverse` 1 / scale, both NaN for a
// block with a NaN or an infinity.
template <bool NV>
__device__ __forceinline__ uint32_t block_scale(float top, float &scale, float &inverse)
{
    const uint32_t bits = __float_as_uint(top) & 0x7fffffffu;
    const float nan = __uint_as_float(0x7fffffffu);
    if (NV) {
        // to nearest even by the conversion, which saturates at 448
        const uint32_t code = max(
            (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(top, 6.0f), __NV_SATFINITE, __NV_E4M3), 1u);
        const bool bad = bits >= 0x7f800000u;
        scale = bad ? nan
                    : __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
        inverse = __frcp_rn(scale);
        return bad ? 0x7fu : code;
    }
    const uint32_t e = bits >> 23;                   // floor(log2 top) + 127
    const uint32_t code = e > 2 ? e - 2 : 0;
    const bool bad = e == 255;
    scale = bad ? nan : __uint_as_float(code > 0 ? code << 23 : 1u << 22);
    inverse = bad ? nan : __uint_as_float((254u - code) << 23);       // 2^(127 - code), exact
    return bad ? 0xffu : code;
}

struct Place {
    int t;                   // row of scale tiles
    int chunk;               // 256 columns
    int r32;                 // this warp's rows: r32, r32 + 32, ..
    int row0, end;           // first row of the tiles, end of their group
};

// This CTA's and warp's place; false for a CTA beyond the last group's tiles.
__device__ __forceinline__ bool find_place(const Groups &gr, int chunks, int *err, int *table,
                                           Place &p)
{
    const unsigned strip = blockIdx.x / (unsigned)chunks;
    p.chunk = (int)(blockIdx.x - strip * (unsigned)chunks);
    p.t = (int)(strip / STRIPS);
    p.r32 = (int)(strip % STRIPS) * 8 + (threadIdx.x >> 5);
    if (gr.offsets == nullptr) {
        p.row0 = p.t * TILE_ROWS;
        p.end = gr.M;
        return p.row0 < gr.M;
    }
    int *start = table, *first = table + gr.G + 1, *sums = table + 2 * (gr.G + 1);
    group_starts<THREADS>(gr, start, err);
    tile_sums<THREADS>(gr.G, start, first, sums, [](int rows) { return ceil_div(rows, TILE_ROWS); });
    if (p.t >= first[gr.G]) return false;
    const int g = group_of(first, gr.G, 1, p.t);
    p.row0 = start[g] + (p.t - first[g]) * TILE_ROWS;
    p.end = start[g + 1];
    return true;
}

template <int TYPE, bool NV>
__global__ void __launch_bounds__(THREADS) quantize_kernel(const Mx4Args p, int chunks, int *err)
{
    constexpr int LANES = NV ? 2 : 4;                // lanes per block
    constexpr int TILES = NV ? 4 : 2;                // scale tiles per CTA along K
    extern __shared__ int table[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Place at;
    if (!find_place(p.groups, chunks, err, table, at)) return;
    const int lane = threadIdx.x & 31;
    const int k = at.chunk * TILE_COLS + lane * 8;
    const int cnt = min(8, max(0, p.K - k));
    const bool write = k < ((p.K + 31) & ~31);       // codes up to a multiple of 32 columns
    const bool block = k - (lane % LANES) * 8 < p.K; // the lane's block has columns
    Raw8<TYPE> raw[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = at.row0 + at.r32 + 32 * i;
        raw[i] = load8<TYPE>(p.X, (long long)row * p.ldx + k, row < at.end ? cnt : 0);
    }
    uint32_t codes = 0;                              // the lane's block's scales, a byte per row
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = at.row0 + at.r32 + 32 * i;
        float v[8], top = 0.0f;
        to_floats<TYPE>(raw[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] *= p.scale;
            top = max_nan(top, fabsf(v[j]));
        }
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        if (!NV) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float s, inv;
        const uint32_t code = block_scale<NV>(top, s, inv);
        uint32_t q = 0;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float a = v[j] * inv, c = v[j + 1] * inv;
            if (NV) {
                // One residual correction (Markstein's): a quotient that is
                // itself a float -- every tie between two codes is, for
                // 16-bit x -- comes out exact, so ties go to even as in the
                // definition; a * inv alone may miss them by a rounding.
                a = __fmaf_rn(__fmaf_rn(-a, s, v[j]), inv, a);
                c = __fmaf_rn(__fmaf_rn(-c, s, v[j + 1]), inv, c);
            }
            q |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(a, c), __NV_E2M1, cudaRoundNearest)
                 << (4 * j);
        }
        if (row < at.end && write)
            *reinterpret_cast<uint32_t *>(p.Q + (long long)row * p.ldq + k / 2) = q;
        if (row < at.end && block) codes |= code << (8 * i);
    }
    // Lane b of a tile's four blocks takes row b's four bytes and stores them.
    const int b = lane / LANES % 4, tile = lane / (4 * LANES);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = __shfl_sync(0xffffffffu, codes, tile * 4 * LANES + i * LANES);
        word |= ((c >> (8 * b)) & 0xffu) << (8 * i);
    }
    const int tiles_k = ceil_div(p.K, NV ? 64 : 128);
    const int kt = at.chunk * TILES + tile;
    if (lane % LANES == 0 && kt < tiles_k)
        *reinterpret_cast<uint32_t *>(p.S + ((long long)at.t * tiles_k + kt) * 512 + 16 * at.r32 +
                                      4 * b) = word;
}

template <int TYPE, bool NV>
__global__ void __launch_bounds__(THREADS) dequantize_kernel(const Mx4Args p, int chunks, int *err)
{
    constexpr int LANES = NV ? 2 : 4;
    constexpr int TILES = NV ? 4 : 2;
    extern __shared__ int table[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Place at;
    if (!find_place(p.groups, chunks, err, table, at)) return;
    const int lane = threadIdx.x & 31;
    const int k = at.chunk * TILE_COLS + lane * 8;
    const int cnt = min(8, max(0, p.K - k));
    if (cnt == 0) return;
    uint32_t q[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = at.row0 + at.r32 + 32 * i;
        q[i] = row < at.end ? *reinterpret_cast<const uint32_t *>(p.Q + (long long)row * p.ldq + k / 2) : 0;
    }
    // 16 bytes: the four rows' scales of the tile's four blocks
    const int b = lane / LANES % 4, kt = at.chunk * TILES + lane / (4 * LANES);
    const uint4 w = *reinterpret_cast<const uint4 *>(
        p.S + ((long long)at.t * ceil_div(p.K, NV ? 64 : 128) + kt) * 512 + 16 * at.r32);
    const uint32_t words[ROWS] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = at.row0 + at.r32 + 32 * i;
        if (row >= at.end) continue;
        const float s = mx4_scale_value(NV, (words[i] >> (8 * b)) & 0xffu);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2(
                (__nv_fp4x2_storage_t)((q[i] >> (4 * j)) & 0xffu), __NV_E2M1));
            const float2 f = __half22float2(h);
            v[j] = p.scale * (f.x * s);
            v[j + 1] = p.scale * (f.y * s);
        }
        store8<TYPE>(p.X, (long long)row * p.ldx + k, cnt, v);
    }
}

template <int TYPE, bool NV>
cudaError_t launch(const Mx4Args &p, bool back, int tile_rows, int *err, cudaStream_t s)
{
    const int chunks = (p.K + TILE_COLS - 1) / TILE_COLS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)tile_rows * STRIPS * chunks));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = p.groups.offsets ? sizeof(int) * (2 * (p.groups.G + 1) + THREADS / 32) : 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return back ? cudaLaunchKernelEx(&cfg, dequantize_kernel<TYPE, NV>, p, chunks, err)
                : cudaLaunchKernelEx(&cfg, quantize_kernel<TYPE, NV>, p, chunks, err);
}

}  // namespace

cudaError_t launch_mx4(const Mx4Args &p, bool back, int tile_rows, int *err, cudaStream_t s)
{
    const bool nv = p.format == 1;
    if (p.type == 0)
        return nv ? launch<0, true>(p, back, tile_rows, err, s) : launch<0, false>(p, back, tile_rows, err, s);
    if (p.type == 1)
        return nv ? launch<1, true>(p, back, tile_rows, err, s) : launch<1, false>(p, back, tile_rows, err, s);
    return nv ? launch<2, true>(p, back, tile_rows, err, s) : launch<2, false>(p, back, tile_rows, err, s);
}

}  // namespace swg
