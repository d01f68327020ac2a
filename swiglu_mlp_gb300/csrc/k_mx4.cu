// k_mx4.cu — microscaled 4-bit floating point: to 4 bits and back.
//
// Both directions stream: 2 bytes (16-bit x) and 1/2 + 1/32 or 1/16 bytes per
// element, each once; at 7 or 8 TB/s that leaves about 14 instructions per
// element and lane, so the arithmetic is kept short too.  To 4 bits a lane has 16
// columns (a block of NVFP4, half a block of MXFP4) of four rows r, r + 32, r + 64,
// r + 96 of a row of scale tiles, whose scales lie side by side in memory; a
// warp has 512 columns.  Lanes swap their blocks' scale bytes so that each
// stores 4 bytes of a tile.
//
// Measured, to 4 bits from bf16: 57344 x 4096 in 96 us (MXFP4) and 100 us
// (NVFP4), 6.2 and 6.0 TB/s of traffic; 8192 x 4096 in 13.7 and 15.3 us; 1024 x
// 4096 in 4.0 and 4.5 us; 1 x 4096 in 2.2 us, a launch.  Back to bf16: 14336 x
// 4096 in 24 us, 6.2 TB/s, most of it written (a plain fill of the result takes
// 30).  256 groups of 8 rows, K = 2048: 7 us each way.
#include <algorithm>

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
constexpr int LANE_COLS = 16;        // columns per lane
constexpr int TILE_COLS = 512;       // columns per CTA: 4 (MXFP4) or 8 (NVFP4) scale tiles
constexpr int TILE_COLS_BACK = 256;  // ... of the way back, 8 per lane
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

// The largest magnitude of 8 stored values, NaN if one is NaN: of 16-bit
// values two at a time.
template <int TYPE>
__device__ __forceinline__ float top8(const Raw8<TYPE> &r)
{
    if (TYPE == 2) {
        float top = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u[4] = {r.w[h % (TYPE == 2 ? 2 : 1)].x, r.w[h % (TYPE == 2 ? 2 : 1)].y,
                                   r.w[h % (TYPE == 2 ? 2 : 1)].z, r.w[h % (TYPE == 2 ? 2 : 1)].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max_nan(top, fabsf(__uint_as_float(u[j])));
        }
        return top;
    }
    uint32_t m[4] = {r.w[0].x & 0x7fff7fffu, r.w[0].y & 0x7fff7fffu, r.w[0].z & 0x7fff7fffu,
                     r.w[0].w & 0x7fff7fffu};
    if (TYPE == 1) {
        auto h = [](uint32_t a) { return *reinterpret_cast<const __nv_bfloat162 *>(&a); };
        const float2 f = __bfloat1622float2(
            __hmax2_nan(__hmax2_nan(h(m[0]), h(m[1])), __hmax2_nan(h(m[2]), h(m[3]))));
        return max_nan(f.x, f.y);
    }
    auto h = [](uint32_t a) { return *reinterpret_cast<const __half2 *>(&a); };
    const float2 f = __half22float2(
        __hmax2_nan(__hmax2_nan(h(m[0]), h(m[1])), __hmax2_nan(h(m[2]), h(m[3]))));
    return max_nan(f.x, f.y);
}

// x / d from an approximation of 1 / d, with one residual correction
// (Markstein's): a quotient that is itself a float comes out exact.
__device__ __forceinline__ float quotient(float x, float d, float inverse)
{
    const float q = x * inverse;
    return __fmaf_rn(__fmaf_rn(-q, d, x), inverse, q);
}

// The scale of a block whose largest magnitude is `top` (NaN if the block has
// one): its byte; `scale` its value and `inverse` about 1 / scale (exactly for
// MXFP4), both NaN for a block with a NaN or an infinity.
template <bool NV>
__device__ __forceinline__ uint32_t block_scale(float top, float &scale, float &inverse)
{
    const uint32_t bits = __float_as_uint(top);
    const float nan = __uint_as_float(0x7fffffffu);
    if (NV) {
        // to nearest even by the conversion, which saturates at 448
        const uint32_t code = max((uint32_t)__nv_cvt_float_to_fp8(quotient(top, 6.0f, 1.0f / 6.0f),
                                                                  __NV_SATFINITE, __NV_E4M3),
                                  1u);
        const bool bad = bits >= 0x7f800000u;
        scale = bad ? nan
                    : __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
        inverse = __fdividef(1.0f, scale);
        return bad ? 0x7fu : code;
    }
    const uint32_t e = bits >> 23;                   // floor(log2 top) + 127
    const uint32_t code = e > 2 ? e - 2 : 0;
    const bool bad = e >= 255;
    scale = bad ? nan : __uint_as_float(code > 0 ? code << 23 : 1u << 22);
    inverse = bad ? nan : __uint_as_float((254u - code) << 23);       // 2^(127 - code)
    return bad ? 0xffu : code;
}

// The value of a scale byte: E8M0 (0xFF is NaN), or E4M3.
__device__ __forceinline__ float scale_value(bool nv, uint32_t c)
{
    if (nv) return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
    return c == 255u ? __int_as_float(0x7fffffff)
                     : __int_as_float(c > 0 ? c << 23 : 1 << 22);
}

struct Place {
    int t;                   // row of scale tiles
    int chunk;               // of columns
    int r;                   // this warp's first row in them; the others are 32 apart, or next to it
    int row0, end;           // first row of the tiles, end of their group
};

// The unit'th row of scale tiles (PER = 128) or four rows of one (PER = 4); false
// beyond the last group's.  Every warp walks the groups itself, 32 at a time or,
// where there may be hundreds, 128, whose offsets it loads together: a table
// for the CTA would cost it two barriers, and it has little to do.  (Offsets are
// clamped as in group_starts.)
template <int PER>
__device__ __forceinline__ bool find_rows(const Groups &gr, int unit, int *err, Place &p)
{
    const int lane = threadIdx.x & 31;
    auto found = [&](int lo, int hi, int tiles, int i) {             // unit i of rows lo .. hi - 1
        const int tile = i * PER / TILE_ROWS;
        p.t = tiles + tile;
        p.r = i * PER % TILE_ROWS;
        p.row0 = lo + tile * TILE_ROWS;
        p.end = hi;
    };
    if (gr.offsets == nullptr) {
        found(0, gr.M, 0, unit);
        return p.row0 + p.r < gr.M;
    }
    constexpr int BATCH = PER == TILE_ROWS ? 1 : 4;
    int top = 0, before = 0, tiles = 0;              // largest offset, units and tiles so far
    bool bad = false;
    for (int base = 0; base < gr.G; base += 32 * BATCH) {
        int v[BATCH + 1];                            // the last: what follows them
#pragma unroll
        for (int r = 0; r <= BATCH; ++r) {
            const int raw = gr.offsets[min(base + 32 * r + (r < BATCH ? lane : 0), gr.G)];
            v[r] = raw < 0 ? 0 : raw > gr.M ? gr.M : raw;
            bad = bad || v[r] != raw;
        }
#pragma unroll
        for (int r = 0; r < BATCH; ++r) {
            if (base + 32 * r >= gr.G) break;
            const int next = __shfl_down_sync(0xffffffffu, v[r], 1);
            const int wrap = __shfl_sync(0xffffffffu, v[r + 1], 0);
            int lo = max(v[r], top), hi = lane < 31 ? next : wrap;
            bad = bad || hi < lo;
            hi = max(hi, lo);
            if (__any_sync(0xffffffffu, bad)) {      // running maxima, the slow way
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, hi, d);
                    if (lane >= d) hi = max(hi, o);
                }
                const int o = __shfl_up_sync(0xffffffffu, hi, 1);
                if (lane > 0) lo = max(lo, o);
                if (lane == 0) atomicCAS(err, 0, ERR_INVALID);
            }
            const int here = base + 32 * r + lane < gr.G ? hi - lo : 0;
            const int n = ceil_div(here, PER), own = ceil_div(here, TILE_ROWS);
            const int all = __reduce_add_sync(0xffffffffu, n);
            if (unit < before + all) {
                int sum = n, own_sum = own;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, sum, d);
                    if (lane >= d) sum += o;
                    if (PER < TILE_ROWS) {
                        const int q = __shfl_up_sync(0xffffffffu, own_sum, d);
                        if (lane >= d) own_sum += q;
                    }
                }
                if (PER == TILE_ROWS) own_sum = sum;
                const int first = before + sum - n;
                const int src = __ffs(__ballot_sync(0xffffffffu, unit >= first && unit < first + n)) - 1;
                found(__shfl_sync(0xffffffffu, lo, src), __shfl_sync(0xffffffffu, hi, src),
                      tiles + __shfl_sync(0xffffffffu, own_sum - own, src),
                      unit - __shfl_sync(0xffffffffu, first, src));
                return true;
            }
            before += all;
            tiles += PER == TILE_ROWS ? all : __reduce_add_sync(0xffffffffu, own);
            top = __shfl_sync(0xffffffffu, hi, 31);
        }
    }
    return false;
}

// This warp's place; false beyond the last group's rows.  FEW = false: a CTA has
// eight neighbouring rows of each 32, of one chunk, whose scales lie side by
// side.  FEW: a warp has four neighbouring rows of a group, and the last of a
// tile's writes the scales, zeros, of the rows that do not exist.  In the other
// form a group of few rows has the warps of a whole tile, nearly all of which
// do only that.
template <bool FEW>
__device__ __forceinline__ bool find_place(const Groups &gr, int chunks, int *err, Place &p)
{
    const unsigned warp = threadIdx.x >> 5;
    if (FEW) {
        const unsigned unit = blockIdx.x * (THREADS / 32) + warp, rows = unit / (unsigned)chunks;
        p.chunk = (int)(unit - rows * (unsigned)chunks);
        return find_rows<ROWS>(gr, (int)rows, err, p);
    }
    const unsigned strip = blockIdx.x / (unsigned)chunks;
    p.chunk = (int)(blockIdx.x - strip * (unsigned)chunks);
    const bool is = find_rows<TILE_ROWS>(gr, (int)(strip / STRIPS), err, p);
    p.r = (int)(strip % STRIPS * 8 + warp);
    return is;
}

template <int TYPE, bool NV, bool FEW>
__global__ void __launch_bounds__(THREADS) quantize_kernel(const Mx4Args p, int chunks, int *err)
{
    constexpr int LANES = NV ? 1 : 2;                // lanes per block
    constexpr int TILES = NV ? 8 : 4;                // scale tiles per chunk along K
    constexpr int APART = FEW ? 1 : 32;              // a warp's four rows
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Place at;
    if (!find_place<FEW>(p.groups, chunks, err, at)) return;
    const int lane = threadIdx.x & 31;
    const int k = at.chunk * TILE_COLS + lane * LANE_COLS;
    const int cnt = min(LANE_COLS, max(0, p.K - k));
    const int width = min(LANE_COLS, max(0, ((p.K + 31) & ~31) - k));  // codes to write
    const bool block = k - (lane % LANES) * LANE_COLS < p.K;           // the block has columns
    Raw8<TYPE> raw[ROWS][2];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = at.row0 + at.r + APART * i;
        const long long o = (long long)row * p.ldx + k;
        const int n = row < at.end ? cnt : 0;
        raw[i][0] = load8<TYPE>(p.X, o, min(n, 8));
        raw[i][1] = load8<TYPE>(p.X, o + 8, max(n - 8, 0));
    }
    uint32_t codes = 0;                              // the lane's block's scales, a byte per row
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = at.row0 + at.r + APART * i;
        // (the factor is positive: the largest of the products is its product)
        float top = p.scale * max_nan(top8<TYPE>(raw[i][0]), top8<TYPE>(raw[i][1]));
        if (!NV) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        float s, inv;
        const uint32_t code = block_scale<NV>(top, s, inv);
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            to_floats<TYPE>(raw[i][h], v);
            q[h] = 0;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float2 x = make_float2(p.scale * v[j], p.scale * v[j + 1]);
                if (NV) {
                    // A tie between two codes is a quotient that is a float, and x
                    // next to one has a quotient at least 8/15 of a float's unit
                    // from it (the scale has 4 bits), so that the corrected
                    // quotient rounds as the exact one does, for any FP32 x; the
                    // product with the inverse alone may miss ties.
                    const float2 inv2 = make_float2(inv, inv);
                    const float2 y = __fmul2_rn(x, inv2);
                    x = __ffma2_rn(__ffma2_rn(make_float2(-y.x, -y.y), make_float2(s, s), x), inv2, y);
                } else {
                    x = make_float2(x.x * inv, x.y * inv);
                }
                q[h] |= (uint32_t)__nv_cvt_float2_to_fp4x2(x, __NV_E2M1, cudaRoundNearest) << (4 * j);
            }
        }
        if (row < at.end) {
            uint8_t *out = p.Q + (long long)row * p.ldq + k / 2;
            if (width == 16)
                *reinterpret_cast<uint2 *>(out) = make_uint2(q[0], q[1]);
            if (block) codes |= code << (8 * i);
        }
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
    const int kt = at.chunk * TILES;
    uint8_t *scales = p.S + ((long long)at.t * tiles_k + kt) * 512;
    const int rows = at.end - at.row0, r = at.r + APART * b;
    if (lane % LANES == 0 && kt + tile < tiles_k && (!FEW || r < rows))
        *reinterpret_cast<uint32_t *>(scales + tile * 512 + 16 * (r % 32) + 4 * (r / 32)) = word;
    if (FEW && at.r + ROWS >= min(rows, TILE_ROWS)) {
        // The tile's last rows: those behind them do not exist, their scales are zero.
        for (int t = 0; t < TILES && kt + t < tiles_k; ++t) {
            uint32_t *of_lane = reinterpret_cast<uint32_t *>(scales + t * 512 + 16 * lane);
            if (lane >= rows) {
                *reinterpret_cast<uint4 *>(of_lane) = make_uint4(0, 0, 0, 0);
            } else {
#pragma unroll
                for (int i = 1; i < 4; ++i)
                    if (lane + 32 * i >= rows) of_lane[i] = 0;
            }
        }
    }
}

// Back: 8 columns per lane, so that a warp's stores of a row are whole lines
// (with 16, as above, two stores share each 32-byte sector: 33 instead of 24 us
// for 14336 x 4096 to bf16).
template <int TYPE, bool NV, bool FEW>
__global__ void __launch_bounds__(THREADS) dequantize_kernel(const Mx4Args p, int chunks, int *err)
{
    constexpr int LANES = NV ? 2 : 4;
    constexpr int TILES = NV ? 4 : 2;
    constexpr int APART = FEW ? 1 : 32;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Place at;
    if (!find_place<FEW>(p.groups, chunks, err, at)) return;
    const int lane = threadIdx.x & 31;
    const int k = at.chunk * TILE_COLS_BACK + lane * 8;
    const int cnt = min(8, max(0, p.K - k));
    if (cnt == 0) return;
    uint32_t q[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = at.row0 + at.r + APART * i;
        q[i] = row < at.end ? *reinterpret_cast<const uint32_t *>(p.Q + (long long)row * p.ldq + k / 2) : 0;
    }
    // 16 bytes: the four rows' scales of the tile's four blocks
    const int b = lane / LANES % 4, kt = at.chunk * TILES + lane / (4 * LANES);
    const uint8_t *scales = p.S + ((long long)at.t * ceil_div(p.K, NV ? 64 : 128) + kt) * 512;
    uint32_t words[ROWS];
    if (FEW) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            words[i] = *reinterpret_cast<const uint32_t *>(scales + 16 * ((at.r + i) % 32) + 4 * (at.r / 32));
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(scales + 16 * at.r);
        words[0] = w.x, words[1] = w.y, words[2] = w.z, words[3] = w.w;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = at.row0 + at.r + APART * i;
        if (row >= at.end) continue;
        const float s = scale_value(NV, (words[i] >> (8 * b)) & 0xffu);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 f = __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2(
                (__nv_fp4x2_storage_t)((q[i] >> (4 * j)) & 0xffu), __NV_E2M1)));
            v[j] = p.scale * (f.x * s);
            v[j + 1] = p.scale * (f.y * s);
        }
        store8<TYPE>(p.X, (long long)row * p.ldx + k, cnt, v);
    }
}

template <int TYPE, bool NV, bool FEW>
cudaError_t launch(const Mx4Args &p, bool back, int *err, cudaStream_t s)
{
    const int cols = back ? TILE_COLS_BACK : TILE_COLS, G = p.groups.G, M = p.groups.M;
    const int chunks = (p.K + cols - 1) / cols;
    // Upper bounds of the units over all groups, and with offsets one more, whose
    // warps find nothing: on the way they look at every offset, also at those
    // behind the last row, and report what they have to clamp.
    const int more = p.groups.offsets != nullptr;
    const long long units = FEW ? M / ROWS + std::min(G, M) + more
                                : (M / TILE_ROWS + std::min(G, M) + more) * 32ll;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((units * chunks + THREADS / 32 - 1) / (THREADS / 32)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return back ? cudaLaunchKernelEx(&cfg, dequantize_kernel<TYPE, NV, FEW>, p, chunks, err)
                : cudaLaunchKernelEx(&cfg, quantize_kernel<TYPE, NV, FEW>, p, chunks, err);
}

template <int TYPE, bool NV>
cudaError_t launch_form(const Mx4Args &p, bool back, int *err, cudaStream_t s)
{
    // FEW for groups of few rows on average, unless they are few themselves:
    // 256 groups of one row, K = 8192, 6.8 us against 112; 32 of 64, 9.4 against
    // 13.3; 32 of 96, 13.6 against 14.7 (K = 2048: 5.7 against 5.3); but 8 of 4,
    // K = 512, 3.3 against 2.7, for its longer way to a warp's rows.
    const int cols = back ? TILE_COLS_BACK : TILE_COLS, G = p.groups.G, M = p.groups.M;
    const long long tiles = (long long)(M / TILE_ROWS + std::min(G, M)) * ((p.K + cols - 1) / cols);
    const bool few = G > 1 && M / G <= 64 && tiles > 40;
    return few ? launch<TYPE, NV, true>(p, back, err, s) : launch<TYPE, NV, false>(p, back, err, s);
}

}  // namespace

cudaError_t launch_mx4(const Mx4Args &p, bool back, int *err, cudaStream_t s)
{
    const bool nv = p.format == 1;
    if (p.type == 0) return nv ? launch_form<0, true>(p, back, err, s) : launch_form<0, false>(p, back, err, s);
    if (p.type == 1) return nv ? launch_form<1, true>(p, back, err, s) : launch_form<1, false>(p, back, err, s);
    return nv ? launch_form<2, true>(p, back, err, s) : launch_form<2, false>(p, back, err, s);
}

}  // namespace swg
