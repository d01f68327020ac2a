// k_rows.cu — rows to their experts and back: dispatch, the weighted sum of a
// token's rows, and that sum's gradients.
//
// All of them stream rows in 16-byte pieces and are bound by memory.  They go by
// tokens, not by rows: what belongs to the token (its row, its sum, its gradient)
// is read or written once and stays in registers while its slots pass by.  Sums
// are in FP32, in the order of the slots.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "groups.cuh"
#include "launch.h"
#include "routing.h"

namespace swg {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int WARPS = 8;             // per CTA of dispatch and combine
constexpr int BATCH = 4;             // slots whose loads are in flight together

template <int TYPE> struct Elem;
template <> struct Elem<0> { using T = __half; };
template <> struct Elem<1> { using T = __nv_bfloat16; };
template <> struct Elem<2> { using T = float; };

template <int TYPE> constexpr int PIECE = TYPE == 2 ? 4 : 8;      // columns in 16 bytes

// `cnt` columns (0 .. PIECE) of a row as they are stored; the others are zero
// and not read.
template <int TYPE>
__device__ __forceinline__ uint4 load_piece(const void *x, long long i, int cnt)
{
    const typename Elem<TYPE>::T *src = static_cast<const typename Elem<TYPE>::T *>(x) + i;
    if (cnt == PIECE<TYPE>) return *reinterpret_cast<const uint4 *>(src);
    uint32_t u[4] = {};
#pragma unroll
    for (int j = 0; j < PIECE<TYPE>; ++j) {
        if (j >= cnt) continue;
        if (TYPE == 2)
            u[j % 4] = reinterpret_cast<const uint32_t *>(src)[j];
        else
            u[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(src)[j] << (16 * (j & 1));
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <int TYPE>
__device__ __forceinline__ void store_piece(void *x, long long i, int cnt, uint4 w)
{
    typename Elem<TYPE>::T *dst = static_cast<typename Elem<TYPE>::T *>(x) + i;
    if (cnt == PIECE<TYPE>) {
        *reinterpret_cast<uint4 *>(dst) = w;
        return;
    }
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < PIECE<TYPE>; ++j) {
        if (j >= cnt) continue;
        if (TYPE == 2)
            reinterpret_cast<uint32_t *>(dst)[j] = u[j % 4];
        else
            reinterpret_cast<uint16_t *>(dst)[j] = (uint16_t)(u[j / 2] >> (16 * (j & 1)));
    }
}

template <int TYPE>
__device__ __forceinline__ void to_floats(uint4 w, float (&v)[PIECE<TYPE>])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (TYPE == 2) {
            v[j % PIECE<TYPE>] = __uint_as_float(u[j]);
        } else {
            const float2 f = TYPE == 1 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[j]))
                                       : __half22float2(*reinterpret_cast<const __half2 *>(&u[j]));
            v[2 * j % PIECE<TYPE>] = f.x;
            v[(2 * j + 1) % PIECE<TYPE>] = f.y;
        }
    }
}

template <int TYPE>
__device__ __forceinline__ uint4 from_floats(const float (&v)[PIECE<TYPE>])
{
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (TYPE == 2) {
            u[j] = __float_as_uint(v[j % PIECE<TYPE>]);
        } else if (TYPE == 1) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j % PIECE<TYPE>], v[(2 * j + 1) % PIECE<TYPE>]);
            u[j] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(v[2 * j % PIECE<TYPE>], v[(2 * j + 1) % PIECE<TYPE>]);
            u[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Lane j's slot of token t: its row, or -1 (a position that does not exist is
// reported).
__device__ __forceinline__ int slot_row(const RowsArgs &p, int t, int *err)
{
    const int lane = threadIdx.x & 31;
    int at = lane < p.top ? p.position[(long long)t * p.top + lane] : -1;
    if (at < -1 || at >= p.R) {
        atomicCAS(err, 0, ERR_INVALID);
        at = -1;
    }
    return at;
}

// The token and the first column of this warp's unit: `pieces` pieces per lane.
template <int TYPE, int U>
__device__ __forceinline__ bool find_unit(const RowsArgs &p, int chunks, int &t, int &col)
{
    const long long unit = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
    t = (int)(unit / chunks);
    col = ((int)(unit - (long long)t * chunks) * 32 * U + (int)(threadIdx.x & 31)) * PIECE<TYPE>;
    return t < p.T;
}

template <int TYPE>
__device__ __forceinline__ int columns(int D, int col)
{
    return min(max(D - col, 0), PIECE<TYPE>);
}

template <int TYPE, int U>
__global__ void __launch_bounds__(32 * WARPS) dispatch_kernel(const RowsArgs p, int chunks, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int t, col;
    if (!find_unit<TYPE, U>(p, chunks, t, col)) return;
    const int at = slot_row(p, t, err);
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = col + u * 32 * PIECE<TYPE>;
        x[u] = load_piece<TYPE>(p.X, t * p.ldx + c, columns<TYPE>(p.D, c));
    }
    for (int j = 0; j < p.top; ++j) {
        const int r = __shfl_sync(ALL, at, j);
        if (r < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = col + u * 32 * PIECE<TYPE>;
            store_piece<TYPE>(p.rows, r * p.ldr + c, columns<TYPE>(p.D, c), x[u]);
        }
    }
}

template <int TYPE, int U>
__global__ void __launch_bounds__(32 * WARPS) combine_kernel(const RowsArgs p, int chunks, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int t, col;
    if (!find_unit<TYPE, U>(p, chunks, t, col)) return;
    const int lane = threadIdx.x & 31;
    const int at = slot_row(p, t, err);
    const float w = p.weights != nullptr && lane < p.top ? p.weights[(long long)t * p.top + lane] : 1.0f;
    int cnt[U];
#pragma unroll
    for (int u = 0; u < U; ++u) cnt[u] = columns<TYPE>(p.D, col + u * 32 * PIECE<TYPE>);
    float sum[U][PIECE<TYPE>] = {};
    for (int j = 0; j < p.top; j += BATCH) {
        uint4 x[BATCH][U];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int r = __shfl_sync(ALL, at, (j + b) & 31);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j + b < p.top && r >= 0)
                    x[b][u] = load_piece<TYPE>(p.rows, r * p.ldr + col + u * 32 * PIECE<TYPE>, cnt[u]);
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int r = __shfl_sync(ALL, at, (j + b) & 31);
            const float f = __shfl_sync(ALL, w, (j + b) & 31);
            if (j + b >= p.top || r < 0) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[PIECE<TYPE>];
                to_floats<TYPE>(x[b][u], v);
#pragma unroll
                for (int i = 0; i < PIECE<TYPE>; ++i) sum[u][i] = fmaf(f, v[i], sum[u][i]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long o = t * p.ldo + col + u * 32 * PIECE<TYPE>;
        if (cnt[u] == 0) continue;
        if (p.beta != 0.0f) {
            const typename Elem<TYPE>::T *old = static_cast<const typename Elem<TYPE>::T *>(p.out) + o;
#pragma unroll
            for (int i = 0; i < PIECE<TYPE>; ++i)
                if (i < cnt[u]) sum[u][i] = fmaf(p.beta, (float)old[i], sum[u][i]);
        }
        store_piece<TYPE>(p.out, o, cnt[u], from_floats<TYPE>(sum[u]));
    }
}

// A CTA per token, U pieces of its row per thread and round.
template <int TYPE, int U>
__global__ void __launch_bounds__(256) combine_grad_kernel(const RowsArgs p, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float part[MAX_TOP][8];               // each warp's part of the products with d_out
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int at = slot_row(p, t, err);
    const float w = p.weights != nullptr && lane < p.top ? p.weights[(long long)t * p.top + lane] : 1.0f;
    const bool products = p.d_weights != nullptr;
    const int step = blockDim.x * PIECE<TYPE>;
    long long first = 0;
    do {                                             // (once for no columns: the products are 0)
        uint4 d[U];
        int cnt[U];
        const int col = (int)first + threadIdx.x * PIECE<TYPE>;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            cnt[u] = columns<TYPE>(p.D, col + u * step);
            d[u] = load_piece<TYPE>(p.X, t * p.ldx + col + u * step, cnt[u]);
        }
        for (int j = 0; j < p.top; j += BATCH) {
            uint4 x[BATCH][U];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int r = __shfl_sync(ALL, at, (j + b) & 31);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (products && j + b < p.top && r >= 0)
                        x[b][u] = load_piece<TYPE>(p.rows, r * p.ldr + col + u * step, cnt[u]);
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int r = __shfl_sync(ALL, at, (j + b) & 31);
                const float f = __shfl_sync(ALL, w, (j + b) & 31);
                if (j + b >= p.top) continue;
                float dot = 0.0f;
                if (r >= 0) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float dv[PIECE<TYPE>], v[PIECE<TYPE>];
                        to_floats<TYPE>(d[u], dv);
                        if (products) {
                            to_floats<TYPE>(x[b][u], v);
#pragma unroll
                            for (int i = 0; i < PIECE<TYPE>; ++i) dot = fmaf(dv[i], v[i], dot);
                        }
#pragma unroll
                        for (int i = 0; i < PIECE<TYPE>; ++i) v[i] = f * dv[i];
                        store_piece<TYPE>(p.out, r * p.ldo + col + u * step, cnt[u], from_floats<TYPE>(v));
                    }
                }
                if (!products) continue;
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(ALL, dot, s);
                if (lane == 0) part[j + b][warp] = first == 0 ? dot : part[j + b][warp] + dot;
            }
        }
        first += U * step;
    } while (first < p.D);
    if (!products) return;
    __syncthreads();
    if (threadIdx.x < p.top) {
        float sum = 0.0f;
        for (int i = 0; i < (int)blockDim.x / 32; ++i) sum += part[threadIdx.x][i];
        p.d_weights[(long long)t * p.top + threadIdx.x] = sum;
    }
}

template <class K, class... A>
cudaError_t go(K kernel, long long ctas, int threads, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int ceil_to_units(int n, int per) { return (n + per - 1) / per; }

template <int TYPE>
cudaError_t dispatch(const RowsArgs &p, int sms, int *err, cudaStream_t s)
{
    // Four pieces per lane, unless that leaves SMs without work.
    const int wide = ceil_to_units(p.D, 32 * 4 * PIECE<TYPE>), narrow = ceil_to_units(p.D, 32 * PIECE<TYPE>);
    if ((long long)p.T * wide >= 4ll * WARPS * sms)
        return go(dispatch_kernel<TYPE, 4>, ((long long)p.T * wide + WARPS - 1) / WARPS, 32 * WARPS, s, p, wide, err);
    return go(dispatch_kernel<TYPE, 1>, ((long long)p.T * narrow + WARPS - 1) / WARPS, 32 * WARPS, s, p, narrow, err);
}

template <int TYPE>
cudaError_t combine(const RowsArgs &p, int sms, int *err, cudaStream_t s)
{
    const int wide = ceil_to_units(p.D, 32 * 2 * PIECE<TYPE>), narrow = ceil_to_units(p.D, 32 * PIECE<TYPE>);
    if ((long long)p.T * wide >= 4ll * WARPS * sms)
        return go(combine_kernel<TYPE, 2>, ((long long)p.T * wide + WARPS - 1) / WARPS, 32 * WARPS, s, p, wide, err);
    return go(combine_kernel<TYPE, 1>, ((long long)p.T * narrow + WARPS - 1) / WARPS, 32 * WARPS, s, p, narrow, err);
}

template <int TYPE>
cudaError_t combine_grad(const RowsArgs &p, int *err, cudaStream_t s)
{
    const int warps = std::max(std::min(ceil_to_units(p.D, 32 * 2 * PIECE<TYPE>), 8), 1);
    return go(combine_grad_kernel<TYPE, 2>, p.T, 32 * warps, s, p, err);
}

}  // namespace

cudaError_t launch_dispatch(const RowsArgs &p, int sms, int *err, cudaStream_t s)
{
    return p.type == 2 ? dispatch<2>(p, sms, err, s) : p.type == 1 ? dispatch<1>(p, sms, err, s) : dispatch<0>(p, sms, err, s);
}

cudaError_t launch_combine(const RowsArgs &p, int sms, int *err, cudaStream_t s)
{
    return p.type == 2 ? combine<2>(p, sms, err, s) : p.type == 1 ? combine<1>(p, sms, err, s) : combine<0>(p, sms, err, s);
}

cudaError_t launch_combine_grad(const RowsArgs &p, int *err, cudaStream_t s)
{
    return p.type == 2 ? combine_grad<2>(p, err, s) : p.type == 1 ? combine_grad<1>(p, err, s) : combine_grad<0>(p, err, s);
}

}  // namespace swg
