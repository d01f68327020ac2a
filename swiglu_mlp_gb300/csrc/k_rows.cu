// k_rows.cu — rows to their experts and back: dispatch, the weighted sum of a
// token's rows, and that sum's gradients.
//
// All of them stream rows in 16-byte pieces and are bound by memory.  They go by
// tokens, not by rows: what belongs to the token (its row, its sum) is read or written
// once and stays in registers while its slots pass by.  The sum's gradient has a product
// for each slot as well, and reads its row again for every four slots, out of the caches.
// Sums are in FP32, in the order of the slots.
//
// 8192 tokens of 4096 bfloat16 columns to two experts each: dispatch 31.3 us, 6.4 TB/s, 0.95
// of a copy; the sum 41 us, 4.9 TB/s, its gradient 59, 5.7.  To eight each: 94, 91 and 171 us,
// 6.4, 6.6 and 6.7 TB/s.  5003 tokens of 2051 binary16 columns, four experts each: the sum
// 23.0 us and its gradient 31.8, 4.5 and 5.8 TB/s (rows of 4112 bytes begin anywhere in a line).
// The reads that a sum waits for are all that its warp has in flight, which shows with few
// slots; spans handed out to resident warps, with the next positions asked for ahead, were no
// faster.  32 tokens of 4096, eight experts each: 2.7 us, one launch.
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

// `cnt` columns (0 .. PIECE) of a row as they are stored.  `roomy`: of a row that another
// one follows, whose pitch has all 16 bytes; the columns behind `cnt` are then whatever
// lies there (one load, that nothing waits for: 5003 tokens of 1003 binary16 columns, four
// experts, sum 18.6 -> 14.6 us, gradient 26.9 -> 18.4).  Of a tensor's last row they are
// zero and not read.
template <int TYPE>
__device__ __forceinline__ uint4 load_piece(const void *x, long long i, int cnt, bool roomy)
{
    const typename Elem<TYPE>::T *src = static_cast<const typename Elem<TYPE>::T *>(x) + i;
    if (cnt == PIECE<TYPE> || (roomy && cnt > 0)) return *reinterpret_cast<const uint4 *>(src);
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

// Zeros behind the first `cnt` columns.
template <int TYPE>
__device__ __forceinline__ void clear_behind(uint4 &w, int cnt)
{
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (TYPE == 2)
            u[j] = j < cnt ? u[j] : 0u;
        else
            u[j] = 2 * j + 1 < cnt ? u[j] : 2 * j < cnt ? u[j] & 0xffffu : 0u;
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
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

// A warp has a span of a token's pieces: the token, and its first and last column.
// Spans are `per` pieces, the last one of a token what is left.
template <int TYPE>
__device__ __forceinline__ bool find_span(const RowsArgs &p, int spans, int per, int &t, int &from, int &to)
{
    const long long unit = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
    t = (int)(unit / spans);
    const int i = (int)(unit - (long long)t * spans);
    from = i * per * PIECE<TYPE>;
    to = i == spans - 1 ? p.D : from + per * PIECE<TYPE>;
    return t < p.T;
}

// Columns of a piece that begins at col, of those before `to`.
template <int TYPE>
__device__ __forceinline__ int columns(int to, long long col)
{
    return (int)min(max(to - col, 0ll), (long long)PIECE<TYPE>);
}

template <int TYPE, int U>
__global__ void __launch_bounds__(32 * WARPS) dispatch_kernel(const RowsArgs p, int spans, int per, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int t, from, to;
    if (!find_span<TYPE>(p, spans, per, t, from, to)) return;
    const int at = slot_row(p, t, err);
    for (long long col = from + (threadIdx.x & 31) * PIECE<TYPE>; __any_sync(ALL, col < to); col += U * 32 * PIECE<TYPE>) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long c = col + u * 32 * PIECE<TYPE>;
            x[u] = load_piece<TYPE>(p.X, t * p.ldx + c, columns<TYPE>(to, c), t + 1 < p.T);
        }
        for (int j = 0; j < p.top; ++j) {
            const int r = __shfl_sync(ALL, at, j);
            if (r < 0) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long c = col + u * 32 * PIECE<TYPE>;
                store_piece<TYPE>(p.rows, r * p.ldr + c, columns<TYPE>(to, c), x[u]);
            }
        }
    }
}

// Columns from col on in the type of the sum: as many as a piece of a row has.
template <int TYPE, int OUT>
__device__ __forceinline__ void store_sum(void *out, long long i, int cnt, const float (&v)[PIECE<TYPE>])
{
    if constexpr (TYPE == OUT) {
        store_piece<OUT>(out, i, cnt, from_floats<OUT>(v));
    } else {                                         // four FP32 columns to 16 bits
        static_assert(TYPE == 2, "only sums of FP32 rows change their type");
        typename Elem<OUT>::T *dst = static_cast<typename Elem<OUT>::T *>(out) + i;
        if (cnt == 4) {
            constexpr int kind = OUT == 1 ? OUT_BF16 : OUT_F16;
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2(v[0], v[1], kind), pack2(v[2], v[3], kind));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < cnt) dst[j] = (typename Elem<OUT>::T)v[j];
        }
    }
}

template <int TYPE, int OUT, int U>
__global__ void __launch_bounds__(32 * WARPS, 4) combine_kernel(const RowsArgs p, int spans, int per, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int t, from, to;
    if (!find_span<TYPE>(p, spans, per, t, from, to)) return;
    const int lane = threadIdx.x & 31;
    const int at = slot_row(p, t, err);
    const float w = p.weights != nullptr && lane < p.top ? p.weights[(long long)t * p.top + lane] : 1.0f;
    for (long long col = from + lane * PIECE<TYPE>; __any_sync(ALL, col < to); col += U * 32 * PIECE<TYPE>) {
        int cnt[U];
#pragma unroll
        for (int u = 0; u < U; ++u) cnt[u] = columns<TYPE>(to, col + u * 32 * PIECE<TYPE>);
        float sum[U][PIECE<TYPE>] = {};
        for (int j = 0; j < p.top; j += BATCH) {
            uint4 x[BATCH][U];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int r = __shfl_sync(ALL, at, (j + b) & 31);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (j + b < p.top && r >= 0)
                        x[b][u] = load_piece<TYPE>(p.rows, r * p.ldr + col + u * 32 * PIECE<TYPE>, cnt[u], r + 1 < p.R);
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
            if (cnt[u] == 0) continue;
            const long long o = t * p.ldo + col + u * 32 * PIECE<TYPE>;
            if (p.beta != 0.0f) {
                const typename Elem<OUT>::T *old = static_cast<const typename Elem<OUT>::T *>(p.out) + o;
#pragma unroll
                for (int i = 0; i < PIECE<TYPE>; ++i)
                    if (i < cnt[u]) sum[u][i] = fmaf(p.beta, (float)old[i], sum[u][i]);
            }
            store_sum<TYPE, OUT>(p.out, o, cnt[u], sum[u]);
        }
    }
}

// A CTA per token, its warps side by side along the row, a piece per lane and round.
template <int TYPE>
__global__ void __launch_bounds__(256) combine_grad_kernel(const RowsArgs p, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float part[MAX_TOP][8];               // each warp's part of the products with d_out
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int t = blockIdx.x, at = slot_row(p, t, err);
    const float w = p.weights != nullptr && lane < p.top ? p.weights[(long long)t * p.top + lane] : 1.0f;
    const bool products = p.d_weights != nullptr;
    const int step = warps * 32 * PIECE<TYPE>;
    float mine = 0.0f;                               // lane j: slot j's product
    for (int j = 0; j < p.top; j += BATCH) {
        float dot[BATCH] = {};
        for (long long col = (warp * 32 + lane) * PIECE<TYPE>; __any_sync(ALL, col < p.D); col += step) {
            const int cnt = columns<TYPE>(p.D, col);
            uint4 d = load_piece<TYPE>(p.X, t * p.ldx + col, cnt, t + 1 < p.T), x[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int r = __shfl_sync(ALL, at, (j + b) & 31);
                if (products && j + b < p.top && r >= 0) x[b] = load_piece<TYPE>(p.rows, r * p.ldr + col, cnt, r + 1 < p.R);
            }
            if (__any_sync(ALL, cnt % PIECE<TYPE> != 0)) {           // (the end of a row)
                clear_behind<TYPE>(d, cnt);
#pragma unroll
                for (int b = 0; b < BATCH; ++b) clear_behind<TYPE>(x[b], cnt);
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int r = __shfl_sync(ALL, at, (j + b) & 31);
                const float f = __shfl_sync(ALL, w, (j + b) & 31);
                if (j + b >= p.top || r < 0) continue;
                float dv[PIECE<TYPE>], v[PIECE<TYPE>];
                to_floats<TYPE>(d, dv);
                if (products) {
                    to_floats<TYPE>(x[b], v);
#pragma unroll
                    for (int i = 0; i < PIECE<TYPE>; ++i) dot[b] = fmaf(dv[i], v[i], dot[b]);
                }
#pragma unroll
                for (int i = 0; i < PIECE<TYPE>; ++i) v[i] = f * dv[i];
                store_piece<TYPE>(p.out, r * p.ldo + col, cnt, from_floats<TYPE>(v));
            }
        }
        if (!products) continue;
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) dot[b] += __shfl_xor_sync(ALL, dot[b], s);
            if (lane == j + b) mine = dot[b];
        }
    }
    if (!products) return;
    if (warps > 1) {
        if (lane < p.top) part[lane][warp] = mine;
        __syncthreads();
        if (warp > 0) return;
        mine = 0.0f;
        if (lane < p.top)
            for (int i = 0; i < warps; ++i) mine += part[lane][i];
    }
    if (lane < p.top) p.d_weights[(long long)t * p.top + lane] = mine;
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

long long ceil_div(long long n, long long per) { return (n + per - 1) / per; }

// Spans that a token's row is cut into, of 32 `lane` pieces: as many as give the SMs
// several waves of warps; of a row's remainder only more than a quarter is its own.
struct Spans {
    int count, per;
    long long ctas;
};
template <int TYPE>
Spans spans_of(const RowsArgs &p, int lane)
{
    const int per = 32 * lane;
    const long long pieces = ceil_div(p.D, PIECE<TYPE>);
    const int count = (int)std::max((pieces + per - 1 - per / 4) / per, 1ll);
    return {count, per, ceil_div((long long)p.T * count, WARPS)};
}

template <int TYPE>
cudaError_t dispatch(const RowsArgs &p, int sms, int *err, cudaStream_t s)
{
    // Four pieces per lane, unless that leaves SMs without work.
    Spans of = spans_of<TYPE>(p, 4);
    if (of.ctas >= 4ll * sms) return go(dispatch_kernel<TYPE, 4>, of.ctas, 32 * WARPS, s, p, of.count, of.per, err);
    of = spans_of<TYPE>(p, 1);
    return go(dispatch_kernel<TYPE, 1>, of.ctas, 32 * WARPS, s, p, of.count, of.per, err);
}

template <int TYPE, int OUT>
cudaError_t combine(const RowsArgs &p, int sms, int *err, cudaStream_t s)
{
    Spans of = spans_of<TYPE>(p, 2);
    if (of.ctas >= 4ll * sms) return go(combine_kernel<TYPE, OUT, 2>, of.ctas, 32 * WARPS, s, p, of.count, of.per, err);
    of = spans_of<TYPE>(p, 1);
    return go(combine_kernel<TYPE, OUT, 1>, of.ctas, 32 * WARPS, s, p, of.count, of.per, err);
}

template <int TYPE>
cudaError_t combine_grad(const RowsArgs &p, int *err, cudaStream_t s)
{
    // The warps that leave the fewest lanes without a piece, the most of equals.
    const long long pieces = ceil_div(p.D, PIECE<TYPE>);
    int warps = 1;
    long long least = ceil_div(pieces, 32);
    for (int w = 2; w <= 8; ++w) {
        const long long rounds = w * ceil_div(pieces, 32ll * w);
        if (rounds <= least) {
            least = rounds;
            warps = w;
        }
    }
    return go(combine_grad_kernel<TYPE>, p.T, 32 * warps, s, p, err);
}

}  // namespace

cudaError_t launch_dispatch(const RowsArgs &p, int sms, int *err, cudaStream_t s)
{
    return p.type == 2 ? dispatch<2>(p, sms, err, s) : p.type == 1 ? dispatch<1>(p, sms, err, s) : dispatch<0>(p, sms, err, s);
}

cudaError_t launch_combine(const RowsArgs &p, int sms, int *err, cudaStream_t s)
{
    if (p.type != 2) return p.type == 1 ? combine<1, 1>(p, sms, err, s) : combine<0, 0>(p, sms, err, s);
    return p.out_type == 2   ? combine<2, 2>(p, sms, err, s)
           : p.out_type == 1 ? combine<2, 1>(p, sms, err, s)
                             : combine<2, 0>(p, sms, err, s);
}

cudaError_t launch_combine_grad(const RowsArgs &p, int *err, cudaStream_t s)
{
    return p.type == 2 ? combine_grad<2>(p, err, s) : p.type == 1 ? combine_grad<1>(p, err, s) : combine_grad<0>(p, err, s);
}

}  // namespace swg
