// groups.cuh — the tables of row groups that the grouped kernels build in
// shared memory from the offsets on the device, with all threads of a CTA.
#pragma once

#include "experts.h"

namespace swg {

constexpr int ERR_INVALID = 1;       // == SWG_ERR_INVALID_ARG

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// start[0..G]: the offsets, clamped to be non-decreasing within [0, M], so
// that every row a kernel derives from them exists; offsets that had to be
// clamped are reported in the error word.  Called by all NT threads; ends
// with a barrier.
template <int NT>
__device__ __forceinline__ void group_starts(const Groups &gr, int *start, int *err)
{
    const int tid = threadIdx.x, G = gr.G;
    if (gr.offsets == nullptr) {         // one group of all rows
        if (tid == 0) {
            start[0] = 0;
            start[1] = gr.M;
        }
        __syncthreads();
        return;
    }
    bool bad = false;
    for (int i = tid; i <= G; i += NT) {
        const int raw = gr.offsets[i];
        const int v = raw < 0 ? 0 : raw > gr.M ? gr.M : raw;
        bad = bad || v != raw;
        start[i] = v;
    }
    __syncthreads();
    for (int i = tid; i < G; i += NT) bad = bad || start[i + 1] < start[i];
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            atomicCAS(err, 0, ERR_INVALID);
            for (int i = 0; i < G; ++i)
                if (start[i + 1] < start[i]) start[i + 1] = start[i];
        }
        __syncthreads();
    }
}

// first[0..G]: how many tiles the groups before g have, a group of `rows`
// rows having tiles_of(rows).  `warp_sums`: NT / 32 ints of shared memory.
// Called by all NT threads; ends with a barrier.
template <int NT, class F>
__device__ __forceinline__ void tile_sums(int G, const int *start, int *first, int *warp_sums,
                                          F tiles_of)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (G == 1) {
        if (tid == 0) {
            first[0] = 0;
            first[1] = tiles_of(start[1] - start[0]);
        }
        __syncthreads();
        return;
    }
    int before = 0;                      // tiles of the rounds before this one
    for (int base = 0; base < G; base += NT) {
        const int i = base + tid;
        const int n = i < G ? tiles_of(start[i + 1] - start[i]) : 0;
        int v = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {          // running sum of the warp
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += o;
        }
        if (lane == 31) warp_sums[warp] = v;
        __syncthreads();
        int lower = 0, all = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            const int s = warp_sums[w];
            lower += w < warp ? s : 0;
            all += s;
        }
        if (i < G) first[i] = before + lower + v - n;
        before += all;
        __syncthreads();
    }
    if (tid == 0) first[G] = before;
    __syncthreads();
}

// Fewer than 32 * WARP_ROUNDS groups fit in the registers of a warp: lane l of
// round r has group 32 r + l.  Through shared memory, by group_starts and
// tile_sums with the barriers between them, calls of 8 or 64 groups of few rows
// took 0.7 or 0.6 us longer, of more rows (8192 x 512 x 512) 0.5.
constexpr int WARP_ROUNDS = 4;

struct WarpGroups {
    int start[WARP_ROUNDS], next[WARP_ROUNDS];       // offsets of the group and of the next
    int G;
    __device__ __forceinline__ int rows(int r) const
    {
        return 32 * r + (int)(threadIdx.x & 31) < G ? next[r] - start[r] : 0;
    }
};

// The offsets, clamped as in group_starts (and reported, if `report`).
__device__ __forceinline__ WarpGroups warp_groups(const Groups &gr, int *err, bool report)
{
    const int lane = threadIdx.x & 31, G = gr.G;
    WarpGroups w;
    w.G = G;
    int v[WARP_ROUNDS + 1];
    bool bad = false;
#pragma unroll
    for (int r = 0; r < WARP_ROUNDS; ++r) {
        const int i = r * 32 + lane;
        const int raw = gr.offsets == nullptr ? (i == 0 ? 0 : gr.M) : gr.offsets[min(i, G)];
        v[r] = raw < 0 ? 0 : raw > gr.M ? gr.M : raw;
        bad = bad || v[r] != raw;
    }
    v[WARP_ROUNDS] = v[WARP_ROUNDS - 1];
    auto neighbours = [&] {
#pragma unroll
        for (int r = 0; r < WARP_ROUNDS; ++r) {
            const int down = __shfl_down_sync(0xffffffffu, v[r], 1);
            const int wrap = __shfl_sync(0xffffffffu, v[r + 1], 0);
            w.start[r] = v[r];
            w.next[r] = lane < 31 ? down : wrap;
        }
    };
    neighbours();
#pragma unroll
    for (int r = 0; r < WARP_ROUNDS; ++r) bad = bad || w.rows(r) < 0;
    if (__any_sync(0xffffffffu, bad)) {              // clamp: the running maximum
        if (report && lane == 0) atomicCAS(err, 0, ERR_INVALID);
        int top = 0;
#pragma unroll
        for (int r = 0; r < WARP_ROUNDS; ++r) {
            v[r] = max(v[r], top);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, v[r], d);
                if (lane >= d) v[r] = max(v[r], o);
            }
            top = __shfl_sync(0xffffffffu, v[r], 31);
        }
        v[WARP_ROUNDS] = top;
        neighbours();
    }
    return w;
}

// first[0..G]: how many tiles the groups before g have, a group of `rows` rows
// having tiles_of(rows).  By one warp; a barrier of the CTA has to follow.
template <class F>
__device__ __forceinline__ void warp_tile_sums(const WarpGroups &w, int *first, F tiles_of)
{
    const int lane = threadIdx.x & 31;
    int before = 0;
#pragma unroll
    for (int r = 0; r < WARP_ROUNDS; ++r) {
        if (32 * r > w.G) break;
        const int n = tiles_of(w.rows(r));
        if (w.G == 1) {
            const int all = __shfl_sync(0xffffffffu, n, 0);
            if (lane < 2) first[lane] = lane * all;
            return;
        }
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += o;
        }
        if (32 * r + lane <= w.G) first[32 * r + lane] = before + sum - n;
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
}

// The group that unit u belongs to, groups having first[g + 1] - first[g]
// tiles of `per` units each: the last g with first[g] * per <= u.  Called by
// whole warps: each step looks at 32 places of the range that is left (halving
// it instead: 5 to 10 dependent reads before a tile's first load, 0.1 to 0.2 us).
__device__ __forceinline__ int group_of(const int *first, int G, int per, int u)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = G;
    while (n > 1) {
        const int step = n <= 32 ? 1 : 32;           // MAX_GROUPS = 32 * 32
        const bool in = lane * step < n && first[lo + lane * step] * per <= u;
        const int at = max(__popc(__ballot_sync(0xffffffffu, in)) - 1, 0) * step;
        lo += at;
        n = min(step, n - at);
    }
    return lo;
}

// The unit'th chunk of at most `per` rows, a power of two, over all groups: its group,
// first row and rows; false beyond the last.  By whole warps, without shared
// memory; offsets are clamped as in group_starts.
__device__ __forceinline__ bool find_chunk(const Groups &gr, int per, int unit, int *err, int &g, int &row0,
                                           int &rows)
{
    const int lane = threadIdx.x & 31;
    if (gr.offsets == nullptr) {
        g = 0;
        row0 = unit * per;
        rows = min(per, gr.M - row0);
        return rows > 0;
    }
    const int shift = __ffs(per) - 1;
    int top = 0, before = 0;                         // largest offset and chunks so far
    bool bad = false;
    for (int base = 0; base < gr.G; base += 32) {
        const int a = gr.offsets[min(base + lane, gr.G)], b = gr.offsets[min(base + lane + 1, gr.G)];
        int lo = a < 0 ? 0 : a > gr.M ? gr.M : a, hi = b < 0 ? 0 : b > gr.M ? gr.M : b;
        bad = bad || lo != a || hi != b || hi < lo;
        lo = max(lo, top);
        hi = max(hi, lo);
        if (__any_sync(0xffffffffu, bad)) {          // running maxima, the slow way
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, hi, d);
                if (lane >= d) hi = max(hi, o);
            }
            const int o = __shfl_up_sync(0xffffffffu, hi, 1);
            if (lane > 0) lo = max(lo, o);
            if (lane == 0) atomicCAS(err, 0, ERR_INVALID);
        }
        const int n = base + lane < gr.G ? (hi - lo + per - 1) >> shift : 0;
        const int all = __reduce_add_sync(0xffffffffu, n);
        if (unit < before + all) {
            int sum = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += o;
            }
            const int first = before + sum - n;
            const int src = __ffs(__ballot_sync(0xffffffffu, unit >= first && unit < first + n)) - 1;
            g = base + src;
            row0 = __shfl_sync(0xffffffffu, lo, src) + (unit - __shfl_sync(0xffffffffu, first, src)) * per;
            rows = min(per, __shfl_sync(0xffffffffu, hi, src) - row0);
            return true;
        }
        before += all;
        top = __shfl_sync(0xffffffffu, hi, 31);
    }
    return false;
}

}  // namespace swg
