// groups.cuh — the table of row groups that the grouped kernels build in
// shared memory from the offsets on the device.
#pragma once

#include "experts.h"

namespace swg {

constexpr int ERR_INVALID = 1;       // == SWG_ERR_INVALID_ARG

// Run by one whole warp.  start[0..G]: the offsets, clamped to be
// non-decreasing within [0, M], so that every row a kernel derives from them
// exists; an offset that had to be clamped is reported in the error word.
__device__ __forceinline__ void group_starts(const Groups &gr, int *start, int *err)
{
    const int lane = threadIdx.x & 31;
    if (gr.offsets == nullptr) {         // one group of all rows
        if (lane == 0) {
            start[0] = 0;
            start[1] = gr.M;
        }
        __syncwarp();
        return;
    }
    const int G = gr.G;
    int top = 0;                         // the largest offset so far
    bool bad = false;
    for (int base = 0; base <= G; base += 32) {
        const int i = base + lane;
        const int raw = i <= G ? gr.offsets[i] : 0;
        int v = raw < 0 ? 0 : raw > gr.M ? gr.M : raw;
        if (lane == 0 && v < top) v = top;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {          // running maximum
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d && o > v) v = o;
        }
        if (i <= G) {
            start[i] = v;
            bad = bad || v != raw;
        }
        top = __shfl_sync(0xffffffffu, v, 31);
    }
    if (bad) atomicCAS(err, 0, ERR_INVALID);
    __syncwarp();
}

// Run by one whole warp.  first[0..G]: how many tiles the groups before g
// have, a group of `rows` rows having tiles_of(rows).
template <class F>
__device__ __forceinline__ void tile_sums(int G, const int *start, int *first, F tiles_of)
{
    const int lane = threadIdx.x & 31;
    int sum = 0;
    for (int base = 0; base < G; base += 32) {
        const int i = base + lane;
        const int n = i < G ? tiles_of(start[i + 1] - start[i]) : 0;
        int v = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {          // running sum
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += o;
        }
        if (i < G) first[i] = sum + v - n;
        sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) first[G] = sum;
    __syncwarp();
}

// The group that tile t (< first[G]) belongs to: the last g with first[g] <= t.
__device__ __forceinline__ int group_of(const int *first, int G, int t)
{
    int lo = 0, hi = G;                  // first[lo] <= t < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

}  // namespace swg
