// grouped_launch.cuh — launch helper of the grouped kernels' translation units.
#pragma once

#include <algorithm>

#include "grouped.cuh"
#include "host.h"
#include "launch.h"

namespace swg {

// Launches at most `units` pairs of CTAs (clusters of two), no more than can
// be resident at once with smem_most bytes of shared memory (`smem`: what this
// call needs of them).  The kernel may be scheduled early behind the kernel
// before it on the stream; it waits for that kernel's end before it reads
// the offsets.
template <auto KERNEL, int THREADS, class... Args>
cudaError_t launch_pairs(int smem, int smem_most, long long units, int sms, cudaStream_t s,
                         const Args &...args)
{
    static DeviceOnce configured;
    static std::atomic<int> resident[DeviceOnce::kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    int pairs = 0;
    if (configured.needed(dev)) {
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_most);
        if (e != cudaSuccess) return e;
        cfg.numAttrs = 1;
        cfg.dynamicSmemBytes = smem_most;
        cfg.gridDim = dim3(2 * (sms / 2));           // a CTA per SM
        e = cudaOccupancyMaxActiveClusters(&pairs, KERNEL, &cfg);
        if (e != cudaSuccess) return e;
        if (pairs < 1) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < DeviceOnce::kDevices) resident[dev].store(pairs);
        configured.mark(dev);
    } else {
        pairs = resident[dev].load();
    }
    cfg.numAttrs = 2;
    cfg.dynamicSmemBytes = smem;
    cfg.gridDim = dim3((unsigned)(2 * std::min<long long>(units, pairs)));
    return cudaLaunchKernelEx(&cfg, KERNEL, args...);
}

template <int MATH, int EPI, bool FEW>
cudaError_t launch_grouped_kernel(const GrpMaps &m, GrpParams p, long long units, int sms,
                                  cudaStream_t s)
{
    using C = GrpCfg<MATH, FEW>;
    const int G = p.groups.G;
    p.stages = C::stages_of(C::STAGE_BYTES, G);
    // Tiles of whole width that are done in a few stages are bound by their
    // results; loads further ahead slow those (MXFP4, 8192 x 8192: K = 1024 49.4
    // us with 6 stages, 47.4 with 5; K = 4096 the other way round, 133 and 138 us
    // for 8192 x 14336; 32 groups of 128 rows, K = 2048: 23.7 and 24.5).
    if (!FEW && p.k_blocks <= 8 && p.groups.M / std::max(G, 1) >= C::TOKENS)
        p.stages = std::min(p.stages, 5);
    p.stages_narrow = C::stages_of(C::NARROW_BYTES, G);
    p.ring_bytes = C::ring_bytes(G);
    return launch_pairs<grouped_kernel<MATH, EPI, FEW>, C::THREADS>(C::smem_bytes(G), SMEM_MOST, units,
                                                                    sms, s, m, p);
}

}  // namespace swg
