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
cudaError_t launch_grouped_kernel(const GrpMaps &m, const GrpParams &p, long long units, int sms,
                                  cudaStream_t s)
{
    using C = GrpCfg<MATH, FEW>;
    return launch_pairs<grouped_kernel<MATH, EPI, FEW>, C::THREADS>(
        C::smem_bytes(p.groups.G), C::smem_bytes(MAX_GROUPS), units, sms, s, m, p);
}

}  // namespace swg
