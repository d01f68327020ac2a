// host.h — host helpers of api.cu that the other C-ABI translation unit
// (api_experts.cu) uses: the device's state, tensor-map encoding, the
// split-K workspace, launch counting and error recording.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

namespace swg {

struct DeviceInfo {
    int sms;       // multiprocessors of the current device
    int *err;      // its device error word
};

// The current device, with its context bound to this thread (SWG_OK or an
// error status, recorded like every other entry point's).
int device_info(DeviceInfo &out);

// Records the runtime's pending error of this thread; returns SWG_ERR_CUDA.
int record_cuda_error();

// Counts one launch of this library and reports a pending launch error.
int count_launch(cudaError_t e);

// FP32 partials of a split call on (current device, stream): grow-only,
// library-owned, freed by swg_shutdown; SWG_ERR_UNSUPPORTED when it would
// have to allocate while the stream is being captured.  They are this call's
// as long as it keeps `held`: until its last kernel is queued.
int stream_workspace(cudaStream_t s, size_t bytes, float *&out, std::unique_lock<std::mutex> &held);

// cuTensorMapEncodeTiled with a swizzle of 128 or 0 (none) bytes, unit
// element strides, no interleave and zero fill; false (recorded) when it
// fails.  strides[i] is the byte stride of dimension i + 1.
bool encode_tiled(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *ptr,
                  const uint64_t *dims, const uint64_t *strides, const uint32_t *box, int swizzle);

}  // namespace swg
