// Host-side services of api.cu for the other files that hold entry points.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cb.h"

namespace cb {

// The current device's SM count and error word.
cb_status host_device(int* sms, int** err);
// Records a CUDA error for cb_last_cuda_error; returns CB_ERR_CUDA.
cb_status host_cuda_fail(cudaError_t e);
// The bound of a device wait (CB_TIMEOUT_MS), in nanoseconds.
uint64_t host_timeout_ns();
// Encodes a bf16 tiled map of rank 4 (zero fill outside; 128-byte swizzle); false if the driver refuses it.
bool host_map_bf16(CUtensorMap* out, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides_bytes,
                   const cuuint32_t* box);

}  // namespace cb
