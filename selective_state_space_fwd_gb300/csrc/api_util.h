// api_util.h -- host-side argument checks shared by the C ABI's entry points.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ssmscan.h"

namespace ssm {

inline size_t elem_size(ssm_dtype t) { return t == SSM_BF16 ? 2 : 4; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a * b without signed overflow, for non-negative operands; false on overflow.
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

// The entry points keep per-device state (the sticky error word of the
// bounded waits, copy streams, the address of the fixed workspace) and look it
// up by the calling thread's current device; `stream` must belong to that
// device, else SSM_ERR_CUDA.  The special handles (0, legacy, per-thread)
// always do.
inline ssm_status current_device_for(cudaStream_t stream, int* dev) {
  if (cudaGetDevice(dev) != cudaSuccess) return SSM_ERR_CUDA;
  if (stream == nullptr || stream == cudaStreamLegacy || stream == cudaStreamPerThread)
    return SSM_OK;
  // A stream being captured into a CUDA graph is not queried for its device
  // (the query would invalidate the capture); the calls then only record work.
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) return SSM_ERR_CUDA;
  if (cap != cudaStreamCaptureStatusNone) return SSM_OK;
  int sdev = -1;
  if (cudaStreamGetDevice(stream, &sdev) != cudaSuccess) return SSM_ERR_CUDA;
  return sdev == *dev ? SSM_OK : SSM_ERR_CUDA;
}

}  // namespace ssm
