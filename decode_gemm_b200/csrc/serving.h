// Shared by the serving-step operators (paged.cu, attention.cu, sample.cu):
// host-side checks of their arguments and the device they run on.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "unweight.h"

namespace uw {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline uw_status map_launch(cudaError_t e) {
  if (e == cudaSuccess) return UW_OK;
  cudaGetLastError();  // a refused launch leaves its error behind; it is reported here
  return e == cudaErrorMemoryAllocation ? UW_ERR_OOM : UW_ERR_CUDA;
}

// The device that holds `p`; UW_ERR_ARG for memory that kernels cannot reach.
inline uw_status device_of(const void* p, int* dev) {
  cudaPointerAttributes at;
  const cudaError_t e = cudaPointerGetAttributes(&at, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e == cudaErrorInvalidValue ? UW_ERR_ARG : UW_ERR_CUDA;
  }
  if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return UW_ERR_ARG;
  *dev = at.device;
  return UW_OK;
}

// Two BF16 values, rounded to nearest even, as they lie in memory.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Multiprocessors of a device, asked for once per device.
int sm_count_of(int dev);

// A cache whose every (page, slot, head) the kernels may address: what the
// header states of uw_paged_cache (paged.cu).
uw_status check_cache(const uw_paged_cache& c);

}  // namespace uw
