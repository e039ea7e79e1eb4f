// Programmatic dependent launch: consecutive kernels of the library on one
// stream overlap one's start-up (barrier set-up, TMEM allocation, table loads,
// reads of the handle's immutable arrays) with the tail of the kernel before.
//
// A kernel launched with launch_pdl must call pdl_wait() before it touches any
// memory an earlier kernel of the stream may write or read (inputs, workspace,
// outputs, hand-off flags); it calls pdl_release() once its own CTAs no longer
// need to hold back the next kernel's start.  Here that is right behind
// pdl_wait(): the next kernel starts once every CTA of this one has called it
// or ended, so where a grid is larger than what fits the GPU at a time (norms and
// rotation, sampling, the attention's join) not before its last CTAs have begun,
// and it takes nothing that this one's CTAs still need.  Since every kernel waits,
// all before it have ended and are visible when pdl_wait() returns.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace uw {

__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void pdl_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The same for a grid of clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, int cluster, dim3 block,
                               size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace uw
