// Launching kernels that follow one another in one call: each may be set up
// while the one before it drains (programmatic dependent launch), and calls
// await_previous() before it touches memory.
#pragma once

#include <cuda_runtime.h>

namespace zero {

// Wait until every kernel launched before this one has finished and its
// writes are visible.  Nothing of another kernel's is read or written before.
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Let the next kernel's blocks take free SMs (they stop at await_previous()).
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*fn)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<Params>(args)...);
}

}  // namespace zero
