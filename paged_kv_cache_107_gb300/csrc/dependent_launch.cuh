// dependent_launch.cuh — launches with programmatic stream serialization.
#pragma once

#include <cuda_runtime.h>

namespace pa {
namespace {

// Launch with programmatic stream serialization: the grid may be scheduled while the
// previous kernel on the stream is still running (its CTAs run the prologue, then wait in
// pdl_wait for that kernel to complete before using anything it wrote).
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

}  // namespace
}  // namespace pa
