// fab_launch.cuh -- launching a kernel behind the one before it in its stream.
#pragma once

#include <cuda_runtime.h>

namespace fab {

// Launches a kernel that may start while the one before it in the stream still
// runs, and waits for that one itself (griddepcontrol.wait) before it touches
// memory: its launch and its first instructions cost no time of their own.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace fab
