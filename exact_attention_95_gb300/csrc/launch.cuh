// launch.cuh -- launches by programmatic stream serialization.
#pragma once

#include <cuda_runtime.h>

namespace attn {

// Launches a kernel that may start while the one before it in the stream ends
// (it waits for that one before it reads anything).  smem: bytes of dynamic shared memory.
template <class... P, class... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, int threads, cudaStream_t stream, size_t smem, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace attn
