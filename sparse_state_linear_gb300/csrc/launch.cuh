// launch.cuh -- kernels that may be launched while the kernel before them in
// the stream is still running (programmatic stream serialization).  Such a
// kernel waits at its start, before it touches global memory, for what comes
// before it; what overlaps is its launch and the scheduling of its blocks.
#pragma once

#include <cuda_runtime.h>

namespace sdm {

// In front of the first access to global memory of every kernel launched by
// launch_behind, in every thread.
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

template <class... Params, class... Args>
cudaError_t launch_behind(void (*kernel)(Params...), unsigned blocks, int threads, size_t smem,
                          cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(blocks);
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...);
}

}  // namespace sdm
