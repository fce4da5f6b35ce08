// kmip_launch.cuh -- kernels of one call that follow one another on a stream.
//
// A kernel launched with launch_next may be set up, and its blocks placed as
// soon as every block of the kernel before it has started, while that one still
// runs; its blocks then stop at after_previous() until the kernel before has
// finished and its results are visible.  So the launch, 1 to 2 us between two
// dependent kernels, costs next to nothing.  Every kernel of such a sequence
// calls after_previous() before it touches memory; launched the plain way (the
// first of a call, which has to follow whatever else is on the stream) it goes
// straight through.
#pragma once

#include <cuda_runtime.h>

namespace kmip {

__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                        cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, P(args)...);
}

}  // namespace kmip
