// launch.cuh -- launches of the layers' kernels, which overlap their starts
// with the end of the kernel before them.
//
// Every kernel launched here begins with begin_after_previous() (the products'
// kernel, which sets up barriers and tensor memory first, with its two halves).
// With programmatic stream serialization its blocks may be placed as soon as
// every block of the kernel before them has begun (if that one is of this kind
// too) and SMs fall free; griddepcontrol.wait then holds each thread until the
// kernel before has completed and its writes are visible.  So nothing of a
// neighbour is read or written early, and one kernel's launch latency runs under
// the other's end.
#pragma once

#include <cuda_runtime.h>

#include "sm100.cuh"

namespace ag {

__device__ __forceinline__ void begin_after_previous() {
  griddep_launch_dependents();
  griddep_wait();
}

template <typename... P, typename... A>
cudaError_t launch_after_previous(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                  cudaStream_t stream, A &&...args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace ag
