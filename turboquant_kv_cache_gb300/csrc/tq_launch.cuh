// Launches of calls that are several kernels in a row.
#pragma once

#include <cuda_runtime.h>

#include "tq_device.cuh"

namespace tq {

// Kernels of one call in a row: a kernel may start when the one before it
// has, and waits here until that one has ended and its writes are visible.
__device__ __forceinline__ void chain_begin() {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
}

// Launches a kernel of a call; chained: its set-up overlaps the kernel before
// it, which it waits for itself (chain_begin).
template <class... P, class... A>
inline bool launch(void (*kern)(P...), int64_t blocks, int threads, bool chained, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = chained ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

}  // namespace tq
