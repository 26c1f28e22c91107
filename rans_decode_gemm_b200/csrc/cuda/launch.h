// launch.h -- host-side kernel launch with programmatic dependent launch:
// the kernel may start while the previous kernel in the stream is still running.
// An ordinary kernel runs only a prologue that touches no global memory, and its
// griddep_wait() orders every global-memory access after that kernel.  A kernel
// that uses none of that kernel's results runs beside it (griddep_beside() in
// ptx.cuh says what it may read and write, and how the next kernel waits for both).
#pragma once
#include <cuda_runtime.h>

namespace ansdev {

template <typename... KArgs, typename... Args>
static cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
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
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

}  // namespace ansdev
