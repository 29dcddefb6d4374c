// Programmatic dependent launch: a kernel may be set up while its predecessor
// in the stream still runs.  Every kernel launched this way begins with
// pdl_begin(), which waits until all earlier work of the stream is done and
// visible, and only then lets its own successor be set up; so the order of
// reads and writes between kernels is that of plain launches, and what is
// saved is the launch latency (1 to 2 us per kernel in a chain of short ones).
// What a call's first kernel found finished when it began, and does not write itself, its
// second kernel may read before pdl_begin(): it is set up when all blocks of the first
// have begun.  Nothing is written before pdl_begin().
#pragma once

#include <cuda_runtime_api.h>

namespace mcs {

#ifdef __CUDACC__
__device__ __forceinline__ void pdl_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// SMs of the current device.
inline cudaError_t sm_count(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem,
                             cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace mcs
