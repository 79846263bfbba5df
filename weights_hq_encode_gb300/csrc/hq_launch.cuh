// hq_launch.cuh -- launches that overlap the end of the kernel before them.
#pragma once
#include <cuda_runtime.h>

namespace hq {

// The first thing a kernel launched by launch_behind does, in every thread:
// waits until all that came before it in the stream has ended and can be
// seen, and lets the launch after it begin likewise.  No thread may leave
// before it, as the next kernel relies on this one's end for all before it.
// Behind it ordinary loads see what came before; loads through the read-only
// path (__ldg) are not for such kernels, whose lifetime begins before their
// inputs are written.
__device__ __forceinline__ void follow_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A launch that may begin while the one before it in the stream still runs
// (its kernel calls follow_launch): the time to start its blocks is hidden.
template <class... Params, class... Args>
int launch_behind(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) == cudaSuccess) return 0;
  cudaGetLastError();                            // reported here, not to the next caller
  return 1;
}

}  // namespace hq
