// A kernel that starts while the one before it in its stream still runs: its CTAs take
// the places that come free, and wait before they touch what that kernel writes. It
// saves most of a launch's latency, about 2 us of a call of two kernels.
#pragma once
#include <cuda_runtime.h>

namespace fm {

// In the kernel before: the next one may start once every CTA has come here (or ended).
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// In a kernel of launch_overlapped: the kernel before has ended and its writes are seen.
// At least one thread of each CTA comes here, so that no kernel ends before those it
// follows.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                              Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace fm
