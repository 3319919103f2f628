// pdl.cuh -- launching a kernel while the one before it in the stream still
// drains (programmatic dependent launch): the later kernel's blocks may start
// as soon as every block of the earlier one has called release_next() (or
// ended), and wait_previous() holds them until the earlier grid is complete and
// its writes are visible.  Every kernel launched this way calls
// wait_previous() before it touches memory, so completion stays in order along
// a chain of such launches; one that touches memory before it (embed_fill_kernel) says which
// launch without this attribute, just before, makes that safe, and still calls it.
#pragma once
#include <cuda_runtime.h>

namespace ssm {

__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void release_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         A&&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace ssm
