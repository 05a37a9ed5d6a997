// Programmatic dependent launch: a kernel is set up while the one before it in
// the stream still runs, and waits on the device for its results.
//
// Every kernel launched with launch_pdl calls pdl_wait() on all paths before
// it reads or writes global memory, and so finishes only after all kernels
// before it have: the order of the stream holds for whatever comes next,
// launched this way or not.
#pragma once

#include <cuda_runtime.h>

namespace fa {

// Waits until the kernels before this one in the stream have finished and
// their writes are visible.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel be set up as soon as all CTAs of this one have started.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace fa
