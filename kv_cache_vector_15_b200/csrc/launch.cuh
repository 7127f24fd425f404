// Launches of the paged cache's kernels.
#pragma once

#include <cuda_runtime.h>

#include "tq_internal.h"

namespace tq {

// A kernel launched by launch_dependent may be set up while the kernel before
// it in the stream ends.  It calls this first, in every thread: what that
// kernel wrote is visible afterwards, and what it read may be written.  Before
// the call a kernel may set up its own shared memory and barriers, and nothing
// else: what it took there and another kernel waits for (tensor memory) would
// be held until that other one has ended.  (An
// earlier set-up yet, by an explicit trigger behind this, measured no difference.)
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Also the cheaper launch on the host: 1.9 us where <<<>>> takes 2.6.
template <typename... Params, typename... Args>
int launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  count_launch();
  return static_cast<int>(e);
}

}  // namespace tq
