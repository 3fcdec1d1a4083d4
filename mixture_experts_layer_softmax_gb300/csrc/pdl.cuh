// Programmatic dependent launch: within a call's own chain of kernels, and between the
// calls that launch with it: their kernels wait at their start (every thread: a block
// that ended without would let the next kernel pass the one before), touch no memory
// before it, and let the next kernel come as soon as all their blocks have.
#pragma once

#include "common.cuh"

namespace moe {

// Programmatic dependent launch: a kernel launched with pdl_launch may be
// scheduled while the previous kernel on the stream is still finishing; it
// waits here, before its first memory access, until that kernel has
// completed and its writes are visible (a no-op without a dependency).  The
// previous kernel lets it be scheduled early with pdl_trigger.
MOE_D void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
MOE_D void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
static cudaError_t pdl_launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// With pdl false a plain launch: the kernel's pdl_wait returns at once and
// it starts only after everything before it on the stream has completed.
template <typename... KArgs, typename... Args>
static cudaError_t launch_maybe_pdl(bool pdl, void (*kern)(KArgs...), dim3 grid, dim3 block,
                                   size_t smem, cudaStream_t s, Args... args) {
  if (pdl) return pdl_launch(kern, grid, block, smem, s, args...);
  kern<<<grid, block, smem, s>>>(args...);
  return cudaGetLastError();
}

}  // namespace moe
