// Programmatic launches: of the shared-prefix decode's passes, the 4-bit pool's kernels, the joining of split units and the
// page operators.
#pragma once
#include <cuda_runtime.h>

namespace pa {

// A kernel launched early is set up while the one before it in its stream ends, and
// waits for that one before its first access to global memory (what precedes the wait
// reads parameters only; but for the shared-prefix decode's pass over own keys, which reads nothing that the
// prefix pass before it writes, and whose wait stands at its end).  What it reads goes past the read-only path (__ldcg, plain loads,
// bulk copies; never __ldg): the kernel before may write it while this one already
// runs.  In every grid some CTA waits, so a grid is over only after all that precede it.  A
// row of calls: decode of 64 contexts 36.4 us each (39.0 without), append of 9800 tokens 18.5 (20.5).
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const Args&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pa
