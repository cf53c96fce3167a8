// Launches of the serving kernels with programmatic dependence: a kernel may be
// put on the SMs while the one in front of it in the stream still drains, and
// waits for its end (wait_for_previous) before it touches global memory (but for
// the decode kernels' status word, which only says that nothing more need be
// done).  Each of these kernels is a few microseconds, of which a full launch
// behind another kernel is one or two.
#pragma once
#include <cuda_runtime.h>

namespace ra {

// Everything the stream did before this kernel is complete and visible.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// The next kernel of the stream may be put on the SMs from here on.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, unsigned smem,
                         cudaStream_t st, A&&... args) {
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
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace ra
