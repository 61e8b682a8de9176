// Launches that may be set up while the kernel before them in the stream still runs (programmatic dependent
// launch).  A kernel launched this way may start early, and touches no global memory but a plan's own tables before
// wait_for_previous(), which returns once every earlier kernel of the stream has finished and its writes are visible;
// each of its threads passes that wait before it ends, so the order is handed on to the kernel after it.  What is saved
// is the launch latency and the set-up of barriers and tensor memory: 2 us of a kernel behind another.
// Such a kernel lives while its inputs are still being written, so it reads them with plain loads: the read-only path
// (__ldg, const __restrict__) wants memory that does not change for as long as the kernel lives.
// Kernels, copies and events of other origin before or after keep the stream's plain order.
#pragma once
#include <cuda_runtime.h>

namespace zl {

__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may be set up as soon as every block of this one has said so (all are then running or done, so it
// takes nothing that this one still needs).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// early = false: an ordinary launch of the same kernel (its wait returns at once).  For kernels that fill the SMs for
// long: their blocks set up early won 2 us of a launch, and cost 1 to 2 % of launches of 250 us and more, which run at
// the power limit (packed batch of 14 337 tokens 251 against 254 us, training step of 26 487 tokens 2246 against 2294).
template <typename... Params, typename... Args>
cudaError_t launch_overlapped_if(bool early, void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                                 cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              const Args&... args) {
  return launch_overlapped_if(true, kernel, grid, block, smem, stream, args...);
}

}  // namespace zl
