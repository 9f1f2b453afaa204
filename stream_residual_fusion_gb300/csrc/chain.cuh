// chain.cuh -- kernels of one call that begin while the one before them still runs (programmatic dependent
// launch): each opens the way for its successor at once, and waits for its predecessor where it first needs
// what that wrote, or before it writes what that reads.
#pragma once
#include <cuda_runtime.h>

#include <utility>

namespace mhc {

// Lets the next kernel's blocks start as soon as there is room for them.
__device__ __forceinline__ void open_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Waits until the kernel before this one, and so every one before that, is done and its writes are seen.
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches `kernel`, which calls wait_previous(), behind the kernel launched last on `stream`; not before its
// end unless `early`.
template <typename... P, typename... A>
cudaError_t launch_behind(bool early, void (*kernel)(P...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t stream,
                          A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(blocks);
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &attr;
  config.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&config, kernel, std::forward<A>(args)...);
}

}  // namespace mhc
