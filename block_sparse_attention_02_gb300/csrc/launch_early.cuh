// launch_early.cuh -- launches that follow one another without a gap.
#pragma once

#include <cuda_runtime.h>

namespace msa {

// A launch that the device may prepare while the kernel before it in the stream still runs; the kernel
// calls wait_for_stream() before its first access to global memory.  Kernels of a few microseconds
// follow one another in 3 us so, where plain launches take 6 (page tables of 8 requests).  cluster: CTAs of a
// thread-block cluster, 1 for none.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                         A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// In a kernel launched while the one before it in the stream may still run: waits until
// everything before is complete and visible.  Called before the first access to global
// memory, so stream order holds.  (No kernel here lets its successor start
// earlier than its own end: with such a trigger at the start, the waiting CTAs cost the
// running kernel more than they gain: a store and expand of 8,192 tokens became a fifth slower.)
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace msa
