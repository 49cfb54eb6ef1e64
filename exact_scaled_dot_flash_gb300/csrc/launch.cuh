// launch.cuh - launches that overlap the end of the one before them on the stream.
#pragma once

#include <cuda_runtime.h>

namespace attn {

// A launch that may come up before the one in front of it on the stream has ended; its kernel waits
// (griddepcontrol.wait) before it touches what that one or an earlier one has written.
// cluster: CTAs of a cluster (in x), 0: none.
template <typename... A>
cudaError_t launch_early(void (*kern)(A...), dim3 grid, int threads, int smem, cudaStream_t st, int cluster, A... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace attn
