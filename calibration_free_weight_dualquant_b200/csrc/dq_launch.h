// dq_launch.h -- launch of the linear layer's kernels, optionally in clusters,
// with programmatic stream serialization: a kernel may be set up (barriers,
// tensor memory, its grid's launch) while the one before it in the stream
// finishes.  Every thread of such a kernel calls griddep_wait() before it
// touches global memory.
#pragma once

#include <cuda_runtime.h>

#include <cstring>

namespace dq {

inline void cluster_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* at, unsigned grid, unsigned block, size_t smem,
                           int cluster) {
  std::memset(cfg, 0, sizeof(*cfg));
  cfg->gridDim = dim3(grid);
  cfg->blockDim = dim3(block);
  cfg->dynamicSmemBytes = smem;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = (unsigned)cluster;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  cfg->attrs = at;
  cfg->numAttrs = 1;
}

template <typename... KArgs, typename... Args>
inline cudaError_t launch_early(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, int cluster,
                                cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute at[2];
  cluster_config(&cfg, at, grid, block, smem, cluster);
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = cluster > 1 ? at : at + 1;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace dq
