// Launch of a kernel that may be set up while the kernel before it on the
// stream ends (programmatic dependent launch).  Such a kernel's threads all call
// pdl_enter() before anything else: it returns when the earlier kernel has
// completed with its memory visible, so the stream's order holds as for a plain
// launch, and then lets the next kernel be set up in turn.  In a decode step the
// operators follow one another and each takes a few microseconds, of which this
// saves the launch latency.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace pa {

// In clusters of `cluster` CTAs.
template <class... Params, class... Args>
cudaError_t launch_in_clusters(void (*kern)(Params...), unsigned grid, unsigned cluster, unsigned block, int smem,
                               cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

template <class... Params, class... Args>
cudaError_t launch_in_order(void (*kern)(Params...), unsigned grid, unsigned block, int smem, cudaStream_t st,
                            Args&&... args) {
  return launch_in_clusters(kern, grid, 1, block, smem, st, std::forward<Args>(args)...);
}

}  // namespace pa
