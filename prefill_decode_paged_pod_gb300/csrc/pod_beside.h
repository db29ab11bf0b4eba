// pod_beside.h — launches of the cache operators' and the decode step's kernels: beside
// the kernel before (programmatic stream serialization; the kernels wait for it inside), in
// clusters where asked.
#pragma once
#include <cuda_runtime.h>

namespace pod {

template <typename... A, typename... B>
cudaError_t launch_beside(void (*kernel)(A...), unsigned grid, unsigned threads, unsigned shared, unsigned cluster,
                          cudaStream_t st, const B&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pod
