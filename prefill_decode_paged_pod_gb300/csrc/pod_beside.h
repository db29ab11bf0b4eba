// pod_beside.h — launches of the decode step's kernels: beside the kernel before
// (programmatic stream serialization; the kernels wait for it inside), in clusters
// where asked, with shared memory past the default allowed once per device.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

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

// Attributes belong to each device: set once per device (`done` and `mu` are the kernel's own).
template <typename K>
cudaError_t allow_shared(K kernel, int bytes, bool wide_clusters, std::atomic<unsigned long long>& done, std::mutex& mu) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  std::lock_guard<std::mutex> lock(mu);
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && wide_clusters)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

}  // namespace pod
