// pod_tree_k8.cu — instantiations of the tree attention for caches of format: E4M3, per-tensor scales.
#include "pod_tree.cuh"

cudaError_t pod_tree_k8(const PodTreeParams& P, int dtype, int d, cudaStream_t stream) {
  return launch_tree_kv<1>(P, dtype, d, stream);
}
