// pod_tree_k8b.cu — instantiations of the tree attention for caches of format: E4M3, block scales.
#include "pod_tree.cuh"

cudaError_t pod_tree_k8b(const PodTreeParams& P, int dtype, int d, cudaStream_t stream) {
  return launch_tree_kv<2>(P, dtype, d, stream);
}
