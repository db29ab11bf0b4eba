// pod_tree_k16.cu — instantiations of the tree attention for caches of format: 16-bit.
#include "pod_tree.cuh"

cudaError_t pod_tree_k16(const PodTreeParams& P, int dtype, int d, cudaStream_t stream) {
  return launch_tree_kv<0>(P, dtype, d, stream);
}
