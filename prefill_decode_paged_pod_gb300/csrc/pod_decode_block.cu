// pod_decode_block.cu — the paged decode over E4M3 caches with block scales.
#include "pod_decode.cuh"

cudaError_t pod::decode_launch_block(int d, bool bf16, DecodeParams& P, cudaStream_t st) {
  return bf16 ? launch_decode<__nv_bfloat16, POD_KV_E4M3_BLOCK>(d, P, st) : launch_decode<__half, POD_KV_E4M3_BLOCK>(d, P, st);
}
