// pod_decode_16.cu — the paged decode over 16-bit caches.
#include "pod_decode.cuh"

cudaError_t pod::decode_launch_16(int d, bool bf16, DecodeParams& P, cudaStream_t st) {
  return bf16 ? launch_decode<__nv_bfloat16, POD_KV_16BIT>(d, P, st) : launch_decode<__half, POD_KV_16BIT>(d, P, st);
}
