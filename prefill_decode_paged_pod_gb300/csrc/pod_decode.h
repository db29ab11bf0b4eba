// pod_decode.h — what the paged decode's host side and its kernels share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pod.h"

namespace pod {

constexpr int kDecodeWarps = 4;                    // of a CTA
constexpr int kDecodeThreads = 32 * kDecodeWarps;

// status bits that the operators of a decode step join into *status
constexpr int kStatusSlot = 4;     // a slot or page outside the pool, a length outside its table
constexpr int kStatusNoRoom = 8;   // a step that did not fit: pages, rows or table width ran out

struct DecodeParams {
  const void* q;                   // [batch, H, d], q_stride elements a row
  const uint8_t* cache;
  const uint8_t* scales;           // exponent bytes of a block-scaled cache
  const int32_t* table;            // [batch, width], table_stride
  const int32_t* lens;             // [batch]
  const int32_t* pages;            // [batch, Hk, num_selected] or nullptr: all pages
  const float* sinks;              // [H] or nullptr
  void* out;                       // [batch, H, d], out_stride
  float* lse;                      // [batch, H] or nullptr
  int32_t* status;
  // workspace: total units of one plane, first unit of every request, the pieces
  long long* total;
  long long* first;
  float* piece_o;                  // [grid * 2][hw][heads of a tile][d], normalised
  float2* piece_at;                // [grid * 2][hw][heads of a tile]: reference and sum of its weights
  long long q_stride, out_stride, table_stride;
  unsigned num_pages;
  int batch, H, Hk, G, width, ps, ps_shift, hnd, num_selected, window;   // ps_shift: -1 where ps is no power of two
  int hw;                          // KV heads of a CTA
  int planes;                      // Hk / hw * head tiles
  int grid;                        // CTAs of the attention kernel
  float scale_log2;                // sm_scale * log2(e) (* k_scale)
  float v_scale;
};

// The launches. The attention kernel's partition of the work, and with it the workspace, is
// made for the CTAs that 152 SMs hold.
cudaError_t decode_launch_16(int d, bool bf16, DecodeParams& P, cudaStream_t st);
cudaError_t decode_launch_scaled(int d, bool bf16, DecodeParams& P, cudaStream_t st);
cudaError_t decode_launch_block(int d, bool bf16, DecodeParams& P, cudaStream_t st);

}  // namespace pod
