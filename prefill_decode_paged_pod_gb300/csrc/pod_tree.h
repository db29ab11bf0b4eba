// pod_tree.h — records and launch parameters of the tree attention, shared by
// the planner (host) and the kernels.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#define POD_TREE_BLOCK 64     // keys per block (one S buffer, one stage)
#define POD_TREE_BLOCKB 128   // the same for block-scaled caches
#define POD_TREE_TILE 128     // packed query rows per tile (TMEM lanes)

// Segment record, one for each run of key blocks that a CTA works through for
// one tile (request, KV head, 128 packed rows); row i of a tile is packed row
// mt * 128 + i: token (.. / G), head g * G + (.. % G).
enum PodTreeSeg {
  TS_G = 0,        // KV head
  TS_ROW0,         // first packed row of the tile within its request
  TS_NROWS,        // rows of the tile
  TS_BLK0, TS_BLK1,// key blocks [blk0, blk1)
  TS_PROW,         // first partial row, -1: the segment covers every block of the tile
  TS_KVLEN,
  TS_NTOK,         // tree tokens of the request
  TS_QROW0,        // first query row of the request
  TS_PAGE0,        // first entry in the page table
  TS_NPAGES,
  TS_BIT_LO, TS_BIT_HI,   // first mask bit of the request (64 bits)
  TS_COPIES,       // 1, 2 or 4: how many key slices the tile's lanes hold
  TS_REC = 16
};
// Merge group: the segments' partial rows of one split tile. Tiles in more than
// POD_TREE_FEW segments are listed first.
#define POD_TREE_FEW 4
enum PodTreeGroup { TG_G = 0, TG_ROW0, TG_NROWS, TG_PROW0, TG_NSEG, TG_QROW0, TG_REC = 8 };
// Status block (int32) at the start of the workspace.
enum { TREE_ST_STATUS = 0, TREE_ST_INTS = 64 };

struct PodTreeParams {
  CUtensorMap tm_k, tm_v;        // boxes of K and of V
  const void *q, *kv;
  const uint8_t* scales;         // block-scaled cache: exponent bytes
  const uint8_t* mask;           // packed tree mask, nullptr: a chain
  long long mask_bytes;
  const float* sinks;
  void* out;
  float* lse;
  const int32_t *segs, *cta_ptr, *pages, *groups;
  float *part_o, *part_lse;
  int32_t* status;
  long long page_rows;           // cache rows of a page, K and V
  int H, Hk, G, ps, ps_shift, hnd, num_pages;
  int kbx;                       // keys per TMA box, 0: gather
  int n_cta, n_groups, n_big;    // merge groups, those of many segments
  float scale_log2;              // sm_scale * log2(e) (* k_scale)
  float v_scale;
};

// kv format: 0 = 16-bit, 1 = E4M3, 2 = E4M3 with block scales
cudaError_t pod_tree_k16(const PodTreeParams& P, int dtype, int d, cudaStream_t stream);
cudaError_t pod_tree_k8(const PodTreeParams& P, int dtype, int d, cudaStream_t stream);
cudaError_t pod_tree_k8b(const PodTreeParams& P, int dtype, int d, cudaStream_t stream);
// A workspace holds another plan from now on: tree plans bound to it have lost it.
void pod_tree_workspace_lost(void* workspace);
cudaError_t pod_tree_merge(const PodTreeParams& P, int dtype, int d, cudaStream_t stream);
