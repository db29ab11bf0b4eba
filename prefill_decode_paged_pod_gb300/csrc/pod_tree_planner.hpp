// pod_tree_planner.hpp — host plan of the tree attention.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <string>
#include <vector>

struct PodTreeArgs {
  const int32_t *q_indptr, *kv_indptr, *kv_indices, *last_page_len;
  int batch, num_pages, H, Hk, d, ps;
  int block;                       // keys per block
  int slots;                       // CTAs that run at once
};

struct PodTreePlanHost {
  int batch = 0, num_pages = 0, H = 0, Hk = 0, G = 0, d = 0, ps = 0, rows = 0;
  long long mask_bits = 0;
  std::vector<int32_t> segs, cta_ptr, pages, groups;
  int n_cta = 0, n_big = 0, n_prows = 0;
  // workspace layout (bytes)
  size_t off_segs = 0, off_cta = 0, off_pages = 0, off_groups = 0, off_part_o = 0, off_part_lse = 0,
         total = 0;
  std::vector<uint8_t> image;      // the part that is uploaded
};

// Returns a pod_status value; on error *err holds the message.
int pod_tree_build_plan(const PodTreeArgs& a, PodTreePlanHost& out, std::string* err);
