// pod_tree_planner.cpp — cuts the tree attention of a batch into CTA work.
//
// A unit is one (request, KV head, tile of 128 packed rows) and costs its key
// blocks plus a fixed price for starting it (query load, pipeline fill,
// epilogue). The units of one KV head and tile index form a plane; a plane is laid
// out in request order and cut at equal cost, through the middle of units where
// it falls so, so every CTA gets the same work up to one block. Planes are cut
// alike: the CTAs at the same place of two planes read the same tokens at the
// same time, other heads' rows beside theirs in memory (an FP8 row of an NHD
// cache is 128 bytes, too little by itself for HBM: 96 requests of 8192 keys with
// per-tensor scales take 383 us with the heads one after another in one plane, 321 so;
// 64 ragged 16-bit ones 389 and 378), and for wide trees the
// same keys, the second time from L2. Where so many planes leave too many CTA
// slots over, a plane takes all heads, one after another. Cut units are merged
// by a second kernel.
#include "pod_tree_planner.hpp"

#include <string.h>

#include <algorithm>

#include "../../include/pod.h"
#include "pod_tree.h"

namespace {

// price of starting a segment, and least keys of a CTA's share, in keys
constexpr int kStartKeys = 192, kMinKeys = 320;
// Units stay whole where the longest is at most this many keys more than the cut
// share, for the merge is a second launch: 3 us in a graph, 6 us in a stream,
// about 1 us for each 100 keys that a lone CTA works through.
constexpr int kWholeKeys = 384;

struct Unit {
  int req, g, mt, blocks;
};

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Walks one plane with a CTA budget of `share` (units are not cut with `whole`);
// calls emit(cta, unit, blk0, blk1) for each segment. Returns the number of CTAs
// used.
template <typename F>
int cut(const std::vector<Unit>& units, int share, bool whole, int kStart, F emit) {
  int cta = 0, used = 0;
  for (size_t u = 0; u < units.size(); ++u) {
    int at = 0;
    while (at < units[u].blocks) {
      const int left = units[u].blocks - at;
      int room = share - used - kStart;
      // too little room to be worth a start: the next CTA begins here
      if (room < 1 || (room < left && used > 0 && (whole || room < 3))) {
        ++cta;
        used = 0;
        room = share - kStart;
      }
      const int take = std::min(left, room);
      emit(cta, (int)u, at, at + take);
      used += kStart + take;
      at += take;
    }
  }
  return units.empty() ? 0 : cta + 1;
}

}  // namespace

int pod_tree_build_plan(const PodTreeArgs& a, PodTreePlanHost& o, std::string* err) {
  auto bad = [&](int code, const std::string& m) {
    *err = m;
    return code;
  };
  const int INV = POD_ERR_INVALID_ARG, UNS = POD_ERR_UNSUPPORTED;
  if (a.batch < 0) return bad(INV, "batch is negative");
  if (a.H < 1 || a.Hk < 1 || a.H % a.Hk != 0)
    return bad(INV, "num_qo_heads must be a positive multiple of num_kv_heads");
  if (a.H > 65536 || a.Hk > 4096) return bad(UNS, "too many heads");
  if (a.d != 64 && a.d != 128 && a.d != 256) return bad(UNS, "head_dim must be 64, 128 or 256");
  if (a.ps < 1 || a.ps > (1 << 20)) return bad(INV, "page_size must be in [1, 2^20]");
  if (a.num_pages < 1 && a.batch > 0) return bad(INV, "the page pool is empty");
  if (a.num_pages >= (1 << 30)) return bad(INV, "the page pool is too large");
  if (a.batch > 0 && (!a.q_indptr || !a.kv_indptr || !a.last_page_len))
    return bad(INV, "a page table array is NULL");
  o.batch = a.batch; o.num_pages = a.num_pages; o.H = a.H; o.Hk = a.Hk; o.G = a.H / a.Hk;
  o.d = a.d; o.ps = a.ps;

  std::vector<int> n(a.batch), kv(a.batch);
  std::vector<long long> bit0(a.batch);
  if (a.batch > 0 && (a.q_indptr[0] != 0 || a.kv_indptr[0] != 0)) return bad(INV, "an indptr does not start at 0");
  // (all of them before a page is looked at: kv_indices ends where kv_indptr does)
  for (int r = 0; r < a.batch; ++r)
    if (a.q_indptr[r + 1] < a.q_indptr[r] || a.kv_indptr[r + 1] < a.kv_indptr[r])
      return bad(INV, "request " + std::to_string(r) + ": an indptr decreases");
  for (int r = 0; r < a.batch; ++r) {
    const std::string who = "request " + std::to_string(r) + ": ";
    const long long nq = (long long)a.q_indptr[r + 1] - a.q_indptr[r];
    const long long np = (long long)a.kv_indptr[r + 1] - a.kv_indptr[r];
    if (np > 0 && (a.last_page_len[r] < 1 || a.last_page_len[r] > a.ps))
      return bad(INV, who + "last_page_len is outside [1, page_size]");
    const long long len = np > 0 ? (np - 1) * a.ps + a.last_page_len[r] : 0;
    if (len > (1ll << 30)) return bad(INV, who + "more than 2^30 keys");   // (key numbers stay below 2^31 in the kernels)
    if (nq > len) return bad(INV, who + "the tree's tokens must be in the cache (kv_len >= q_len)");
    if (nq * o.G > 0x7fffff00ll) return bad(INV, who + "too many query rows");
    if (np > 0 && !a.kv_indices) return bad(INV, "kv_indices is NULL");
    for (int p = a.kv_indptr[r]; p < a.kv_indptr[r + 1]; ++p)
      if (a.kv_indices[p] < 0 || a.kv_indices[p] >= a.num_pages)
        return bad(INV, who + "a page index is outside the pool");
    n[r] = (int)nq;
    kv[r] = (int)len;
    bit0[r] = o.mask_bits;
    o.mask_bits += nq * nq;
  }
  o.rows = a.batch ? a.q_indptr[a.batch] : 0;
  if ((long long)o.rows * a.H > (1ll << 40)) return bad(INV, "too many query rows");
  const int npages = a.batch ? a.kv_indptr[a.batch] : 0;
  o.pages.assign(a.kv_indices ? a.kv_indices : nullptr, a.kv_indices ? a.kv_indices + npages : nullptr);

  const int kStart = (kStartKeys + a.block - 1) / a.block, kMinCut = (kMinKeys + a.block - 1) / a.block;
  // planes of units, and the smallest equal share that the CTA slots allow
  int max_mt = 0;
  for (int r = 0; r < a.batch; ++r)
    max_mt = std::max(max_mt, (int)(((long long)n[r] * o.G + POD_TREE_TILE - 1) / POD_TREE_TILE));
  using Planes = std::vector<std::vector<Unit>>;
  long long cost = 0, longest = 0;
  auto planes_of = [&](bool by_head) {
    Planes planes((size_t)max_mt * (by_head ? a.Hk : 1));
    cost = longest = 0;
    for (int mt = 0; mt < max_mt; ++mt)
      for (int r = 0; r < a.batch; ++r) {
        if ((long long)n[r] * o.G <= (long long)mt * POD_TREE_TILE) continue;
        const int blocks = (kv[r] + a.block - 1) / a.block;
        for (int g = 0; g < a.Hk; ++g)
          planes[by_head ? (size_t)mt * a.Hk + g : mt].push_back({r, g, mt, blocks});
        cost += (long long)a.Hk * (blocks + kStart);
        longest = std::max(longest, (long long)blocks);
      }
    return planes;
  };
  auto share_of = [&](const Planes& planes) {
    auto ctas = [&](int share) {
      long long c = 0;
      for (auto& p : planes) c += cut(p, share, false, kStart, [](int, int, int, int) {});
      return c;
    };
    const long long most = 1 << 29, even = cost / std::max(1, a.slots);
    int lo = (int)std::min(std::max(even, (long long)kMinCut + kStart), most);
    int hi = (int)std::max((long long)lo, std::min(cost + kStart + 1, most));
    if (ctas(lo) <= a.slots) return lo;
    while (lo + 1 < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (ctas(mid) <= a.slots) hi = mid;
      else lo = mid;
    }
    // (a plane is one CTA at least: with more planes than slots the CTAs run in
    // waves, and the balanced share is taken)
    return ctas(hi) <= a.slots ? hi : (int)std::min(std::max(even, longest + kStart), most);
  };
  Planes planes = planes_of(false);
  int share = share_of(planes);
  if (a.Hk > 1 && (long long)max_mt * a.Hk <= a.slots) {
    Planes by_head = planes_of(true);
    const int s = share_of(by_head);
    if (s <= share + share / 32) {       // up to 3 % more work a CTA
      planes = std::move(by_head);
      share = s;
    }
  }

  bool whole = false;
  if (!planes.empty() && (longest + kStart - share) * a.block <= kWholeKeys) {
    const int all = (int)std::max<long long>(longest + kStart, share);
    long long c = 0;
    for (auto& p : planes) c += cut(p, all, true, kStart, [](int, int, int, int) {});
    if (c <= a.slots) {
      share = all;
      whole = true;
    }
  }

  // segments in CTA order; split tiles get partial rows and a merge group
  struct Seg {
    int cta, unit, b0, b1;
  };
  std::vector<int32_t> rec, few;
  o.cta_ptr.assign(1, 0);
  long long prows = 0;
  for (const auto& plane : planes) {
    std::vector<Seg> s;
    cut(plane, share, whole, kStart, [&](int c, int u, int b0, int b1) { s.push_back({c, u, b0, b1}); });
    for (size_t i = 0; i < s.size();) {
      size_t e = i;
      while (e < s.size() && s[e].unit == s[i].unit) ++e;
      const Unit& un = plane[s[i].unit];
      const int rows = std::min(POD_TREE_TILE, n[un.req] * o.G - un.mt * POD_TREE_TILE);
      const int pieces = (int)(e - i);
      if (pieces > 1) {
        const int32_t g[TG_REC] = {un.g, un.mt * POD_TREE_TILE, rows, (int32_t)prows, pieces, a.q_indptr[un.req], 0, 0};
        std::vector<int32_t>& to = pieces > POD_TREE_FEW ? o.groups : few;
        to.insert(to.end(), g, g + TG_REC);
      }
      for (size_t j = i; j < e; ++j) {
        int32_t r[TS_REC] = {};
        r[TS_G] = un.g;
        r[TS_ROW0] = un.mt * POD_TREE_TILE;
        r[TS_NROWS] = rows;
        r[TS_BLK0] = s[j].b0;
        r[TS_BLK1] = s[j].b1;
        r[TS_PROW] = pieces > 1 ? (int32_t)prows : -1;
        r[TS_KVLEN] = kv[un.req];
        r[TS_NTOK] = n[un.req];
        r[TS_QROW0] = a.q_indptr[un.req];
        r[TS_PAGE0] = a.kv_indptr[un.req];
        r[TS_NPAGES] = a.kv_indptr[un.req + 1] - a.kv_indptr[un.req];
        r[TS_BIT_LO] = (int32_t)(uint32_t)(bit0[un.req] & 0xffffffffll);
        r[TS_BIT_HI] = (int32_t)(bit0[un.req] >> 32);
        r[TS_COPIES] = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
        if (pieces > 1) prows += rows;
        rec.insert(rec.end(), r, r + TS_REC);
        const bool last = j + 1 == s.size() || s[j + 1].cta != s[j].cta;
        if (last) o.cta_ptr.push_back((int32_t)(rec.size() / TS_REC));
      }
      i = e;
    }
  }
  // groups of many pieces first, then those of a few
  o.n_big = (int)(o.groups.size() / TG_REC);
  o.groups.insert(o.groups.end(), few.begin(), few.end());
  if (prows > 0x7fffffff) return bad(INV, "too many split rows");
  o.segs = std::move(rec);
  o.n_cta = (int)o.cta_ptr.size() - 1;
  o.n_prows = (int)prows;

  size_t at = TREE_ST_INTS * sizeof(int32_t);
  auto put = [&](size_t bytes) {
    const size_t r = up256(at);
    at = r + bytes;
    return r;
  };
  o.off_segs = put(o.segs.size() * 4);
  o.off_cta = put(o.cta_ptr.size() * 4);
  o.off_pages = put(o.pages.size() * 4);
  o.off_groups = put(o.groups.size() * 4);
  o.image.assign(up256(at), 0);
  auto copy = [&](size_t off, const std::vector<int32_t>& v) {
    if (!v.empty()) memcpy(o.image.data() + off, v.data(), v.size() * 4);
  };
  copy(o.off_segs, o.segs);
  copy(o.off_cta, o.cta_ptr);
  copy(o.off_pages, o.pages);
  copy(o.off_groups, o.groups);
  o.off_part_o = put((size_t)o.n_prows * a.d * 4);
  o.off_part_lse = put((size_t)o.n_prows * 4);
  o.total = up256(at);
  return POD_OK;
}
