// pod_tree.cuh — attention of drafted token trees over a paged cache (sm_103a).
//
// Mathematics. Request r has n drafted tokens, the last n of its kv_len keys.
// Token i sees every context key t < kv_len - n and drafted key j where the
// tree mask's bit (i, j) is set; out = softmax(s q.k) v over the visible keys,
// base-2 LSE. One pass with a running maximum m and sum l per row, in fp32:
//   p = 2^(x - m), l = l 2^(m' - m) + sum p, O = O 2^(m' - m) + P V.
//
// A tile is one KV head's 128 packed rows (tokens x query heads); every key
// loaded serves them all. Warp roles of a CTA (256 threads, two CTAs per SM,
// one at head_dim 256):
//   warps 0-3  one TMEM lane (row) per thread: Q into shared memory, then per
//              64-key block tcgen05.ld of S, mask, softmax, P back into TMEM;
//              final output or fp32 partial;
//   warp 4     one thread issues tcgen05.mma: S = Q K^T (two S buffers), then
//              O += P V with P read from TMEM;
//   warp 5     K (FP8: K and V codes) as TMA boxes through the page table;
//   warp 6     V boxes (16-bit); FP8: warps 6 and 7 widen the codes to fp16.
//   Page sizes that are not a power of two of at least 8 are gathered with
//   cp.async by the loader warps.
//
// Few rows: a tile of at most 32 (64) rows is held 4 (2) times in the 128
// lanes, and copy c works on its own quarter (half) of every block's keys, with
// zeros in P elsewhere. The matrix unit does the same work, the softmax, which
// would cost 128 rows whatever their number, a quarter (half) of it; the copies
// are joined at the end like split key ranges.
//
// FP8 caches: E4M3 codes are exact in fp16, so both products run in fp16
// (P with 11 significant bits). A query row is scaled by the power of two that
// brings its largest value to [2^13, 2^14): exact down to 2^-27 of that value.
// Per-tensor scales are constants of the softmax and of the output. Block
// scales are powers of two per key: K's multiplies the key's column of S, V's
// the column of P relative to the largest V scale met so far (O is rescaled
// when that one grows, as for the running maximum).
#pragma once
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>
#include <mutex>
#include <type_traits>

#include "pod_device.cuh"
#include "pod_tree.h"

using namespace pod;

namespace {

constexpr int kTreeThreads = 256;
constexpr int BK = POD_TREE_BLOCK;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int KV>
struct TLayout {
  static constexpr int NKB = D / 64;
  static constexpr int QBLK = POD_TREE_TILE * 128;   // 128 rows x 64 elements
  static constexpr int KVBLK = BK * 128;             // 64 keys x 64 elements
  static constexpr int STAGE = NKB * KVBLK;          // one block of K or V, 16-bit
  static constexpr int NK = KV == 0 ? 3 : 2, NV = KV == 0 ? 2 : 1;
  static constexpr int RAW = BK * D;                 // one block of K or V codes
  static constexpr int NR = KV == 0 ? 0 : 2;         // raw ring (K and V codes)
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = NKB * QBLK;
  static constexpr int V_OFF = K_OFF + NK * STAGE;
  static constexpr int R_OFF = V_OFF + NV * STAGE;
  static constexpr int BAR_OFF = R_OFF + NR * 2 * RAW;
  // BAR_OFF + 0: barriers, +176: TMEM address, +180: abort flag, +192: block
  // factors of two blocks (K as floats, V as halves)
  static constexpr int FAC_OFF = BAR_OFF + 192;
  static constexpr int FAC_K = BK * 4, FAC_V = BK * 2;
  static constexpr int END = FAC_OFF + (KV == 2 ? 2 * (FAC_K + FAC_V) : 0);
  // The copies' join holds 32 output columns of the 128 lanes (16 KB) in the Q
  // region, and m and l of the lanes behind them (at head_dim 64 Q has no room
  // for these).
  static constexpr int JOIN = 32;
  static constexpr int JOIN_BYTES = POD_TREE_TILE * JOIN * 4;
  static constexpr int ML_OFF = NKB > 1 ? Q_OFF + JOIN_BYTES : END;
  static constexpr int TOTAL = NKB > 1 ? END : END + POD_TREE_TILE * 8;
  static constexpr int TM_S = 0, TM_O = 2 * BK;
  static constexpr int TMEM_COLS = TM_O + D <= 256 ? 256 : 512;
  static_assert(JOIN_BYTES <= NKB * QBLK, "the join must fit the Q region");
};

enum {
  TB_QFULL = 0,
  TB_KFULL = 1,    // [3]
  TB_KEMPTY = 4,   // [3]
  TB_VFULL = 7,    // [2]
  TB_VEMPTY = 9,   // [2]
  TB_SFULL = 11,   // [2]
  TB_PFULL = 13,   // [2]
  TB_PVDONE = 15,  // [2]
  TB_RFULL = 17,   // [2]
  TB_REMPTY = 19,  // [2]
  TB_FINAL = 21,
  TB_COUNT = 22
};

// W (16, 32 or 64) consecutive TMEM columns of the warp's 32 lanes
template <int W>
POD_DEV void tmem_ldw(uint32_t a, float* v);
template <>
POD_DEV void tmem_ldw<64>(uint32_t a, float* v) { tmem_ld64(a, v); }
template <>
POD_DEV void tmem_ldw<32>(uint32_t a, float* v) { tmem_ld32(a, v); }
template <>
POD_DEV void tmem_ldw<16>(uint32_t a, float* v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]),
        "=r"(u[15])
      : "r"(a)
      : "memory");
}
POD_DEV void tmem_st8(uint32_t a, const uint32_t* u) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

POD_DEV bool tree_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}
// Meetings of the four softmax warps. A warp whose wait ran out still comes to
// the next vote, where all of them leave together.
POD_DEV void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
POD_DEV bool softmax_vote(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// one lane of the converged warp, always the same
POD_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
POD_DEV uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
POD_DEV void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
POD_DEV void stsf(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }

POD_DEV void sts_half(uint32_t a, float v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(__half_as_ushort(__float2half_rn(v))) : "memory");
}
POD_DEV uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// exponent byte -> 2^(byte - 127), and 2^(byte - ref) for byte <= ref
POD_DEV float exp_byte(int b) { return b == 0 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)b << 23); }
POD_DEV float exp_below(int b, int ref) { return __uint_as_float((uint32_t)max(127 - (ref - b), 0) << 23); }

// Page-table view of one segment: the cache row of key t.
struct KeyAt {
  const int32_t* pages;
  int npages, ps, shift;
  POD_DEV int page(int t) const {
    const int i = shift >= 0 ? t >> shift : t / ps;
    return __ldg(pages + (i < npages ? i : npages - 1));
  }
  POD_DEV int slot(int t) const { return shift >= 0 ? t & (ps - 1) : t % ps; }
};

// ============================================================ softmax warps
// One segment for tiles held C times. Returns false when a wait ran out.
template <typename T, typename E, int D, int KV, int C>
__device__ bool tree_softmax(const PodTreeParams& P, uint8_t* smem, uint32_t tmem, const int32_t* seg,
                             int& sc0, volatile int* abort_flag) {
  using L = TLayout<D, KV>;
  constexpr int RB = 128 / C, W = BK / C;           // rows and columns of a copy
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem), bar0 = sbase + L::BAR_OFF;
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
  const int cp = tid / RB, rr = tid % RB;           // copy (uniform per warp) and row of the tile
  const int nrows = seg[TS_NROWS], kv_len = seg[TS_KVLEN], ntok = seg[TS_NTOK];
  const int blk0 = seg[TS_BLK0], nb = seg[TS_BLK1] - blk0;
  const int prow = seg[TS_PROW];
  const int G = P.G, H = P.H, D8 = D / 8;
  const bool valid = rr < nrows;
  const int packed = seg[TS_ROW0] + (valid ? rr : 0);
  const int tok = packed / G, head = seg[TS_G] * G + packed % G;
  const size_t grow = (size_t)(seg[TS_QROW0] + tok) * H + head;

  // ---- Q row into shared memory (every MMA of the last segment has finished
  // with it: its last S has been read)
  float qscale = P.scale_log2;
  {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(P.q) + grow * D);
    float up = 1.f;
    if constexpr (KV != 0) {
      float amax = 0.f;
#pragma unroll 4
      for (int c = 0; c < D8; ++c) {
        const uint4 v = __ldg(src + c);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Pack<T>::unpack(u[i]);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      // 2^e with amax * 2^e in [2^13, 2^14), the factor kept a normal float
      const int ex = (int)(__float_as_uint(amax) >> 23);      // biased exponent
      int e = 13 - (ex - 127);
      e = amax > 0.f ? min(max(e, -126), 126) : 0;
      up = __uint_as_float((uint32_t)(127 + e) << 23);
      qscale *= __uint_as_float((uint32_t)(127 - e) << 23);
    }
#pragma unroll 4
    for (int c = 0; c < D8; ++c) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (valid) v = __ldg(src + c);
      if constexpr (KV != 0) {
        uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Pack<T>::unpack(u[i]);
          u[i] = Pack<__half>::two(f.x * up, f.y * up);
        }
        v = make_uint4(u[0], u[1], u[2], u[3]);
      }
      sts128(sbase + L::Q_OFF + (c >> 3) * L::QBLK + sw128_off(tid, c & 7), v);
    }
    fence_proxy_async();
    mbar_arrive(BAR(TB_QFULL));
  }

  const long long bit0 = ((long long)seg[TS_BIT_HI] << 32) | (uint32_t)seg[TS_BIT_LO];
  const int ctx = kv_len - ntok;
  KeyAt at{P.pages + seg[TS_PAGE0], seg[TS_NPAGES], P.ps, P.ps_shift};
  const uint32_t kfac0 = sbase + L::FAC_OFF, vfac0 = kfac0 + 2 * L::FAC_K;
  // block scales: this lane's exponent bytes of the next block (keys lane and
  // lane + 32; keys past the last read the last)
  int kb0 = 0, kb1 = 0, vb0 = 0, vb1 = 0, vref = 0;
  auto load_bytes = [&](int blk) {
    const int t0 = min(blk * BK + lane, kv_len - 1), t1 = min(blk * BK + 32 + lane, kv_len - 1);
    const size_t vstep = (size_t)P.ps * P.Hk;
    auto off = [&](int t) {
      const size_t p = (size_t)at.page(t) * 2 * vstep;
      return p + (P.hnd ? (size_t)seg[TS_G] * P.ps + at.slot(t) : (size_t)at.slot(t) * P.Hk + seg[TS_G]);
    };
    const size_t o0 = off(t0), o1 = off(t1);
    kb0 = __ldg(P.scales + o0);
    kb1 = __ldg(P.scales + o1);
    vb0 = __ldg(P.scales + o0 + vstep);
    vb1 = __ldg(P.scales + o1 + vstep);
  };
  if constexpr (KV == 2) load_bytes(blk0);

  const float NEG_INF = -INFINITY;
  float m_ref = NEG_INF, l = 0.f;
  bool ok = true;
  for (int j = 0; j < nb; ++j) {
    const int kb = (blk0 + j) * BK;
    const int sc = sc0 + j, b = sc & 1;
    float o_scale = 1.f;
    if constexpr (KV == 2) {
      const int top = __reduce_max_sync(0xffffffffu, max(vb0, vb1));
      if (top > vref) {                              // O is kept in units of 2^(vref - 127)
        o_scale = exp_below(vref, top);
        vref = top;
      }
      // warps 0 and 1 write the keys' factors. The warps meet once a block:
      // the factors of block j + 2 are written after the meeting of j + 1, which
      // every warp reaches after its reads of block j.
      if (warp < 2) {
        const int key = warp * 32 + lane, eb = warp ? kb1 : kb0, ev = warp ? vb1 : vb0;
        stsf(kfac0 + (j & 1) * L::FAC_K + 4 * key, exp_byte(eb));
        sts_half(vfac0 + (j & 1) * L::FAC_V + 2 * key, exp_below(ev, vref));
      }
      if (!softmax_vote(ok)) return false;
      if (j + 1 < nb) load_bytes(blk0 + j + 1);
    }
    if (!tree_wait(BAR(TB_SFULL + b), (sc >> 1) & 1, abort_flag)) {
      ok = false;
      if (KV == 2) continue;
      break;
    }
    tc_fence_after();
    const uint32_t s_addr = tmem + lane_base + L::TM_S + b * BK;
    float s[W];
    tmem_ldw<W>(s_addr + cp * W, s);
    if constexpr (KV == 2) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 f = lds128(kfac0 + (j & 1) * L::FAC_K + 4 * (cp * W + i));
        s[i] *= __uint_as_float(f.x);
        s[i + 1] *= __uint_as_float(f.y);
        s[i + 2] *= __uint_as_float(f.z);
        s[i + 3] *= __uint_as_float(f.w);
      }
    }
    const int c0 = kb + cp * W;                      // first key of this copy's columns
    if (c0 + W > ctx) {
      // keys of the tree, or past the last: bit i says whether key c0 + i is seen
      uint64_t see = 0;
      const int skip = max(ctx - c0, 0);             // context keys at the front
      const int j0 = c0 + skip - ctx;                // first tree key of the columns
      if (j0 < ntok) {
        see = P.mask ? load_bits64(P.mask, P.mask_bytes, bit0 + (long long)tok * ntok + j0)
                     : (tok - j0 >= 63 ? ~0ull : tok < j0 ? 0ull : (2ull << (tok - j0)) - 1ull);
        const int left = ntok - j0;
        if (left < 64) see &= (1ull << left) - 1ull;
      }
      if (skip) see = skip < 64 ? (see << skip) | ((1ull << skip) - 1ull) : ~0ull;
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (!((see >> i) & 1ull)) s[i] = NEG_INF;
    }
    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int i = 4; i < W; i += 8) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        mx[u] = i + 4 + u < W ? max3(mx[u], s[i + u], s[i + 4 + u]) : fmaxf(mx[u], s[i + u]);
    }
    const float bmax = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
    const float m_new = fmaxf(m_ref, bmax * qscale);
    const bool rescale = m_new > m_ref + 8.0f;       // also for the first finite maximum
    const float m_use = rescale ? m_new : m_ref;
    const float m_sub = m_use == NEG_INF ? 0.f : m_use;
    float rs = 0.f;
    uint32_t pk[W / 2];
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const float e0 = ex2(fmaf(s[i], qscale, -m_sub)), e1 = ex2(fmaf(s[i + 1], qscale, -m_sub));
      const float e2 = ex2(fmaf(s[i + 2], qscale, -m_sub)), e3 = ex2(fmaf(s[i + 3], qscale, -m_sub));
      rs += (e0 + e1) + (e2 + e3);
      pk[i / 2] = Pack<E>::two(e0, e1);
      pk[i / 2 + 1] = Pack<E>::two(e2, e3);
    }
    if constexpr (KV == 2) {
#pragma unroll
      for (int i = 0; i < W; i += 8) {               // (exact, down to fp16's subnormals)
        const uint4 f = lds128(vfac0 + (j & 1) * L::FAC_V + 2 * (cp * W + i));
        pk[i / 2] = hmul2_u32(pk[i / 2], f.x);
        pk[i / 2 + 1] = hmul2_u32(pk[i / 2 + 1], f.y);
        pk[i / 2 + 2] = hmul2_u32(pk[i / 2 + 2], f.z);
        pk[i / 2 + 3] = hmul2_u32(pk[i / 2 + 3], f.w);
      }
    }
    const bool need = (rescale && m_ref != NEG_INF) || (KV == 2 && o_scale != 1.f);
    if (j > 0 && __any_sync(0xffffffffu, need)) {
      // O holds P V up to the last block: wait for it, then rescale in TMEM
      const int sp = sc - 1;
      if (!tree_wait(BAR(TB_PVDONE + (sp & 1)), (sp >> 1) & 1, abort_flag)) {
        ok = false;
        if (KV == 2) continue;
        break;
      }
      tc_fence_after();
      const float a_m = rescale && m_ref != NEG_INF ? ex2(m_ref - m_use) : 1.f;
      const float alpha = a_m * o_scale;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(tmem + lane_base + L::TM_O + c, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= alpha;
        tmem_st32(tmem + lane_base + L::TM_O + c, o);
      }
      l *= a_m;
    }
    m_ref = m_use;
    l += rs;
    // P over the first 32 columns of S: this copy's keys, zeros for the others'
    if constexpr (C == 1) {
      tmem_st32u(s_addr, pk);
    } else {
      const uint32_t zero[8] = {};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if constexpr (C == 4) tmem_st8(s_addr + 8 * c, c == cp ? pk : zero);
        else tmem_st8(s_addr + 8 * c, (c >> 1) == cp ? pk + 8 * (c & 1) : zero);
      }
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(BAR(TB_PFULL + b));
  }
  if (ok) {
    const int sl = sc0 + nb - 1;
    ok = tree_wait(BAR(TB_PVDONE + (sl & 1)), (sl >> 1) & 1, abort_flag);
  }
  if (C > 1 || KV == 2) ok = softmax_vote(ok);
  if (!ok) return false;
  tc_fence_after();
  sc0 += nb;

  // ---- output: final rows, or partial rows of a split tile
  float v_scale = P.v_scale;
  if constexpr (KV == 2) v_scale = exp_byte(vref);
  T* __restrict__ outg = static_cast<T*>(P.out);
  if constexpr (C == 1) {
    float denom = l;
    if (P.sinks && prow < 0) denom += ex2(P.sinks[head] * kLog2e - m_ref);
    const float inv = denom == 0.f ? 0.f : v_scale / denom;   // (a NaN row stays NaN)
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tmem_ld32(tmem + lane_base + L::TM_O + c, o);
      if (!valid) continue;
      if (prow < 0) {
        T* dst = outg + grow * D + c;
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          *reinterpret_cast<uint4*>(dst + i) =
              make_uint4(Pack<T>::two(o[i] * inv, o[i + 1] * inv), Pack<T>::two(o[i + 2] * inv, o[i + 3] * inv),
                         Pack<T>::two(o[i + 4] * inv, o[i + 5] * inv), Pack<T>::two(o[i + 6] * inv, o[i + 7] * inv));
      } else {
        float* dst = P.part_o + (size_t)(prow + rr) * D + c;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4*>(dst + i) = make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
      }
    }
    if (valid) {
      const float lse = l == 0.f ? NEG_INF : m_ref + log2f(l);
      if (prow < 0) {
        if (P.lse) P.lse[grow] = lse;
      } else {
        P.part_lse[prow + rr] = lse;
      }
    }
  } else {
    // join the copies through the Q region, JOIN columns at a time
    float* ml = reinterpret_cast<float*>(smem + L::ML_OFF);
    ml[2 * tid] = m_ref;
    ml[2 * tid + 1] = l;
    constexpr int CH = L::JOIN / 4;                  // 16-byte chunks of a lane's part
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += L::JOIN) {
      softmax_sync();                                // the last part has been read
#pragma unroll 1
      for (int c = 0; c < L::JOIN; c += 32) {
        float o[32];
        tmem_ld32(tmem + lane_base + L::TM_O + c0 + c, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // (chunks turned by the lane: eight lanes of a store meet eight bank groups)
          const int ch = (c / 4 + i + tid) & (CH - 1);
          sts128(sbase + L::Q_OFF + tid * (CH * 16) + ch * 16, *reinterpret_cast<uint4*>(o + 4 * i));
        }
      }
      softmax_sync();
      for (int idx = tid; idx < nrows * CH; idx += 128) {
        const int r = idx / CH, ch = idx - r * CH;
        float M = NEG_INF;
#pragma unroll
        for (int c = 0; c < C; ++c) M = fmaxf(M, ml[2 * (c * RB + r)]);
        const float Ms = M == NEG_INF ? 0.f : M;
        float wsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int ln = c * RB + r;
          const float w = ex2(ml[2 * ln] - Ms);
          wsum += w * ml[2 * ln + 1];
          const uint4 u = lds128(sbase + L::Q_OFF + ln * (CH * 16) + ((ch + ln) & (CH - 1)) * 16);
          acc.x = fmaf(w, __uint_as_float(u.x), acc.x);
          acc.y = fmaf(w, __uint_as_float(u.y), acc.y);
          acc.z = fmaf(w, __uint_as_float(u.z), acc.z);
          acc.w = fmaf(w, __uint_as_float(u.w), acc.w);
        }
        const int pr = seg[TS_ROW0] + r;
        const int hd = seg[TS_G] * G + pr % G;
        const size_t gr = (size_t)(seg[TS_QROW0] + pr / G) * H + hd;
        float denom = wsum;
        if (P.sinks && prow < 0) denom += ex2(P.sinks[hd] * kLog2e - Ms);
        const float inv = denom == 0.f ? 0.f : v_scale / denom;
        const int col = c0 + ch * 4;
        if (prow < 0)
          *reinterpret_cast<uint2*>(outg + gr * D + col) =
              make_uint2(Pack<T>::two(acc.x * inv, acc.y * inv), Pack<T>::two(acc.z * inv, acc.w * inv));
        else
          *reinterpret_cast<float4*>(P.part_o + (size_t)(prow + r) * D + col) =
              make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (col == 0) {
          const float lse = wsum == 0.f ? NEG_INF : M + log2f(wsum);
          if (prow < 0) {
            if (P.lse) P.lse[gr] = lse;
          } else {
            P.part_lse[prow + r] = lse;
          }
        }
      }
    }
    softmax_sync();                                  // the Q region is free again
  }
  tc_fence_before();
  return true;
}

// ============================================================ the kernel
template <typename T, int D, int KV>
__global__ void __launch_bounds__(kTreeThreads, D == 256 ? 1 : 2)
    pod_tree_kernel(const __grid_constant__ PodTreeParams P) {
  using L = TLayout<D, KV>;
  using E = typename std::conditional<KV == 0, T, __half>::type;   // operand type of the MMAs
  extern __shared__ __align__(1024) uint8_t smem[];
  // the merge kernel may be scheduled now; it waits for this grid's completion
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (uniform, and known to be)
  const uint32_t sbase = smem_u32(smem), bar0 = sbase + L::BAR_OFF;
  static_assert(TB_COUNT * 8 <= 176, "barriers overlap the TMEM slot");
  if ((sbase & 1023u) != 0u) {                       // 128B-swizzle atoms need 1024-byte alignment
    if (tid == 0) atomicOr(P.status, POD_STATUS_ALIGN);
    return;
  }
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::BAR_OFF + 180);
  if (warp == 4) {
    tmem_alloc(sbase + L::BAR_OFF + 176, L::TMEM_COLS);
    tmem_relinquish();
  }
  const bool tma = P.kbx > 0;
  if (tid == 0) {
    const uint32_t load16 = tma ? 1u : 96u;          // gather: three warps
    mbar_init(BAR(TB_QFULL), 128);
    for (int s = 0; s < 3; ++s) {
      mbar_init(BAR(TB_KFULL + s), KV == 0 ? load16 : 64u);
      mbar_init(BAR(TB_KEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(BAR(TB_VFULL + s), KV == 0 ? load16 : 64u);
      mbar_init(BAR(TB_VEMPTY + s), 1);
      mbar_init(BAR(TB_SFULL + s), 1);
      mbar_init(BAR(TB_PFULL + s), 128);
      mbar_init(BAR(TB_PVDONE + s), 1);
      mbar_init(BAR(TB_RFULL + s), tma ? 1u : 32u);
      mbar_init(BAR(TB_REMPTY + s), 64);
    }
    mbar_init(BAR(TB_FINAL), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::BAR_OFF + 176);
  const int seg0 = P.cta_ptr[blockIdx.x], seg1 = P.cta_ptr[blockIdx.x + 1];
  bool ok = true;
  volatile int never = 0;                            // an abort flag that nobody raises

  if (warp < 4) {
    int sc0 = 0;
    for (int i = seg0; i < seg1 && ok; ++i) {
      const int32_t* seg = P.segs + (size_t)i * TS_REC;
      const int copies = seg[TS_COPIES];
      ok = copies == 4   ? tree_softmax<T, E, D, KV, 4>(P, smem, tmem, seg, sc0, abort_flag)
           : copies == 2 ? tree_softmax<T, E, D, KV, 2>(P, smem, tmem, seg, sc0, abort_flag)
                         : tree_softmax<T, E, D, KV, 1>(P, smem, tmem, seg, sc0, abort_flag);
    }
  } else if (warp == 4) {
    // ---------------------------------------------------------- MMA issuer
    // Per segment: QK_0, [QK_1, PV_0], ..., PV_{nb-1}. QK_{j+2} reuses the
    // columns of S_j / P_j; MMAs issued by one thread run in order. The whole
    // warp walks the loop and one elected lane issues: addresses and
    // descriptors then stay in uniform registers (a loop under `lane == 0`
    // moved each of them there for every MMA: 85 clocks an instruction).
    const uint32_t id_qk = idesc_f16(Pack<E>::kBF16, 128, BK, false, false);
    const uint32_t id_pv = idesc_f16(Pack<E>::kBF16, 128, D, false, true);
    // V stage: 16-key steps inside a box of vb keys ([box][64-column part][key])
    const int vb = KV == 0 && tma ? P.kbx : BK;
    const uint32_t v_box = (uint32_t)(vb * L::NKB * 128);
    const uint64_t v_desc0 = sdesc_sw128(sbase + L::V_OFF, (uint32_t)vb * 128u,
                                         vb >= 16 ? 1024u : (uint32_t)L::NKB * 1024u);
    uint32_t v_step[BK / 16];
#pragma unroll
    for (int k = 0; k < BK / 16; ++k) v_step[k] = (uint32_t)(k * 16 / vb) * v_box + (uint32_t)(k * 16 % vb) * 128u;
    const uint64_t q_desc0 = sdesc_sw128(sbase + L::Q_OFF, 16, 1024);
    const uint64_t k_desc0 = sdesc_sw128(sbase + L::K_OFF, 16, 1024);
    int ks = 0, vs = 0;                              // ring positions, and their phases
    uint32_t kph = 0, vph = 0;
    int sc0 = 0;
    for (int i = seg0; i < seg1 && ok; ++i) {
      const int32_t* seg = P.segs + (size_t)i * TS_REC;
      const int blk0 = seg[TS_BLK0], nb = seg[TS_BLK1] - blk0, kv_len = seg[TS_KVLEN];
      if (!tree_wait(BAR(TB_QFULL), (i - seg0) & 1, abort_flag)) { ok = false; break; }
      tc_fence_after();
      for (int j = 0; j <= nb; ++j) {
        if (j < nb) {
          if (!tree_wait(BAR(TB_KFULL + ks), kph, abort_flag)) { ok = false; break; }
          tc_fence_after();
          if (KV == 0 && !tma) fence_proxy_async();
          const int b = (sc0 + j) & 1;
          const uint32_t d_s = tmem + L::TM_S + b * BK;
          const uint64_t kd = k_desc0 + (uint32_t)(ks * L::STAGE >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_f16_ss(d_s, q_desc0 + (((k >> 2) * L::QBLK + (k & 3) * 32) >> 4),
                         kd + (((k >> 2) * L::KVBLK + (k & 3) * 32) >> 4), id_qk, k > 0 ? 1u : 0u);
            mma_commit(BAR(TB_SFULL + b));
            mma_commit(BAR(TB_KEMPTY + ks));
          }
          __syncwarp();
          if (++ks == L::NK) { ks = 0; kph ^= 1; }
        }
        if (j > 0) {
          const int sc = sc0 + j - 1, b = sc & 1;
          if (!tree_wait(BAR(TB_VFULL + vs), vph, abort_flag)) { ok = false; break; }
          if (!tree_wait(BAR(TB_PFULL + b), (sc >> 1) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          // 16-key steps past kv_len carry P = 0: skip them. Rows at or past
          // kv_len in the last step are unused slots of the last page, or
          // nothing: zero them, so that P = 0 never meets a non-finite value.
          const int keys = min(kv_len - (blk0 + j - 1) * BK, BK), ksteps = (keys + 15) >> 4;
          if (KV == 0 && (keys & 15)) {
            const uint32_t va = sbase + L::V_OFF + vs * L::STAGE;
            for (int x = lane; x < (ksteps * 16 - keys) * L::NKB * 8; x += 32) {
              const int r = keys + x / (L::NKB * 8), h = x / 8 % L::NKB, c = x % 8;
              sts128(va + (uint32_t)(r / vb) * v_box + h * vb * 128 + sw128_off(r % vb, c), make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async();
            __syncwarp();
          } else if (KV == 0 && !tma) {
            fence_proxy_async();
          }
          const uint64_t vd = v_desc0 + (uint32_t)(vs * L::STAGE >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              if (k < ksteps)
                mma_f16_ts(tmem + L::TM_O, tmem + L::TM_S + b * BK + k * 8, vd + (v_step[k] >> 4), id_pv,
                           (j > 1 || k > 0) ? 1u : 0u);
            mma_commit(BAR(TB_PVDONE + b));
            mma_commit(BAR(TB_VEMPTY + vs));
          }
          __syncwarp();
          if (++vs == L::NV) { vs = 0; vph ^= 1; }
        }
      }
      sc0 += nb;
    }
  } else if (KV == 0 && tma) {
    // ---------------------------------------------------------- K and V boxes
    if (warp < 7) {
      const bool is_v = warp == 6;
      const void* tm = is_v ? &P.tm_v : &P.tm_k;
      const int NS = is_v ? L::NV : L::NK;
      const int groups = BK / P.kbx, per = is_v ? 1 : L::NKB;     // boxes of a block: groups x per
      const int gi = lane / per, part = lane - gi * per;
      const bool mine = gi < groups;
      // keys are read once unless another tile of the request reads them too
      const uint64_t pol = l2_policy_evict_first();
      int fill = 0;
      if (lane == 0) tma_prefetch_desc(tm);
      for (int i = seg0; i < seg1 && ok; ++i) {
        const int32_t* seg = P.segs + (size_t)i * TS_REC;
        const int g = seg[TS_G], npages = seg[TS_NPAGES];
        const bool shared_keys = (long long)seg[TS_NTOK] * P.G > POD_TREE_TILE;
        const int32_t* pages = P.pages + seg[TS_PAGE0];
        const int b1 = seg[TS_BLK1];
        auto page_of = [&](int blk) {
          const int p = (blk * BK + gi * P.kbx) >> P.ps_shift;
          return mine && p < npages ? __ldg(pages + p) : P.num_pages;
        };
        int page = page_of(seg[TS_BLK0]);
        for (int blk = seg[TS_BLK0]; blk < b1; ++blk) {
          const int s = fill % NS;
          const int empty = (is_v ? TB_VEMPTY : TB_KEMPTY) + s, full = (is_v ? TB_VFULL : TB_KFULL) + s;
          if (!tree_wait(BAR(empty), ((fill / NS) & 1) ^ 1, abort_flag)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(BAR(full), (uint32_t)L::STAGE);
          __syncwarp();
          if (mine) {
            const int tin = (blk * BK + gi * P.kbx) & (P.ps - 1);
            const uint32_t dst = is_v ? sbase + L::V_OFF + s * L::STAGE + gi * P.kbx * L::NKB * 128
                                      : sbase + L::K_OFF + s * L::STAGE + part * L::KVBLK + gi * P.kbx * 128;
            // (a page past the request's last is out of the pool: TMA fills zeros)
            if (shared_keys)
              tma_load_5d(dst, tm, 0, tin, part, g, 2 * page + (is_v ? 1 : 0), BAR(full));
            else
              tma_load_5d_hint(dst, tm, 0, tin, part, g, 2 * page + (is_v ? 1 : 0), BAR(full), pol);
          }
          ++fill;
          if (blk + 1 < b1) page = page_of(blk + 1);
        }
      }
      // no copy is in flight when the CTA ends, also after an abort
      for (int f = max(fill - NS, 0); f < fill; ++f)
        tree_wait(BAR((is_v ? TB_VFULL : TB_KFULL) + f % NS), (f / NS) & 1, &never);
    }
  } else if (KV == 0) {
    // ---------------------------------------------------------- gather, 16-bit
    const int lt = tid - 160;                        // 0..95
    const T* __restrict__ kvg = static_cast<const T*>(P.kv);
    const size_t vstep = (size_t)P.ps * P.Hk * D;
    constexpr int CPR = D / 8, CH = BK * CPR;
    int fill = 0, vfill = 0;
    for (int i = seg0; i < seg1 && ok; ++i) {
      const int32_t* seg = P.segs + (size_t)i * TS_REC;
      const int g = seg[TS_G], kv_len = seg[TS_KVLEN], b1 = seg[TS_BLK1];
      KeyAt at{P.pages + seg[TS_PAGE0], seg[TS_NPAGES], P.ps, P.ps_shift};
      auto gather = [&](int blk, bool is_v, uint32_t dst) {
#pragma unroll 4
        for (int x = lt; x < CH; x += 96) {
          const int key = x / CPR, c = x - key * CPR, t = blk * BK + key;
          const int tt = t < kv_len ? t : kv_len - 1;
          const size_t page = (size_t)at.page(tt);
          const int slot = at.slot(tt);
          const T* src = kvg + (page * 2 * P.ps * P.Hk + (P.hnd ? (size_t)g * P.ps + slot : (size_t)slot * P.Hk + g)) * D +
                         (is_v ? vstep : 0) + c * 8;
          cp_async16(dst + (c >> 3) * L::KVBLK + sw128_off(key, c & 7), src, t < kv_len ? 16u : 0u);
        }
      };
      for (int blk = seg[TS_BLK0]; blk < b1; ++blk) {
        const int s = fill % L::NK;
        if (!tree_wait(BAR(TB_KEMPTY + s), ((fill / L::NK) & 1) ^ 1, abort_flag)) { ok = false; break; }
        gather(blk, false, sbase + L::K_OFF + s * L::STAGE);
        cp_async_mbar_arrive(BAR(TB_KFULL + s));
        ++fill;
        const int v = vfill % L::NV;
        if (!tree_wait(BAR(TB_VEMPTY + v), ((vfill / L::NV) & 1) ^ 1, abort_flag)) { ok = false; break; }
        gather(blk, true, sbase + L::V_OFF + v * L::STAGE);
        cp_async_mbar_arrive(BAR(TB_VFULL + v));
        ++vfill;
      }
    }
    cp_async_wait_all();
  } else if (warp == 5) {
    // ---------------------------------------------------------- FP8 codes, K and V
    const uint8_t* __restrict__ kvg = static_cast<const uint8_t*>(P.kv);
    const size_t vstep = (size_t)P.ps * P.Hk * D;
    const int groups = tma ? BK / P.kbx : 0;
    const int gi = lane >> 1, is_v = lane & 1;
    const bool mine = gi < groups;
    const uint64_t pol = l2_policy_evict_first();
    int fill = 0;
    for (int i = seg0; i < seg1 && ok; ++i) {
      const int32_t* seg = P.segs + (size_t)i * TS_REC;
      const int g = seg[TS_G], npages = seg[TS_NPAGES], kv_len = seg[TS_KVLEN], b1 = seg[TS_BLK1];
      const bool shared_keys = (long long)seg[TS_NTOK] * P.G > POD_TREE_TILE;
      KeyAt at{P.pages + seg[TS_PAGE0], npages, P.ps, P.ps_shift};
      auto page_of = [&](int blk) {
        const int p = (blk * BK + gi * P.kbx) >> P.ps_shift;
        return mine && p < npages ? __ldg(at.pages + p) : P.num_pages;
      };
      int page = tma ? page_of(seg[TS_BLK0]) : 0;
      for (int blk = seg[TS_BLK0]; blk < b1; ++blk) {
        const int s = fill % 2;
        if (!tree_wait(BAR(TB_REMPTY + s), ((fill / 2) & 1) ^ 1, abort_flag)) { ok = false; break; }
        const uint32_t dst = sbase + L::R_OFF + s * 2 * L::RAW;
        if (tma) {
          if (lane == 0) mbar_arrive_expect_tx(BAR(TB_RFULL + s), 2 * L::RAW);
          __syncwarp();
          if (mine) {
            const int tin = (blk * BK + gi * P.kbx) & (P.ps - 1);
            const uint32_t a = dst + is_v * L::RAW + gi * P.kbx * D;
            if (shared_keys) tma_load_4d(a, &P.tm_k, 0, tin, g, 2 * page + is_v, BAR(TB_RFULL + s));
            else tma_load_4d_hint(a, &P.tm_k, 0, tin, g, 2 * page + is_v, BAR(TB_RFULL + s), pol);
          }
          if (blk + 1 < b1) page = page_of(blk + 1);
        } else {
          constexpr int CPR = D / 16;
#pragma unroll 4
          for (int x = lane; x < BK * CPR; x += 32) {
            const int key = x / CPR, c = x - key * CPR, t = blk * BK + key;
            const int tt = t < kv_len ? t : kv_len - 1;
            const int slot = at.slot(tt);
            const uint8_t* src = kvg + ((size_t)at.page(tt) * 2 * P.ps * P.Hk +
                                        (P.hnd ? (size_t)g * P.ps + slot : (size_t)slot * P.Hk + g)) * D + c * 16;
            cp_async16(dst + key * D + c * 16, src, t < kv_len ? 16u : 0u);
            cp_async16(dst + L::RAW + key * D + c * 16, src + vstep, t < kv_len ? 16u : 0u);
          }
          cp_async_mbar_arrive(BAR(TB_RFULL + s));
        }
        ++fill;
      }
    }
    if (!tma) cp_async_wait_all();
    for (int f = max(fill - 2, 0); f < fill; ++f)    // no copy is in flight when the CTA ends
      tree_wait(BAR(TB_RFULL + f % 2), (f / 2) & 1, &never);
  } else if constexpr (KV != 0) {
    // ---------------------------------------------------------- widen the codes
    // Thread = key: its K row, then its V row, 16 codes at a time into the
    // swizzled fp16 stages. The chunk order is turned by the key, so the 8
    // lanes of a load or store phase meet different banks. V rows at or past
    // kv_len become zeros.
    const int key = tid - 192;
    int fill = 0;
    for (int i = seg0; i < seg1 && ok; ++i) {
      const int32_t* seg = P.segs + (size_t)i * TS_REC;
      const int kv_len = seg[TS_KVLEN], b1 = seg[TS_BLK1];
      for (int blk = seg[TS_BLK0]; blk < b1; ++blk) {
        const int r = fill % 2, s = fill % L::NK, v = fill % L::NV;
        if (!tree_wait(BAR(TB_RFULL + r), (fill / 2) & 1, abort_flag)) { ok = false; break; }
        const uint32_t raw = sbase + L::R_OFF + r * 2 * L::RAW + key * D;
        const bool live = blk * BK + key < kv_len;
        auto widen = [&](uint32_t src, uint32_t dst, bool keep) {
          constexpr int NCH = D / 16;
#pragma unroll
          for (int c = 0; c < NCH; ++c) {
            const int ch = (c + key) & (NCH - 1);
            uint4 w = lds128(src + ch * 16);
            if (!keep) w = make_uint4(0, 0, 0, 0);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t h[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              h[2 * q] = e4m3x2_to<__half>((uint16_t)(u[q] & 0xffffu));
              h[2 * q + 1] = e4m3x2_to<__half>((uint16_t)(u[q] >> 16));
            }
            const uint32_t part = dst + (ch >> 2) * L::KVBLK;
            const int c2 = (ch & 3) * 2;
            sts128(part + sw128_off(key, c2), make_uint4(h[0], h[1], h[2], h[3]));
            sts128(part + sw128_off(key, c2 + 1), make_uint4(h[4], h[5], h[6], h[7]));
          }
          fence_proxy_async();
        };
        if (!tree_wait(BAR(TB_KEMPTY + s), ((fill / L::NK) & 1) ^ 1, abort_flag)) { ok = false; break; }
        widen(raw, sbase + L::K_OFF + s * L::STAGE, true);
        mbar_arrive(BAR(TB_KFULL + s));
        if (!tree_wait(BAR(TB_VEMPTY + v), ((fill / L::NV) & 1) ^ 1, abort_flag)) { ok = false; break; }
        widen(raw + L::RAW, sbase + L::V_OFF + v * L::STAGE, live);
        mbar_arrive(BAR(TB_VFULL + v));
        mbar_arrive(BAR(TB_REMPTY + r));
        ++fill;
      }
    }
  }
  if (!ok) {
    *abort_flag = 1;
    if (lane == 0) atomicOr(P.status, POD_STATUS_TIMEOUT);
  }

  // ------------------------------------------------------------ teardown:
  // every MMA has finished before TMEM is given back
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    if (elect_one()) mma_commit(BAR(TB_FINAL));
    __syncwarp();
    mbar_wait(BAR(TB_FINAL), 0, &never);
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

template <typename T, int D, int KV>
cudaError_t launch_tree(const PodTreeParams& P, cudaStream_t stream) {
  constexpr int SMEM = TLayout<D, KV>::TOTAL;
  static_assert(SMEM <= (D == 256 ? 232448 : 115712), "shared memory of the CTAs on an SM");
  // the attributes belong to each device: set once per device
  static std::atomic<unsigned long long> done{0ull};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit == 0ull || !(done.load(std::memory_order_acquire) & bit)) {
    std::lock_guard<std::mutex> lock(mu);
    e = cudaFuncSetAttribute(pod_tree_kernel<T, D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(pod_tree_kernel<T, D, KV>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  pod_tree_kernel<T, D, KV><<<P.n_cta, kTreeThreads, SMEM, stream>>>(P);
  return cudaGetLastError();
}

template <int KV>
cudaError_t launch_tree_kv(const PodTreeParams& P, int dtype, int d, cudaStream_t st) {
  if (dtype == 1)
    return d == 64 ? launch_tree<__nv_bfloat16, 64, KV>(P, st)
           : d == 128 ? launch_tree<__nv_bfloat16, 128, KV>(P, st)
                      : launch_tree<__nv_bfloat16, 256, KV>(P, st);
  return d == 64 ? launch_tree<__half, 64, KV>(P, st)
         : d == 128 ? launch_tree<__half, 128, KV>(P, st)
                    : launch_tree<__half, 256, KV>(P, st);
}

}  // namespace
