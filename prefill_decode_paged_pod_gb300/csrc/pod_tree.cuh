// pod_tree.cuh — attention of drafted token trees over a paged cache (sm_103a).
//
// Mathematics. Request r has n drafted tokens, the last n of its kv_len keys.
// Token i sees every context key t < kv_len - n and drafted key j where the
// tree mask's bit (i, j) is set; out = softmax(s q.k) v over the visible keys,
// base-2 LSE. One pass with a running maximum m and sum l per row, in fp32:
//   p = 2^(x - m), l = l 2^(m' - m) + sum p, O = O 2^(m' - m) + P V.
//
// P is an operand of the matrix unit: for 16-bit caches it is rounded to the cache's
// type, off by 2^-8 (bf16) or 2^-11 of each weight; l sums it unrounded.
//
// A tile is one KV head's 128 packed rows (tokens x query heads); every key
// loaded serves them all. Warp roles of a CTA (256 threads, two CTAs per SM,
// one at head_dim 256):
//   warps 0-3  one TMEM lane (row) per thread: Q into shared memory, then per
//              key block tcgen05.ld of S, mask, softmax, P back into TMEM;
//              final output or fp32 partial;
//   warp 4     one lane issues tcgen05.mma: S = Q K^T, and O += P V with P read
//              from TMEM (double-buffered S: warp 7 issues these);
//   warp 5, 6  K and V as TMA boxes through the page table; page sizes that are
//              not a power of two of at least 8 are gathered by the other warps with
//              cp.async.
//
// Few rows: a tile of at most 32 (64) rows is held 4 (2) times in the 128
// lanes, and copy c works on its own quarter (half) of every block's keys, with
// zeros in P elsewhere. The matrix unit does the same work, the softmax, which
// would cost 128 rows whatever their number, a quarter (half) of it; the copies
// are joined at the end like split key ranges.
//
// FP8 caches go into the products as they are (kind::f8f6f4, E4M3 operands).
// A query row is scaled by the power of two that brings
// its largest value to [128, 256) and split into E4M3 parts, two for bf16 rows
// (4 + 4 significant bits, all it has), three for fp16 rows (11 bits); parts
// below 2^-17 of the row's largest value lose bits. P (the largest
// between 2^6 and 2^8.5) is carried in parts. bf16 results:
// two E4M3 parts, 4 bits and the fp16 remainder to 4 bits, at most 2^-9 + 2^-11 of
// p off, and 2^-15 of the largest weight at the bottom. fp16 results, by Veltkamp
// splitting: 4 bits in E4M3 and twice 3 bits in E5M2, whose range goes on below, 2^-12 of p and 2^-22 of the
// largest weight. (An
// earlier form widened the codes to fp16 in shared memory; the two warps that
// did it set the pace: 620 us for 96 requests of 8192 keys, now 412, and 321 with
// per-tensor scales.) These are constants of the softmax and of the output. Block scales are powers of
// two per key: K's multiplies the key's column of S, V's the column of P
// relative to the largest V scale met so far.
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
constexpr float kLog2e = 1.4426950408889634f;

template <typename T, int D, int KV>
struct TLayout {
  static constexpr bool F8 = KV != 0;
  static constexpr int BK = KV == 2 ? POD_TREE_BLOCKB : POD_TREE_BLOCK;   // keys per block
  static constexpr int ES = F8 ? 1 : 2;                // operand bytes
  static constexpr int ROWB = D * ES < 128 ? D * ES : 128;   // bytes of a row part
  static constexpr int PARTS = D * ES / ROWB;          // row parts
  static constexpr int PEL = ROWB / ES;                // elements of a row part
  static constexpr int QP = !F8 ? 1 : Pack<T>::kBF16 ? 2 : 3;   // precision parts of Q
  static constexpr int PP = QP;                        // parts of P
  static constexpr int QPART = POD_TREE_TILE * ROWB;   // one row part of one precision part
  static constexpr int KVPART = BK * ROWB;             // one row part of a block of K or V
  static constexpr int STAGE = PARTS * KVPART;
  static constexpr int NK = KV == 2 ? 2 : KV == 1 ? 4 : 3;
  static constexpr int NV = KV != 1 ? 2 : QP == 3 && D == 128 ? 3 : 4;
  static constexpr int Q_OFF = 0;
  static constexpr int Q_BYTES = QP * PARTS * QPART;
  static constexpr int K_OFF = Q_BYTES;
  static constexpr int V_OFF = K_OFF + NK * STAGE;
  static constexpr int BAR_OFF = V_OFF + NV * STAGE;
  // BAR_OFF + 0: barriers, +192: TMEM address, +196: abort flag, +200: the
  // warps' largest V exponents of two blocks, +240: the block's factors (K,
  // then V). One set for the CTA: a set for each warp would spare the meetings,
  // and a loader warp for the exponent bytes the loads, but both made the code
  // larger than the instruction cache and the loop slower (when the loop took 405 us
  // for 96 requests of 8192 keys: 409 and 430).
  static constexpr int WM_OFF = BAR_OFF + 200;
  static constexpr int FAC_OFF = BAR_OFF + 240;
  // (floats, or bf16 beside the three Q parts of fp16 rows of 128 elements, which
  // leave no room for more)
  static constexpr int FAC = QP == 3 && D == 128 ? 2 : 4;
  static constexpr int END = FAC_OFF + (KV == 2 ? 2 * BK * FAC : 0);
  // The copies' join goes through the Q region: first m and l of the 128 lanes,
  // then twice half of their output columns.
  static constexpr int JOIN = D / 2;
  static constexpr int TOTAL = END;
  static_assert(POD_TREE_TILE * JOIN * 4 <= Q_BYTES && POD_TREE_TILE * 8 <= Q_BYTES, "the join must fit the Q region");
  // TMEM: S buffers, then O. Two buffers let Q K^T of the next block run beside
  // the softmax of this one: 96 requests of 8192 keys with per-tensor scales took
  // 352 us in blocks of 128 keys with one, 326 in blocks of 64 with two. Block
  // scales cost the softmax warps a meeting a block, so these keep blocks of 128
  // (427 us; 487 with 64), which leave room for one where two CTAs share the SM.
  static constexpr int NSB = KV == 2 && D <= 128 ? 1 : 2;
  // (with two, warp 7 issues MMAs and two warps gather; else three)
  static constexpr int GW = NSB > 1 ? 2 : 3;
  static constexpr int TM_S = 0, TM_O = NSB * BK;
  static constexpr int TMEM_COLS = TM_O + D <= 256 ? 256 : 512;
  static_assert(TM_O + D <= 512 && (D > 128 || TMEM_COLS == 256), "TMEM columns");
  // MMA steps: 32 bytes of a K-major row, KSTEP keys of V
  static constexpr int DSTEPS = D * ES / 32, KSTEP = 32 / ES, KSTEPS = BK / KSTEP;
  // P = 2^(x - m): the reference m is set so that the largest P is 2^TOP, and
  // moves (O is rescaled) when one would pass 2^LIMIT. E4M3 ends at 448; TOP well
  // below it spares most of the rescaling (at TOP = 7 every other block of 128
  // random keys had a row that needed it).
  static constexpr float TOP = F8 ? 6.f : 0.f, LIMIT = F8 ? 8.5f : 8.f;
  // Block scales: where the V factors differ by no more binades, the largest logit
  // sets m, and the smallest parts of P stay at or below their rounding (2^-15 of
  // the largest weight beside 2^-9 of each; with three parts 2^-22 beside 2^-12).
  static constexpr int SPREAD = PP == 3 ? 10 : 6;

  static POD_DEV uint32_t swz(int r, int c) { return ROWB == 128 ? sw128_off(r, c) : sw64_off(r, c); }
  static POD_DEV uint64_t desc(uint32_t a, uint32_t lbo, uint32_t sbo) {
    return ROWB == 128 ? sdesc_sw128(a, lbo, sbo) : sdesc_sw64(a, lbo, sbo);
  }
};

enum {
  TB_QFULL = 0,
  TB_KFULL = 1,    // [4]
  TB_KEMPTY = 5,   // [4]
  TB_VFULL = 9,    // [4]
  TB_VEMPTY = 13,  // [4]
  TB_SFULL = 17,   // [2]
  TB_PFULL = 19,   // [2]
  TB_PVDONE = 21,  // [2]
  TB_FINAL = 23,
  TB_COUNT = 24
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
POD_DEV void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
POD_DEV void stsf(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
POD_DEV void sts16(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"((unsigned short)v) : "memory");
}
// bf16 of a power of two (exact, subnormals too): its upper 16 bits
POD_DEV uint32_t pow2_bf16(float v) { return __float_as_uint(v) >> 16; }

// x to BITS significant bits by Veltkamp splitting.
template <int BITS>
POD_DEV uint64_t head2(uint64_t x) {
  const float c = (float)((1 << (24 - BITS)) + 1);
  const uint64_t t = mul2(x, pack2(c, c));
  return add2(t, fma2(t, pack2(-1.f, -1.f), x));     // (products with -1 are exact)
}
// Four values below 448 (two pairs) in parts whose sum they are (byte i: value i):
// two E4M3 words (the second of the difference to the fp16 value), or (three parts)
// an E4M3 and two E5M2 words. Two parts by splitting in fp32, as the three are
// made, took 5 % longer over a block-scaled cache.
template <int PARTS>
POD_DEV void split4(uint64_t x01, uint64_t x23, uint32_t* w) {
  if constexpr (PARTS == 2) {
    float x[4];
    unpack2(x01, x[0], x[1]);
    unpack2(x23, x[2], x[3]);
    e4m3_hi_lo4(x[0], x[1], x[2], x[3], w[0], w[1]);
    return;
  }
  const uint64_t neg = pack2(-1.f, -1.f);
  const uint64_t x[2] = {x01, x23};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // below E4M3's normal range the head is a multiple of 2^-9, so that the code is
    // exactly it and the rest goes to the other parts
    const uint64_t v = add2(add2(head2<4>(x[i]), pack2(24576.f, 24576.f)), pack2(-24576.f, -24576.f));
    uint64_t r = fma2(v, neg, x[i]);
    const uint64_t m = head2<3>(r);
    r = fma2(m, neg, r);
    float a, b;
    unpack2(v, a, b);
    const uint32_t h = f32x2_to_e4m3x2(a, b);
    unpack2(m, a, b);
    const uint32_t l = f32x2_to_e5m2x2(a, b);
    unpack2(r, a, b);
    const uint32_t k = f32x2_to_e5m2x2(a, b);
    w[0] = i ? w[0] | (h << 16) : h;
    w[1] = i ? w[1] | (l << 16) : l;
    w[PARTS - 1] = i ? w[PARTS - 1] | (k << 16) : k;
  }
}

// exponent byte -> 2^(byte - 127), and 2^(byte - ref) for byte <= ref
POD_DEV float exp_byte(int b) { return b == 0 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)b << 23); }
POD_DEV float exp_below(int b, int ref) { return __uint_as_float((uint32_t)max(127 - (ref - b), 0) << 23); }

// Factors of keys key .. key + 3, as two pairs.
template <int FACB>
POD_DEV void factors4(uint32_t base, int key, uint64_t* f) {
  if constexpr (FACB == 4) {
    const uint4 v = lds128(base + 4 * key);
    f[0] = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
  } else {
    const uint2 v = ld_shared_v2(base + 2 * key);
    f[0] = pack2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    f[1] = pack2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
}

// Page-table view of one segment: the cache row (in rows of D elements, K) of
// key t (below kv_len) and KV head g.
struct KeyAt {
  const int32_t* pages;
  long long page_rows;                               // rows of a page, K and V
  int ps, shift, hk, hnd, g;
  POD_DEV int page(int t) const { return __ldg(pages + (shift >= 0 ? t >> shift : t / ps)); }
  POD_DEV int in_page(int t) const {
    const int slot = shift >= 0 ? t & (ps - 1) : t % ps;
    return hnd ? g * ps + slot : slot * hk + g;
  }
  POD_DEV long long row(int t, int page) const { return page * page_rows + in_page(t); }
};
POD_DEV KeyAt key_at(const PodTreeParams& P, const int32_t* seg) {
  return KeyAt{P.pages + seg[TS_PAGE0], P.page_rows, P.ps, P.ps_shift, P.Hk, P.hnd, seg[TS_G]};
}

// 64 bits of a packed array from bit `pos`; bytes at or past `nbytes` read as zero.
// (Plain loads, here and of Q: a kernel that starts beside the one before must not
// take what that one writes for constant.)
POD_DEV uint64_t tree_bits64(const uint8_t* m, long long nbytes, long long pos) {
  const long long b0 = pos >> 3;
  const int sh = (int)(pos & 7);
  uint64_t lo = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (b0 + k < nbytes) lo |= (uint64_t)m[b0 + k] << (8 * k);
  const uint64_t hi = b0 + 8 < nbytes ? (uint64_t)m[b0 + 8] : 0ull;
  return sh ? (lo >> sh) | (hi << (64 - sh)) : lo;
}

// What one row sees at the end of its request.
struct TreeView {
  const uint8_t* mask;
  long long mask_bytes, bit0;                        // the row's first bit
  int ctx, ntok, tok;
  // bit i says whether key c0 + i is seen
  POD_DEV uint64_t seen(int c0) const {
    uint64_t see = 0;
    const int skip = max(ctx - c0, 0);               // context keys at the front
    const int j0 = c0 + skip - ctx;                  // first tree key
    if (j0 < ntok) {
      see = mask ? tree_bits64(mask, mask_bytes, bit0 + j0)
                 : (tok - j0 >= 63 ? ~0ull : tok < j0 ? 0ull : (2ull << (tok - j0)) - 1ull);
      const int left = ntok - j0;
      if (left < 64) see &= (1ull << left) - 1ull;
    }
    if (skip) see = skip < 64 ? (see << skip) | ((1ull << skip) - 1ull) : ~0ull;
    return see;
  }
};

// Block scales: the row's largest logit + log2(V factor) over N columns of S (col0:
// the first one's place in the block, which starts at key kb). Rarely needed, and
// a call, so that the loop around it keeps its registers.
template <int FACB, int N>
__device__ __noinline__ float weighted_max(uint32_t s_addr, uint32_t kfac, uint32_t vfac, int col0, float qscale,
                                           int kb, const TreeView& tv) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < N; c += 16) {
    float x[16];
    tmem_ldw<16>(s_addr + c, x);
    const int c0 = kb + col0 + c;
    const uint64_t see = c0 + 16 > tv.ctx ? tv.seen(c0) : ~0ull;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      uint64_t k[2], v[2];
      factors4<FACB>(kfac, col0 + c + i, k);
      factors4<FACB>(vfac, col0 + c + i, v);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float s[2], g[2];
        unpack2(mul2(pack2(x[i + 2 * u], x[i + 2 * u + 1]), k[u]), s[0], s[1]);
        unpack2(v[u], g[0], g[1]);
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if ((see >> (i + 2 * u + w)) & 1ull)
            top = fmaxf(top, fmaf(s[w], qscale, (float)((int)(__float_as_uint(g[w]) >> 23) - 127)));
      }
    }
  }
  return top;
}

// ============================================================ softmax warps
// One segment for tiles held C times. Returns false when a wait ran out.
template <typename T, int D, int KV, int C>
__device__ bool tree_softmax(const PodTreeParams& P, uint8_t* smem, uint32_t tmem, const int32_t* seg,
                             int& sc0, volatile int* abort_flag) {
  using L = TLayout<T, D, KV>;
  constexpr int BK = L::BK, NSB = L::NSB;
  constexpr int RB = 128 / C;                        // rows of a copy
  constexpr int TW = BK / C;                         // its keys in a block,
  // in NH runs of W columns (FP8: what stays in registers beside the parts of P)
  constexpr int WM = L::F8 ? 32 : 64, W = TW < WM ? TW : WM, NH = TW / W;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem), bar0 = sbase + L::BAR_OFF;
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
  const int cp = tid / RB, rr = tid % RB;            // copy (uniform per warp) and row of the tile
  const int nrows = seg[TS_NROWS], kv_len = seg[TS_KVLEN], ntok = seg[TS_NTOK];
  const int blk0 = seg[TS_BLK0], nb = seg[TS_BLK1] - blk0;
  const int prow = seg[TS_PROW];
  const int G = P.G, H = P.H;
  const bool valid = rr < nrows;
  const int packed = seg[TS_ROW0] + (valid ? rr : 0);
  const int tok = packed / G, head = seg[TS_G] * G + packed % G;
  const size_t grow = (size_t)(seg[TS_QROW0] + tok) * H + head;

  // ---- Q row into shared memory (every MMA of the last segment has finished
  // with it: its last S has been read)
  float qscale = P.scale_log2;
  {
    // A warp brings its 32 lanes' rows together, D / 8 lanes a row: a thread that
    // reads its own row alone takes 16 bytes of a line at a time, and the 2048
    // line visits took 2700 clocks a segment.
    constexpr int LPQ = D / 8, RPI = 32 / LPQ;       // lanes of a row, rows at a time
    const int sub = lane / LPQ, ch = lane % LPQ;
    const uint32_t live = __ballot_sync(0xffffffffu, valid);
    int my_e = 0;
    constexpr int NI = 32 / RPI, GRP = L::F8 ? 4 : NI < 16 ? NI : 16;
    uint4 next[GRP];
    auto ask = [&](int i0) {                         // rows of iterations i0 .. i0 + GRP - 1
#pragma unroll
      for (int k = 0; k < GRP; ++k) {
        const int ln = (i0 + k) * RPI + sub;
        const size_t g = (size_t)__shfl_sync(0xffffffffu, (unsigned long long)grow, ln);
        next[k] = make_uint4(0, 0, 0, 0);
        if ((live >> ln) & 1) next[k] = reinterpret_cast<const uint4*>(static_cast<const T*>(P.q) + g * D)[ch];
      }
    };
    auto put = [&](int i, const uint4& v) {          // the rows of iteration i into shared memory
      const int row = warp * 32 + i * RPI + sub;
      if constexpr (!L::F8) {
        sts128(sbase + L::Q_OFF + (ch >> 3) * L::QPART + L::swz(row, ch & 7), v);
      } else {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        float x[8], amax = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = Pack<T>::unpack(u[k]);
          x[2 * k] = f.x;
          x[2 * k + 1] = f.y;
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int o = LPQ / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o, LPQ));
        // 2^e with amax * 2^e in [128, 256), both factors normal floats
        int e = 7 - ((int)(__float_as_uint(amax) >> 23) - 127);
        e = amax > 0.f ? min(max(e, -126), 126) : 0;
        // (a row with an infinity becomes NaN, as its logits are, not a saturated code)
        const float up = __uint_as_float(amax == INFINITY ? 0x7fffffffu : (uint32_t)(127 + e) << 23);
#pragma unroll
        for (int k = 0; k < RPI; ++k) {
          const int ek = __shfl_sync(0xffffffffu, e, k * LPQ);
          if (lane == i * RPI + k) my_e = ek;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= up;
        const int part = ch * 8 / L::ROWB, cc = ch * 8 % L::ROWB / 16;
#pragma unroll
        for (int p = 0; p < L::QP; ++p) {            // part p: what parts 0..p-1 left, to E4M3
          uint32_t w[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t code = f32x2_to_e4m3x2(x[2 * k], x[2 * k + 1]);
            w[k >> 1] |= code << (16 * (k & 1));
            const float2 f = Pack<__half>::unpack(e4m3x2_to<__half>((uint16_t)code));
            x[2 * k] -= f.x;
            x[2 * k + 1] -= f.y;
          }
          sts64(sbase + L::Q_OFF + (p * L::PARTS + part) * L::QPART + L::swz(row, cc) + (ch & 1) * 8, w[0], w[1]);
        }
      }
    };
    ask(0);
    // (FP8: four rows' worth of code, not the whole tile's: run once a segment, it
    // would come from beyond the instruction cache)
#pragma unroll 1
    for (int i0 = 0; i0 < NI; i0 += GRP) {
      uint4 vs[GRP];
#pragma unroll
      for (int k = 0; k < GRP; ++k) vs[k] = next[k];
      if (i0 + GRP < NI) ask(i0 + GRP);
#pragma unroll
      for (int k = 0; k < GRP; ++k) put(i0 + k, vs[k]);
    }
    if constexpr (L::F8) qscale *= __uint_as_float((uint32_t)(127 - my_e) << 23);
    fence_proxy_async();
    mbar_arrive(BAR(TB_QFULL));
  }

  const int ctx = kv_len - ntok;
  const TreeView tv{P.mask, P.mask_bytes,
                    (((long long)seg[TS_BIT_HI] << 32) | (uint32_t)seg[TS_BIT_LO]) + (long long)tok * ntok, ctx, ntok, tok};
  // block scales: the exponent bytes of this thread's key (tid) of the next
  // block, and its page of the one after (a byte's address waits for its page);
  // keys past the last read the last
  const uint32_t kfac = sbase + L::FAC_OFF, vfac = kfac + BK * L::FAC;
  int kbyte = 0, vbyte = 0, page = 0, vref = 0;
  const KeyAt at = key_at(P, seg);
  auto my_key = [&](int blk) { return min(blk * BK + tid, kv_len - 1); };
  auto load_bytes = [&](int blk) {
    const long long r = at.row(my_key(blk), page);
    kbyte = __ldg(P.scales + r);
    vbyte = __ldg(P.scales + r + (long long)P.ps * P.Hk);
    page = at.page(my_key(blk + 1));                 // (for the block after)
  };
  if constexpr (KV == 2) {
    page = at.page(my_key(blk0));
    load_bytes(blk0);
  }

  const float NEG_INF = -INFINITY;
  float m_ref = NEG_INF, l = 0.f;
  bool ok = true;
  for (int j = 0; j < nb; ++j) {
    const int kb = (blk0 + j) * BK;
    const int sc = sc0 + j, b = sc % NSB;
    float o_scale = 1.f;
    bool wide = false;                               // V factors of many binades
    if constexpr (KV == 2) {
      // The warps meet twice a block: at the first meeting all of them have read
      // the last block's factors and written their largest and smallest V
      // exponent, at the second the factors are there.
      volatile uint32_t* wm = reinterpret_cast<volatile uint32_t*>(smem + L::WM_OFF) + 4 * (j & 1);
      const int hi_w = __reduce_max_sync(0xffffffffu, vbyte), lo_w = __reduce_min_sync(0xffffffffu, vbyte);
      if (lane == 0) wm[warp] = (uint32_t)hi_w << 16 | (uint32_t)(255 - lo_w);
      if (!softmax_vote(ok)) return false;
      const uint32_t w4 = __vmaxu2(__vmaxu2(wm[0], wm[1]), __vmaxu2(wm[2], wm[3]));
      const int hi = (int)(w4 >> 16), lo = 255 - (int)(w4 & 0xffffu);
      if (hi > vref) {
        // O is kept in units of 2^(m_ref + vref): what vref gains m_ref loses,
        // as far as l, in units of 2^m_ref, keeps its range
        const int gain = hi - vref, room = max(100 - ((int)(__float_as_uint(l) >> 23 & 255u) - 127), 0);
        const int d = min(min(gain, room), 120);
        o_scale = exp_below(d, gain);
        m_ref -= (float)d;
        l *= __uint_as_float((uint32_t)(127 + d) << 23);
        vref = hi;
      }
      wide = vref - lo > L::SPREAD;
      if constexpr (L::FAC == 4) {
        stsf(kfac + 4 * tid, exp_byte(kbyte));
        stsf(vfac + 4 * tid, exp_below(vbyte, vref));
      } else {
        sts16(kfac + 2 * tid, pow2_bf16(exp_byte(kbyte)));
        sts16(vfac + 2 * tid, pow2_bf16(exp_below(vbyte, vref)));
      }
      if (j + 1 < nb) load_bytes(blk0 + j + 1);
      softmax_sync();
    }
    if (!tree_wait(BAR(TB_SFULL + b), (sc / NSB) & 1, abort_flag)) {
      ok = false;
      if (KV == 2) continue;
      break;
    }
    tc_fence_after();
    const uint32_t s_addr = tmem + lane_base + L::TM_S + b * BK;
    const int my0 = cp * TW;                         // this copy's first column
    // S of W columns: raw products with the keys' factors, hidden keys at -inf
    auto load_s = [&](int col, float* s) {
      tmem_ldw<W>(s_addr + col, s);
      if constexpr (KV == 2) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
          uint64_t f[2];
          factors4<L::FAC>(kfac, col + i, f);
          unpack2(mul2(pack2(s[i], s[i + 1]), f[0]), s[i], s[i + 1]);
          unpack2(mul2(pack2(s[i + 2], s[i + 3]), f[1]), s[i + 2], s[i + 3]);
        }
      }
      const int c0 = kb + col;                       // first key of the run
      if (c0 + W > ctx) {                            // keys of the tree, or past the last
        const uint64_t see = tv.seen(c0);
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (!((see >> i) & 1ull)) s[i] = NEG_INF;
      }
    };
    auto max_s = [&](const float* s) {
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int i = 4; i < W; i += 8) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          mx[u] = i + 4 + u < W ? max3(mx[u], s[i + u], s[i + 4 + u]) : fmaxf(mx[u], s[i + u]);
      }
      return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
    };
    // The reference m has to suit P, which holds V's factors too: a key of a large
    // factor that this row does not see, or hardly, must not push the others' P
    // out of E4M3's range. Factors within SPREAD binades of the largest: the
    // logits' maximum does. Else it is the maximum of logit plus factor, at most
    // 96 below the former (l, a sum without the factors, stays below 2^127).
    float far = NEG_INF;
    if constexpr (KV == 2)
      if (wide) far = weighted_max<L::FAC, TW>(s_addr + my0, kfac, vfac, my0, qscale, kb, tv);
    float s[W];
    float bmax = NEG_INF;
#pragma unroll
    for (int h = NH - 1; h >= 0; --h) {              // (run 0 stays in registers)
      load_s(my0 + h * W, s);
      bmax = fmaxf(bmax, max_s(s));
    }
    float top = bmax * qscale;
    if (KV == 2 && wide) top = fmaxf(far, top - 96.f);
    const bool rescale = top > m_ref + L::LIMIT;     // also for the first finite maximum
    const float m_use = rescale ? top - L::TOP : m_ref;
    const float m_sub = m_use == NEG_INF ? 0.f : m_use;
    // P goes over S: 16-bit, two keys a column; FP8, four keys a column, 8 columns
    // of each part for each 32 keys. Run h of P lies over columns of S that run h
    // or an earlier one has read.
    const uint64_t qs2 = pack2(qscale, qscale), ms2 = pack2(-m_sub, -m_sub);
    uint64_t rs[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      if (h > 0) load_s(my0 + h * W, s);
      constexpr int N = L::F8 && W >= 32 ? 32 : 16;  // keys of 8 columns (of 4: half a step)
#pragma unroll
      for (int q = 0; q < W; q += N) {
        uint64_t e[N / 2];
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          float a, b2;
          unpack2(fma2(pack2(s[q + i], s[q + i + 1]), qs2, ms2), a, b2);
          e[i / 2] = pack2(ex2(a), ex2(b2));
          rs[i / 2 & 1] = add2(rs[i / 2 & 1], e[i / 2]);
        }
        const uint32_t col = (uint32_t)(my0 + h * W + q) / L::KSTEP * (8 * L::PP);
        uint32_t parts[L::PP][8];
        if constexpr (!L::F8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float a, b2;
            unpack2(e[i], a, b2);
            parts[0][i] = Pack<T>::two(a, b2);
          }
        } else {
          if constexpr (KV == 2) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
              uint64_t f[2];
              factors4<L::FAC>(vfac, my0 + h * W + q + i, f);
              e[i / 2] = mul2(e[i / 2], f[0]);
              e[i / 2 + 1] = mul2(e[i / 2 + 1], f[1]);
            }
          }
#pragma unroll
          for (int i = 0; i < N / 4; ++i) {
            uint32_t w[L::PP];
            split4<L::PP>(e[2 * i], e[2 * i + 1], w);
#pragma unroll
            for (int p = 0; p < L::PP; ++p) {
              if (N == 32) {
                parts[p][i] = w[p];
              } else {                               // (zeros for the neighbour copy's keys)
                parts[p][i] = cp & 1 ? 0u : w[p];
                parts[p][i + 4] = cp & 1 ? w[p] : 0u;
              }
            }
          }
        }
#pragma unroll
        for (int p = 0; p < L::PP; ++p) tmem_st8(s_addr + col + 8 * p, parts[p]);
      }
    }
    if constexpr (C > 1) {                           // zeros for the other copies' keys
      const uint32_t zero[8] = {};
#pragma unroll
      for (int c = 0; c < BK / L::KSTEP; ++c)        // key steps
        if (TW < L::KSTEP ? c != cp >> 1 : c / (TW < L::KSTEP ? 1 : TW / L::KSTEP) != cp)
#pragma unroll
          for (int p = 0; p < L::PP; ++p) tmem_st8(s_addr + 8 * (c * L::PP + p), zero);
    }
    const bool need = (rescale && m_ref != NEG_INF) || (KV == 2 && o_scale != 1.f);
    if (j > 0 && __any_sync(0xffffffffu, need)) {
      // O holds P V up to the last block: wait for it, then rescale in TMEM
      const int sp = sc - 1;
      if (!tree_wait(BAR(TB_PVDONE + sp % NSB), (sp / NSB) & 1, abort_flag)) {
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
    {
      float a, b2;
      unpack2(add2(rs[0], rs[1]), a, b2);
      l += a + b2;
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(BAR(TB_PFULL + b));
  }
  if (ok) {
    const int sl = sc0 + nb - 1;
    ok = tree_wait(BAR(TB_PVDONE + sl % NSB), (sl / NSB) & 1, abort_flag);
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
    // a row without keys is 0, whatever its sink (-inf less the reference, -inf too, is
    // NaN; a large V scale over a low one's 2^x infinite); a NaN row stays NaN
    const float inv = l == 0.f ? 0.f : v_scale / denom;
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
    // Join the copies through the Q region, 8 threads a row, 16 rows at a time: a
    // thread's rows, their weights and places are made once.
    float* ml = reinterpret_cast<float*>(smem + L::Q_OFF);
    ml[2 * tid] = m_ref;
    ml[2 * tid + 1] = l;
    softmax_sync();
    constexpr int RT = RB / 16;                      // rows of a thread
    const int l8 = tid & 7;
    float w[RT][C];
    size_t at[RT];
#pragma unroll
    for (int k = 0; k < RT; ++k) {
      const int r = (tid >> 3) + 16 * k;
      float M = NEG_INF;
#pragma unroll
      for (int c = 0; c < C; ++c) M = fmaxf(M, ml[2 * (c * RB + r)]);
      const float Ms = M == NEG_INF ? 0.f : M;
      float wsum = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        w[k][c] = ex2(ml[2 * (c * RB + r)] - Ms);
        wsum += w[k][c] * ml[2 * (c * RB + r) + 1];
      }
      const int pr = seg[TS_ROW0] + min(r, nrows - 1), tk = pr / G, hd = seg[TS_G] * G + pr - tk * G;
      const size_t gr = (size_t)(seg[TS_QROW0] + tk) * H + hd;
      float denom = wsum;
      if (P.sinks && prow < 0) denom += ex2(P.sinks[hd] * kLog2e - Ms);
      const float inv = wsum == 0.f ? 0.f : v_scale / denom;
#pragma unroll
      for (int c = 0; c < C; ++c) w[k][c] *= inv;
      at[k] = prow < 0 ? gr : (size_t)(prow + r);
      if (l8 == 0 && r < nrows) {
        const float lse = wsum == 0.f ? NEG_INF : M + log2f(wsum);
        if (prow >= 0) P.part_lse[at[k]] = lse;
        else if (P.lse) P.lse[gr] = lse;
      }
    }
    constexpr int CH = L::JOIN / 4;                  // 16-byte chunks of a lane's part
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += L::JOIN) {
      softmax_sync();                                // what was there has been read
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
#pragma unroll
      for (int k = 0; k < RT; ++k) {
        const int r = (tid >> 3) + 16 * k;
        if (r >= nrows) break;
#pragma unroll
        for (int ch = l8; ch < CH; ch += 8) {
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int ln = c * RB + r;
            const uint4 u = lds128(sbase + L::Q_OFF + ln * (CH * 16) + ((ch + ln) & (CH - 1)) * 16);
            acc.x = fmaf(w[k][c], __uint_as_float(u.x), acc.x);
            acc.y = fmaf(w[k][c], __uint_as_float(u.y), acc.y);
            acc.z = fmaf(w[k][c], __uint_as_float(u.z), acc.z);
            acc.w = fmaf(w[k][c], __uint_as_float(u.w), acc.w);
          }
          const size_t to = at[k] * D + c0 + ch * 4;
          if (prow < 0)
            *reinterpret_cast<uint2*>(outg + to) = make_uint2(Pack<T>::two(acc.x, acc.y), Pack<T>::two(acc.z, acc.w));
          else
            *reinterpret_cast<float4*>(P.part_o + to) = acc;
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
  using L = TLayout<T, D, KV>;
  constexpr int BK = L::BK, NSB = L::NSB;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (uniform, and known to be)
  const uint32_t sbase = smem_u32(smem), bar0 = sbase + L::BAR_OFF;
  static_assert(TB_COUNT * 8 <= 192, "barriers overlap the TMEM slot");
  if ((sbase & 1023u) != 0u) {                       // 128B-swizzle atoms need 1024-byte alignment
    if (tid == 0) atomicOr(P.status, POD_STATUS_ALIGN);
    return;
  }
  // (asked for before the set-up below, which takes as long)
  const int seg0 = P.cta_ptr[blockIdx.x], seg1 = P.cta_ptr[blockIdx.x + 1];
  if (warp == 5 && lane < 2 && P.kbx > 0) tma_prefetch_desc(lane ? &P.tm_v : &P.tm_k);
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::BAR_OFF + 196);
  if (warp == 4) {
    tmem_alloc(sbase + L::BAR_OFF + 192, L::TMEM_COLS);
    tmem_relinquish();
  }
  const bool tma = P.kbx > 0;
  if (tid == 0) {
    const uint32_t loads = tma ? 1u : 32u * L::GW;   // gather: two or three warps
    mbar_init(BAR(TB_QFULL), 128);
    for (int s = 0; s < 4; ++s) {
      mbar_init(BAR(TB_KFULL + s), loads);
      mbar_init(BAR(TB_KEMPTY + s), 1);
      mbar_init(BAR(TB_VFULL + s), loads);
      mbar_init(BAR(TB_VEMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(BAR(TB_SFULL + s), 1);
      mbar_init(BAR(TB_PFULL + s), 128);
      mbar_init(BAR(TB_PVDONE + s), 1);
    }
    mbar_init(BAR(TB_FINAL), NSB);
    *abort_flag = 0;
    fence_mbar_init();
  }
  asm volatile("prefetch.global.L1 [%0];" ::"l"(P.segs + (size_t)seg0 * TS_REC));
  tc_fence_before();
  __syncthreads();
  // The next kernel (the merge, or another call's) may be scheduled now; it waits for
  // this grid's completion. Not before: a next tree kernel takes tensor memory before
  // it waits, and must not take what a CTA of this one, which it waits for, still needs.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (launched while the kernel before may still run: the plan, which only copies
  // write, may be read before this, tensors and the partial rows not)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::BAR_OFF + 192);
  bool ok = true;
  volatile int never = 0;                            // an abort flag that nobody raises

  if (warp < 4) {
    int sc0 = 0;
    for (int i = seg0; i < seg1 && ok; ++i) {
      const int32_t* seg = P.segs + (size_t)i * TS_REC;
      const int copies = seg[TS_COPIES];
      ok = copies == 4   ? tree_softmax<T, D, KV, 4>(P, smem, tmem, seg, sc0, abort_flag)
           : copies == 2 ? tree_softmax<T, D, KV, 2>(P, smem, tmem, seg, sc0, abort_flag)
                         : tree_softmax<T, D, KV, 1>(P, smem, tmem, seg, sc0, abort_flag);
    }
  } else if (warp == 4 || (NSB > 1 && warp == 7)) {
    // ---------------------------------------------------------- MMA issuers
    // Two S buffers: warp 4 issues the Q K^T, as soon as the P V that reads the
    // buffer's last P has finished, warp 7 the P V. One S buffer: warp 4 issues
    // PV_j and QK_{j+1} in turn (MMAs issued by one thread run in order). A whole
    // warp walks its loop and one elected lane issues: addresses and descriptors
    // then stay in uniform registers (a loop under `lane == 0` moved each of them
    // there for every MMA: 85 clocks an instruction). The second warp takes the
    // waits of one product off the other's: 16 requests of 64 tokens and 4100 keys
    // went from 137 to 129 us with pages of 64; with pages of 16 they stayed at 136.
    const uint32_t id_qk = L::F8 ? idesc_f8(false, 128, BK, false, false) : idesc_f16(Pack<T>::kBF16, 128, BK, false, false);
    const uint32_t id_pv = L::F8 ? idesc_f8(false, 128, D, false, true) : idesc_f16(Pack<T>::kBF16, 128, D, false, true);
    // V stage: 16-bit TMA boxes of vb keys lie as [box][row part][key], anything
    // else as [row part][key]
    const int vb = !L::F8 && tma ? P.kbx : BK;
    const uint32_t v_box = (uint32_t)(vb * L::PARTS * L::ROWB);
    const uint64_t v_desc0 = L::desc(sbase + L::V_OFF, (uint32_t)(vb * L::ROWB),
                                     vb >= L::KSTEP ? 8u * L::ROWB : 8u * L::ROWB * L::PARTS);
    uint32_t v_step[L::KSTEPS];
#pragma unroll
    for (int k = 0; k < L::KSTEPS; ++k)
      v_step[k] = ((uint32_t)(k * L::KSTEP / vb) * v_box + (uint32_t)(k * L::KSTEP % vb) * L::ROWB) >> 4;
    const uint64_t q_desc0 = L::desc(sbase + L::Q_OFF, 16, 8 * L::ROWB);
    const uint64_t k_desc0 = L::desc(sbase + L::K_OFF, 16, 8 * L::ROWB);
    int ks = 0, vs = 0, sc0 = 0;                     // ring positions, with their phases
    uint32_t kph = 0, vph = 0;
    // Q K^T of the block in K stage `slot` into S buffer b
    auto issue_qk = [&](int b, uint64_t kd, int slot) {
#pragma unroll
      for (int p = 0; p < L::QP; ++p)
#pragma unroll
        for (int k = 0; k < L::DSTEPS; ++k) {
          constexpr int SPP = L::ROWB / 32;          // steps of a row part
          const uint64_t qd = q_desc0 + (((p * L::PARTS + k / SPP) * L::QPART + (k % SPP) * 32) >> 4);
          const uint64_t bd = kd + (((k / SPP) * L::KVPART + (k % SPP) * 32) >> 4);
          const uint32_t d_s = tmem + L::TM_S + b * BK;
          if constexpr (L::F8) mma_f8_ss(d_s, qd, bd, id_qk, p + k > 0 ? 1u : 0u);
          else mma_f16_ss(d_s, qd, bd, id_qk, k > 0 ? 1u : 0u);
        }
      mma_commit(BAR(TB_SFULL + b));
      mma_commit(BAR(TB_KEMPTY + slot));
    };
    auto wait_k = [&]() -> bool {
      if (!tree_wait(BAR(TB_KFULL + ks), kph, abort_flag)) return false;
      if (!tma) fence_proxy_async();
      return true;
    };
    auto next_k = [&]() {
      if (++ks == L::NK) { ks = 0; kph ^= 1; }
    };
    // O += P V of a block (its S buffer b, `keys` keys below kv_len), and with
    // `qk` the next block's Q K^T right behind it
    auto pv = [&](bool first, int keys, int b, uint32_t parity, bool qk, int qb, uint64_t kd) -> bool {
      if (!tree_wait(BAR(TB_VFULL + vs), vph, abort_flag)) return false;
      // Key steps past kv_len carry P = 0: skip them. Rows at or past kv_len in
      // the last step are unused slots of the last page, or nothing: zero them,
      // so that P = 0 never meets a non-finite value.
      const int ksteps = (keys + L::KSTEP - 1) / L::KSTEP;
      const uint64_t vd = v_desc0 + (uint32_t)(vs * L::STAGE >> 4);
      const uint32_t a_p = tmem + L::TM_S + b * BK;
      if (keys % L::KSTEP) {
        const uint32_t va = sbase + L::V_OFF + vs * L::STAGE;
        constexpr int CPP = L::ROWB / 16;            // 16-byte chunks of a row part
        for (int x = lane; x < (ksteps * L::KSTEP - keys) * L::PARTS * CPP; x += 32) {
          const int r = keys + x / (L::PARTS * CPP), h = x / CPP % L::PARTS, c = x % CPP;
          sts128(va + (uint32_t)(r / vb) * v_box + (h * vb + r % vb) * L::ROWB + c * 16, make_uint4(0, 0, 0, 0));
        }
        fence_proxy_async();
        __syncwarp();
      } else if (!tma) {
        fence_proxy_async();
      }
      if (!tree_wait(BAR(TB_PFULL + b), parity, abort_flag)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < L::KSTEPS; ++k)
          if (k < ksteps) {
            if constexpr (L::F8) {
#pragma unroll
              for (int p = 0; p < L::PP; ++p)
                mma_f8_ts(tmem + L::TM_O, a_p + 8 * (k * L::PP + p), vd + v_step[k],
                          p > 0 && L::PP == 3 ? idesc_f8(true, 128, D, false, true) : id_pv,
                          (!first || k > 0 || p > 0) ? 1u : 0u);
            } else {
              mma_f16_ts(tmem + L::TM_O, a_p + k * 8, vd + v_step[k], id_pv, (!first || k > 0) ? 1u : 0u);
            }
          }
        mma_commit(BAR(TB_PVDONE + b));
        mma_commit(BAR(TB_VEMPTY + vs));
        if (qk) issue_qk(qb, kd, ks);
      }
      __syncwarp();
      if (++vs == L::NV) { vs = 0; vph ^= 1; }
      return true;
    };
    for (int i = seg0; i < seg1 && ok; ++i) {
      const int32_t* seg = P.segs + (size_t)i * TS_REC;
      const int blk0 = seg[TS_BLK0], nb = seg[TS_BLK1] - blk0, kv_len = seg[TS_KVLEN];
      auto keys_of = [&](int j) { return min(kv_len - (blk0 + j) * BK, BK); };
      if (warp == 4) {
        if (!tree_wait(BAR(TB_QFULL), (i - seg0) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
      }
      if constexpr (NSB > 1) {
        for (int j = 0; j < nb && ok; ++j) {
          const int sc = sc0 + j, b = sc % NSB;
          if (warp == 4) {
            const uint64_t kd = k_desc0 + (uint32_t)(ks * L::STAGE >> 4);
            ok = wait_k() && (sc < NSB || tree_wait(BAR(TB_PVDONE + b), (sc / NSB - 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) issue_qk(b, kd, ks);
            __syncwarp();
            next_k();
          } else {
            ok = pv(j == 0, keys_of(j), b, (sc / NSB) & 1, false, 0, 0);
          }
        }
      } else {
        for (int j = -1; j < nb; ++j) {
          const uint64_t kd = k_desc0 + (uint32_t)(ks * L::STAGE >> 4);
          const bool has_k = j + 1 < nb;
          if (has_k && !wait_k()) { ok = false; break; }
          if (j >= 0) {
            if (!pv(j == 0, keys_of(j), 0, (sc0 + j) & 1, has_k, 0, kd)) { ok = false; break; }
          } else {
            tc_fence_after();
            if (elect_one()) issue_qk(0, kd, ks);
            __syncwarp();
          }
          if (has_k) next_k();
        }
      }
      sc0 += nb;
    }
  } else if (tma) {
    // ---------------------------------------------------------- K and V boxes
    if (warp < 7) {
      const bool is_v = warp == 6;
      const void* tm = is_v ? &P.tm_v : &P.tm_k;
      const int NS = is_v ? L::NV : L::NK;
      // boxes of a block: groups of kbx keys, a box for each row part; a 16-bit V
      // box holds every part. (No eviction hint: with evict-first where a key serves
      // one tile only, and so two forms of the load, wide trees took 134 us, not 129,
      // 64 ragged requests 386, not 383.)
      const bool whole = is_v && !L::F8;
      const int groups = BK / P.kbx, per = whole ? 1 : L::PARTS;
      const int gi = lane / per, part = lane - gi * per;
      const bool mine = gi < groups;
      int fill = 0;
      for (int i = seg0; i < seg1 && ok; ++i) {
        const int32_t* seg = P.segs + (size_t)i * TS_REC;
        const int g = seg[TS_G], npages = seg[TS_NPAGES];
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
            const uint32_t stage = sbase + (is_v ? L::V_OFF : L::K_OFF) + s * L::STAGE;
            const uint32_t dst = stage + (whole ? gi * P.kbx * L::PARTS * L::ROWB
                                                : part * L::KVPART + gi * P.kbx * L::ROWB);
            // (a page past the request's last is out of the pool: TMA fills zeros)
            tma_load_5d(dst, tm, 0, tin, part, g, 2 * page + (is_v ? 1 : 0), BAR(full));
          }
          ++fill;
          if (blk + 1 < b1) page = page_of(blk + 1);
        }
      }
      // no copy is in flight when the CTA ends, also after an abort
      for (int f = max(fill - NS, 0); f < fill; ++f)
        tree_wait(BAR((is_v ? TB_VFULL : TB_KFULL) + f % NS), (f / NS) & 1, &never);
    }
  } else {
    // ---------------------------------------------------------- gather
    // Every lane finds the rows of BK / 32 keys of the next block while the
    // copies of this one are issued; a warp copies 32 / CPR keys at a time,
    // their rows passed by shuffle.
    constexpr int CPR = D * L::ES / 16;              // 16-byte chunks of a row
    constexpr int KPI = 32 / CPR, NQ = BK / 32;
    const int w = warp - 5;
    const uint8_t* __restrict__ kvg = static_cast<const uint8_t*>(P.kv);
    const long long vstep = (long long)P.ps * P.Hk;
    const int sub = lane / CPR, c = lane % CPR;
    const int part = c / (L::ROWB / 16), cc = c % (L::ROWB / 16);
    int fill = 0;
    for (int i = seg0; i < seg1 && ok; ++i) {
      const int32_t* seg = P.segs + (size_t)i * TS_REC;
      const int kv_len = seg[TS_KVLEN], b1 = seg[TS_BLK1];
      const KeyAt at = key_at(P, seg);
      long long row[NQ];
      int page[NQ];
      auto my_key = [&](int blk, int q) { return min(blk * BK + q * 32 + lane, kv_len - 1); };
#pragma unroll
      for (int q = 0; q < NQ; ++q) page[q] = at.page(my_key(seg[TS_BLK0], q));
      for (int blk = seg[TS_BLK0]; blk < b1; ++blk) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          row[q] = at.row(my_key(blk, q), page[q]);
          if (blk + 1 < b1) page[q] = at.page(my_key(blk + 1, q));
        }
        const int left = kv_len - blk * BK;
        auto copy = [&](uint32_t dst, long long step) {
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
#pragma unroll 4
            for (int x = w; x < 32 / KPI; x += L::GW) {
              const int k = x * KPI + sub, key = q * 32 + k;
              const long long r = __shfl_sync(0xffffffffu, row[q], k) + step;
              cp_async16(dst + part * L::KVPART + L::swz(key, cc), kvg + r * (D * L::ES) + c * 16,
                         key < left ? 16u : 0u);
            }
          }
        };
        const int s = fill % L::NK, v = fill % L::NV;
        if (!tree_wait(BAR(TB_KEMPTY + s), ((fill / L::NK) & 1) ^ 1, abort_flag)) { ok = false; break; }
        copy(sbase + L::K_OFF + s * L::STAGE, 0);
        cp_async_mbar_arrive(BAR(TB_KFULL + s));
        if (!tree_wait(BAR(TB_VEMPTY + v), ((fill / L::NV) & 1) ^ 1, abort_flag)) { ok = false; break; }
        copy(sbase + L::V_OFF + v * L::STAGE, vstep);
        cp_async_mbar_arrive(BAR(TB_VFULL + v));
        ++fill;
      }
    }
    cp_async_wait_all();
  }
  if (!ok) {
    *abort_flag = 1;
    if (lane == 0) atomicOr(P.status, POD_STATUS_TIMEOUT);
  }

  // ------------------------------------------------------------ teardown:
  // every MMA has finished before TMEM is given back
  tc_fence_before();
  __syncthreads();
  if (NSB > 1 && warp == 7) {
    if (elect_one()) mma_commit(BAR(TB_FINAL));
    __syncwarp();
  }
  if (warp == 4) {
    if (elect_one()) mma_commit(BAR(TB_FINAL));
    __syncwarp();
    mbar_wait(BAR(TB_FINAL), 0, &never);
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// Shared memory asked for: at least 88 KB, so that an SM holds two CTAs of 256 TMEM
// columns and no third, whatever registers they take, nor two beside one of
// pod_kernel's (57728 bytes or more): a CTA of the kernel before that has no columns
// yet never meets two of this one that hold all 512 and wait for it. (The L1 does
// not lose by it: the carve-out is the largest in any case.)
template <typename T, int D, int KV>
constexpr int tree_smem() {
  return TLayout<T, D, KV>::TOTAL > 88 * 1024 ? TLayout<T, D, KV>::TOTAL : 88 * 1024;
}

template <typename T, int D, int KV>
cudaError_t launch_tree(const PodTreeParams& P, cudaStream_t stream) {
  constexpr int SMEM = tree_smem<T, D, KV>();
  constexpr int SM_BYTES = 228 * 1024, CTA_BYTES = SMEM + 1024, CTAS = TLayout<T, D, KV>::TMEM_COLS == 512 ? 1 : 2;
  static_assert(CTAS * CTA_BYTES <= SM_BYTES, "shared memory of the CTAs on an SM");
  static_assert((CTAS + 1) * CTA_BYTES > SM_BYTES && CTAS * CTA_BYTES + 57728 > SM_BYTES,
                "CTAs on an SM beyond its tensor memory");
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)P.n_cta);
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // Set up beside the kernel before, a call after another is 1 to 4 % shorter (64
  // ragged requests 388 -> 385 us, four short ones 11.7 -> 11.2); over block scales
  // it was longer (96 requests of 2 to 4 tokens 333 -> 354 us).
  cfg.numAttrs = KV == 2 ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, pod_tree_kernel<T, D, KV>, P);
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
