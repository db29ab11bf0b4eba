// pod_decode.cuh — attention of one token per request over its paged cache, with
// lengths, block table and (optionally) selected pages on the device.
//
// Mathematics. For the G query heads of a KV head: x = s q.k over the visible keys,
// p = 2^(x - m), l = sum p, o = sum p v / l. m is a reference that may lag behind the
// running maximum, by 8 or 2 at most: it moves, and O with it, only when a logit passes it by
// more than that (one vote a tile instead of shuffles for the maximum; the lag is a factor
// that l and O share). Pieces of a request's keys join by reference and sum (a base-2 LSE would
// lose the sum beside large references). Over a
// block-scaled cache O has a reference of its own, that of p * 2^(V's exponent).
//
// Layout. Both products run transposed, S^T = K Q^T and O^T = V^T P^T, as
// mma.sync m16n8k16 with keys (then head elements) in the 16 rows and the query
// heads of a KV head in the 8 columns: a decode step has few query heads, and this
// wastes none of 8. (tcgen05 has 64 or 128 rows to fill, and the step reads each key
// once: it is bound by memory.) The order of the reduced index is free in a product,
// and so is that of the rows of O^T: so a lane takes up to 32 contiguous bytes of a key as
// its elements of K's fragments, and of V's as rows, and K and V go from memory to the
// matrix unit without shared memory in between. P^T changes from accumulator to operand by
// movmatrix. P is carried in two 16-bit parts (off by 2^-17 of a weight in bf16, 2^-22 in
// fp16): the matrix unit has time. Codes of FP8 caches are widened to fp16, exactly; bf16
// results over them take P in one fp16 part. fp16 ends at 2^-24, so the second part is carried
// times 2^11, in a sum of its own: weights down to 2^-21 of the largest keep all these bits, and
// those below are off by 2^-43 of the largest (in one sum they were off by 2^-32 of it, which is
// much where one key takes nearly all the weight and its V is small).
//
// Work split. The keys of every (KV head, request) are cut into units of one tile a
// warp; the units of all, laid out head by head, are dealt to the CTAs of one
// launch in equal runs. Every CTA finds its run from the lengths on the device, so
// nothing is planned on the host and a captured launch serves later lengths. A
// run's pieces of a request that is cut go to the workspace; the merge kernel joins them in
// the order of the keys.
//
// Bound by memory: twelve warps an SM with up to 8 KB of keys each on their way, and the next
// tile's rows asked for into L2. Measured on two GB300s, in graphs, of the measured copy rate: 64
// requests of 512 to 16384 keys, 32/8 heads of 128, bf16: 326 to 333 us, 101 to 103 %; one request
// of 131072 keys, 64/8 heads: 86 to 88 us, 91 %; 96 requests of 4096 to 12288 keys over block-scaled
// FP8: 244 to 253 us, 89 to 92 % (per-tensor scales 238 to 247; HND pages 238 and 230): the
// conversions and the softmax of twice as many keys a byte, and rows of 128 bytes a kilobyte apart. 32-byte loads
// and page numbers two tiles ahead made 332 of 352 and 260 of 307 us. K and V through a ring of
// asynchronous copies in shared memory took 430 and 310, K's codes as E4M3 operands (the legacy E4M3
// mma) 295, the next segment's first tile asked for before the warps' sums join 331 and 270.
#pragma once
#include <limits.h>
#include <math.h>

#include "pod_beside.h"
#include "pod_decode.h"
#include "pod_device.cuh"

namespace pod {
namespace {

constexpr int kShortUnits = 8, kShortCtas = 256;    // of the kernel for short rows: units a CTA, CTAs in clusters

template <typename T, int D, int FMT, int NT>
struct DecodeShape {
  static constexpr int E = FMT == POD_KV_16BIT ? 2 : 1;           // bytes of an element
  static constexpr int MT = FMT == POD_KV_16BIT ? (D == 64 ? 2 : 1) : (D == 64 ? 4 : D == 128 ? 2 : 1);
  static constexpr int TK = 16 * MT;                              // keys of a warp's tile
  static constexpr int HT = 8 * NT;                               // query heads of a tile
  // A lane's chunk of a key: a quarter of K's row, an eighth of V's, at most 32 bytes.
  static constexpr int WK = D * E / 16 < 8 ? D * E / 16 : 8;      // 32-bit words of a chunk of K
  static constexpr int CK = WK * 4 / E, NK = D / (4 * CK);        // its elements; chunks of a key
  static constexpr int WV = D * E / 32 < 8 ? D * E / 32 : 8;      // of V
  static constexpr int CV = WV * 4 / E, NV = D / (8 * CV);
  static constexpr int IDX = (TK + 31) / 32;                      // tile keys of a lane
  // 16-bit parts of a weight: two, but for fp16 weights of bf16 results, where one is off by at
  // most 2^-11 of the weight, an eighth of what the result's own rounding may be off by. (Two
  // there: 96 block-scaled requests 244 -> 248 us, with 16 query heads a KV head 307 -> 353, of
  // head_dim 64 159 -> 168; per-tensor scales 238 -> 242.)
  static constexpr int PARTS = FMT != POD_KV_16BIT && Pack<T>::kBF16 ? 1 : 2;
};

// N 32-bit words, read once (zeros where not `live`)
template <int N>
POD_DEV void load_words(uint32_t* r, const uint8_t* p, bool live) {
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = 0u;
  if (!live) return;
  if constexpr (N == 8)
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
  else if constexpr (N == 4)
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "l"(p));
  else
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p));
}
// 8 x 8 matrix of 16-bit values, a register's pair in row lane / 4: its transpose
POD_DEV uint32_t turn8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
POD_DEV uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
// 2^(byte - 127)
POD_DEV float pow2_of(int byte) {
  return byte == 0 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)byte << 23);
}

// Weights leave the exponential times 2^weight_up, under a reference that is at most lag()
// below the maximum. Sums of the largest bf16 values stay below fp32's. fp16 weights stay below
// 2^15, and what is left below the largest counts: fp16's numbers end at 2^-24, so one part is off
// by up to 2^-(25 + weight_up) of the largest weight. So a single part has little lag (8 and 2^7
// left 2^-32 of the largest weight, 2^-38 now; 16 query heads a KV head over block scales 299 ->
// 306 us, for the reference moves more often, the others nothing to 1 %); two parts reach 2^-43
// with the larger one.
template <typename T, int FMT>
constexpr float weight_up() {
  return !Pack<T>::kBF16 ? 7.f : FMT == POD_KV_16BIT ? -24.f : 13.f;
}
template <typename T, int FMT>
constexpr float lag() {
  return Pack<T>::kBF16 && FMT != POD_KV_16BIT ? 2.f : 8.f;
}
constexpr float kNoKey = -3.4028234663852886e38f;    // the reference before the first key: the lowest number
constexpr float kFar = 65536.f;                      // base-2 logits to which V's exponent is not added as they are

// o += a * hi, + a * lo where PARTS is 2. fp16's lo comes times 2^11 and is summed by itself (in
// o's own sum, without the factor: 16 query heads a KV head over block scales 331 us, 353 now, over
// per-tensor scales 317 and 334; block scales with head_dim 64 163 and 167, 256 260 and 268; the
// other forms the same to 1 %).
template <bool BF16, int PARTS>
POD_DEV void mma_parts(float* o, const uint32_t* a, const uint32_t* hi, const uint32_t* lo) {
  if constexpr (PARTS == 2 && !BF16) {
    float x[4];
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(lo[0]), "r"(lo[1]), "f"(0.f));
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(x[i], 0x1p-11f, o[i]);
  }
  mma16816<BF16>(o, a, hi[0], hi[1]);
  if constexpr (PARTS == 2 && BF16) mma16816<BF16>(o, a, lo[0], lo[1]);
}

// a / b of numbers that are not negative: 32 bits where they do (a third of the instructions)
POD_DEV long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// Keys of request r that the call reads, as indices v in [0, count): key first + v
// of the cache, or slot v % ps of the selected page v / ps.
struct Keys {
  int len, first, count;
};
POD_DEV Keys keys_of(const DecodeParams& P, int r) {
  Keys k;
  k.len = min(max(P.lens[r], 0), P.width * P.ps);   // (the product is at most 2^30)
  if (P.pages) {
    k.first = 0;
    k.count = min((k.len + P.ps - 1) / P.ps, P.num_selected) * P.ps;
  } else {
    k.first = P.window < 0 ? 0 : max(0, k.len - 1 - P.window);
    k.count = k.len - k.first;
  }
  return k;
}

// LSE and output scale of a row under its sink: exp(sink) joins the denominator
POD_DEV float sink_factor(float lse, float sink) {
  const float s = sink * 1.4426950408889634f;
  return s > lse ? ex2(lse - s) / (1.f + ex2(lse - s)) : 1.f / (1.f + ex2(s - lse));
}

// What the four warps of a CTA leave in shared memory: sums under references of their own.
template <int D, int HT>
struct alignas(16) DecodeShared {
  float o[kDecodeWarps][HT][D];
  float m[3][kDecodeWarps][HT];    // r, l, and O's reference from r on
};

template <int D, int HT>
POD_DEV int offsetof_m(int what, int w, int h) {
  return (kDecodeWarps * HT * D + (what * kDecodeWarps + w) * HT + h) * 4;
}

// A warp's tiles at v, v + step, ... below v1 of a request's keys, for `heads` query heads from h0 on.
template <typename T, int D, int FMT, int NT>
POD_DEV void attend(const DecodeParams& P, const Keys& K, int row, int hk, int h0, int heads, int v, int step, int v1,
                    DecodeShared<D, 8 * NT>& sh) {
  using S = DecodeShape<T, D, FMT, NT>;
  using M = typename std::conditional<FMT == POD_KV_16BIT, T, __half>::type;   // operands of the products
  constexpr bool MBF = Pack<M>::kBF16;
  constexpr float kUp = weight_up<T, FMT>(), kLag = lag<T, FMT>();
  constexpr int MT = S::MT, TK = S::TK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // r: the reference of l, less the weights' factor 2^kUp; rv: that of O, counted from r on. (V's
  // exponent is added to a logit only once r is off it, and every rounding of a reference is one
  // towards smaller weights, so logits of any size neither lose V's exponent nor pass fp16's range.
  // As sums of logit and exponent, which lost it from some 2^20 on, over block scales: 251.3 us, 252.3
  // now, with 16 query heads a KV head 306 and 321, with fp16 results of these 353 and 363 to 389, as the
  // compiler lays them out.)
  float o[NT][S::NV][S::CV / 2][4], r[NT][2], rv[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int b = 0; b < S::NV; ++b)
#pragma unroll
      for (int i = 0; i < S::CV / 2; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[n][b][i][c] = 0.f;
    r[n][0] = r[n][1] = kNoKey;
    rv[n][0] = rv[n][1] = l[n][0] = l[n][1] = 0.f;
  }

  // ---- addresses: rows of d elements; a key's K row is index * key_step + rows of the head
  const long long row_bytes = (long long)D * S::E;
  const long long key_step = P.hnd ? row_bytes : row_bytes * P.Hk;
  const long long v_off = (long long)P.ps * P.Hk * row_bytes;
  const uint8_t* kbase = P.cache + (P.hnd ? (long long)hk * P.ps : (long long)hk) * row_bytes;
  const unsigned page_step = 2u * (unsigned)P.ps * (P.hnd ? (unsigned)P.Hk : 1u);
  const int32_t* table = P.table + (long long)row * P.table_stride;
  const int32_t* sel = P.pages ? P.pages + ((long long)row * P.Hk + hk) * P.num_selected : nullptr;

  // Where a tile's keys lie, lane i: key i. Three steps, an iteration of the loop apart so
  // that none waits for its load: the position in the table (its entry in the list of
  // pages), the page, the keys' rows.
  struct Place {
    int page, in;
  };
  auto place = [&](int v, int j) {
    Place p = {-1, -1};
    v += j * 32 + lane;
    if ((TK >= 32 || lane < TK) && v < v1) {
      const int w = v + K.first, at = P.ps_shift >= 0 ? w >> P.ps_shift : w / P.ps;
      p.in = w - at * P.ps;
      p.page = sel ? sel[at] : at;
    }
    return p;
  };
  auto page_at = [&](Place& p) {
    // (a page past the request's last, or a slot past its last key: not visible)
    if (sel && p.in >= 0 && (p.page < 0 || p.page >= P.width || p.page * P.ps + p.in >= K.len)) p.in = -1;
    if (p.in >= 0) p.page = table[p.page];
  };
  auto index_of = [&](const Place& p) {            // 0xffffffff: not visible
    if (p.in < 0) return 0xffffffffu;
    if ((unsigned)p.page >= P.num_pages) {
      if (P.status) atomicOr(P.status, kStatusSlot);
      return 0xffffffffu;
    }
    return (unsigned)p.page * page_step + (unsigned)p.in;
  };

  uint32_t kr[MT][2][S::NK][S::WK], vr[MT][4][S::NV][S::WV];
  unsigned idx[S::IDX], seen[S::IDX];              // rows of the tile that is loaded next; visible keys of the one at hand
  uint32_t ek[S::IDX], ev[S::IDX];                 // exponent bytes of K and V, a lane's own keys
  auto load_k = [&]() {
#pragma unroll
    for (int s = 0; s < MT; ++s)
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const unsigned i = __shfl_sync(0xffffffffu, idx[s / 2], (s & 1) * 16 + a * 8 + g);
        const uint8_t* p = kbase + (long long)i * key_step + t * (S::WK * 4);
#pragma unroll
        for (int b = 0; b < S::NK; ++b) load_words<S::WK>(kr[s][a][b], p + b * (S::WK * 16), i != 0xffffffffu);
      }
    if constexpr (FMT == POD_KV_E4M3_BLOCK) {
#pragma unroll
      for (int j = 0; j < S::IDX; ++j) {
        ek[j] = ev[j] = 127;
        if (idx[j] != 0xffffffffu) {
          const uint8_t* p =
              P.scales + (P.hnd ? (long long)idx[j] + (long long)hk * P.ps : (long long)idx[j] * P.Hk + hk);
          ek[j] = p[0];
          ev[j] = p[(long long)P.ps * P.Hk];
        }
      }
    }
  };
  auto load_v = [&]() {
#pragma unroll
    for (int s = 0; s < MT; ++s)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const unsigned i = __shfl_sync(0xffffffffu, idx[s / 2], (s & 1) * 16 + (a >> 1) * 8 + 2 * t + (a & 1));
        const uint8_t* p = kbase + v_off + (long long)i * key_step + g * (S::WV * 4);
#pragma unroll
        for (int b = 0; b < S::NV; ++b) load_words<S::WV>(vr[s][a][b], p + b * (S::WV * 32), i != 0xffffffffu);
      }
  };

  Place p0[S::IDX], p1[S::IDX], p2[S::IDX];        // with their position, with their page
#pragma unroll
  for (int j = 0; j < S::IDX; ++j) {
    p0[j] = place(v, j);
    p2[j] = place(v + step, j);
    p1[j] = place(v + 2 * step, j);
  }
#pragma unroll
  for (int j = 0; j < S::IDX; ++j) {
    page_at(p0[j]);
    page_at(p2[j]);
  }
  // ---- Q as the columns of S^T, and the factor that takes a column to base-2 logits
  uint32_t qf[NT][S::NK][S::CK / 2];
  float xs[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = n * 8 + g;
    const T* src = static_cast<const T*>(P.q) + (long long)row * P.q_stride + (long long)(h0 + h) * D;
    uint32_t w[S::NK][S::CK / 2];
#pragma unroll
    for (int b = 0; b < S::NK; ++b)
#pragma unroll
      for (int c = 0; c < S::CK / 8; ++c) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (h < heads) r = *reinterpret_cast<const uint4*>(src + (b * 4 + t) * S::CK + c * 8);
        w[b][4 * c] = r.x; w[b][4 * c + 1] = r.y; w[b][4 * c + 2] = r.z; w[b][4 * c + 3] = r.w;
      }
    if constexpr (FMT == POD_KV_16BIT) {
      xs[n][0] = xs[n][1] = P.scale_log2;
#pragma unroll
      for (int b = 0; b < S::NK; ++b)
#pragma unroll
        for (int i = 0; i < S::CK / 2; ++i) qf[n][b][i] = w[b][i];
    } else {
      // fp16 operands: the row by the power of two that brings its largest element to
      // [2^14, 2^15), so that bf16 rows keep all bits down to 2^-38 of it
      float am = 0.f;
#pragma unroll
      for (int b = 0; b < S::NK; ++b)
#pragma unroll
        for (int i = 0; i < S::CK / 2; ++i) {
          const float2 f = Pack<T>::unpack(w[b][i]);
          am = fmaxf(am, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const int ex = (int)(__float_as_uint(am) >> 23) - 127;            // (-127: zeros and subnormals)
      const int e = ex >= 128 ? 0 : min(14 - ex, 126);
      const float up = __uint_as_float((uint32_t)(127 + e) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int b = 0; b < S::NK; ++b)
#pragma unroll
        for (int i = 0; i < S::CK / 2; ++i) {
          const float2 f = Pack<T>::unpack(w[b][i]);
          qf[n][b][i] = Pack<M>::two(f.x * up, f.y * up);
        }
      const float d0 = __shfl_sync(0xffffffffu, down, 8 * t), d1 = __shfl_sync(0xffffffffu, down, 8 * t + 4);
      xs[n][0] = d0 * P.scale_log2;
      xs[n][1] = d1 * P.scale_log2;
    }
  }

#pragma unroll
  for (int j = 0; j < S::IDX; ++j) idx[j] = index_of(p0[j]);
  if (v < v1) {
    load_k();
    load_v();
  }
  for (; v < v1; v += step) {
#pragma unroll
    for (int j = 0; j < S::IDX; ++j) {
      seen[j] = __ballot_sync(0xffffffffu, idx[j] != 0xffffffffu);
      idx[j] = index_of(p2[j]);
      p2[j] = p1[j];
      page_at(p2[j]);
      p1[j] = place(v + 3 * step, j);
    }
    // The next tile's rows set out for L2, a lane a key, before there are registers for them
    // (block-scaled FP8 263 -> 250 us, 16 query heads a KV head over it 350 -> 308; 16-bit rows 336 ->
    // 332 and 378 -> 360). Rows of 64 bytes would bring in their neighbours (158 -> 173), and pages of one
    // slot ask for too many places at once (279 -> 488, in HND 330 -> 593; of two slots 269 and 261, of four
    // 259 -> 250).
    if (D * S::E >= 128 && P.ps >= 4) {
#pragma unroll
      for (int j = 0; j < S::IDX; ++j)
        if (idx[j] != 0xffffffffu) {
          const uint8_t* p = kbase + (long long)idx[j] * key_step;
#pragma unroll
          for (int c = 0; c < D * S::E; c += 128) {
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p + c));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p + v_off + c));
          }
        }
    }
    // ---- S^T, a key a row (g, g + 8 of every 16), the heads 2t and 2t + 1 of every 8
    float x[MT][NT][4];
#pragma unroll
    for (int s = 0; s < MT; ++s) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[s][n][c] = 0.f;
#pragma unroll
      for (int b = 0; b < S::NK; ++b) {
#pragma unroll
        for (int i = 0; i < S::WK / 2; ++i) {
          const uint32_t* w0 = kr[s][0][b];
          const uint32_t* w1 = kr[s][1][b];
          if constexpr (FMT == POD_KV_16BIT) {
            const uint32_t a[4] = {w0[2 * i], w1[2 * i], w0[2 * i + 1], w1[2 * i + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<MBF>(x[s][n], a, qf[n][b][2 * i], qf[n][b][2 * i + 1]);
          } else {
#pragma unroll
            for (int j = 2 * i; j < 2 * i + 2; ++j) {
              const uint32_t a[4] = {e4m3x2_to<__half>((uint16_t)w0[j]), e4m3x2_to<__half>((uint16_t)w1[j]),
                                     e4m3x2_to<__half>((uint16_t)(w0[j] >> 16)),
                                     e4m3x2_to<__half>((uint16_t)(w1[j] >> 16))};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<MBF>(x[s][n], a, qf[n][b][2 * j], qf[n][b][2 * j + 1]);
            }
          }
        }
      }
    }
    float k_of[S::IDX], v_of[S::IDX];            // K's scale and V's exponent of the lane's own keys
    if constexpr (FMT == POD_KV_E4M3_BLOCK) {
#pragma unroll
      for (int j = 0; j < S::IDX; ++j) {
        k_of[j] = pow2_of((int)ek[j]);
        v_of[j] = (float)((int)ev[j] - 127);
      }
    }
    load_k();
    // ---- logits, the references, the weights
    float xe[MT][2];                             // V's exponents of the lane's keys
    bool past = false;
#pragma unroll
    for (int s = 0; s < MT; ++s)
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int src = (s & 1) * 16 + a * 8 + g;
        const bool live = seen[s / 2] >> src & 1;
        float ks = 1.f;
        xe[s][a] = 0.f;
        if constexpr (FMT == POD_KV_E4M3_BLOCK) {
          ks = __shfl_sync(0xffffffffu, k_of[s / 2], src);
          xe[s][a] = __shfl_sync(0xffffffffu, v_of[s / 2], src);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float& y = x[s][n][2 * a + c];
            // (the two scales first: each by itself may take the product out of fp32)
            if constexpr (FMT == POD_KV_E4M3_BLOCK) y = live ? y * (ks * xs[n][c]) : -INFINITY;
            else y = live ? y * xs[n][c] : -INFINITY;
            past |= y > __fadd_rd(r[n][c], kUp + kLag);
          }
        if constexpr (FMT == POD_KV_E4M3_BLOCK)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float t0, t1;
            const uint64_t e2 = add2(pack2(x[s][n][2 * a], x[s][n][2 * a + 1]), pack2(-r[n][0], -r[n][1]));
            unpack2(add2(e2, pack2(xe[s][a], xe[s][a])), t0, t1);
            past |= t0 > rv[n][0] + (kUp + kLag) || t1 > rv[n][1] + (kUp + kLag);
          }
      }
    if (__any_sync(0xffffffffu, past)) {
      auto below = [](float top) { return kUp > 0.f ? __fadd_ru(top, -kUp) : top - kUp; };
      auto most = [&](int n, int c, auto value) {
        float top = -INFINITY;
#pragma unroll
        for (int s = 0; s < MT; ++s)
#pragma unroll
          for (int a = 0; a < 2; ++a) top = fmaxf(top, value(x[s][n][2 * a + c], xe[s][a]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        return top;
      };
      float to[NT][2], tov[NT][2];                 // the new r; the largest of logit and exponent
      bool large = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float top = most(n, c, [](float y, float) { return y; });
          if constexpr (FMT == POD_KV_E4M3_BLOCK) tov[n][c] = most(n, c, [](float y, float e) { return y + e; });
          to[n][c] = fmaxf(r[n][c], below(top));
          large |= fabsf(top) >= kFar && top > kNoKey;
        }
      if constexpr (FMT == POD_KV_E4M3_BLOCK) {
        const bool far = __any_sync(0xffffffffu, large);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tov[n][c] -= to[n][c];
            if (far) tov[n][c] = most(n, c, [&](float y, float e) { return y - to[n][c] + e; });
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float by = r[n][c] - to[n][c];
          float f = ex2(by);
          r[n][c] = to[n][c];
          l[n][c] *= f;
          if constexpr (FMT == POD_KV_E4M3_BLOCK) {
            const float old = rv[n][c] + by;
            rv[n][c] = fmaxf(old, below(tov[n][c]));
            f = ex2(old - rv[n][c]);
          }
#pragma unroll
          for (int b = 0; b < S::NV; ++b)
#pragma unroll
            for (int i = 0; i < S::CV / 2; ++i) {
              o[n][b][i][c] *= f;
              o[n][b][i][2 + c] *= f;
            }
        }
    }
    uint32_t ph[MT][NT][2], pl[MT][NT][2];       // P^T as operand: keys 2t.., 2t + 8..; head g
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int s = 0; s < MT; ++s)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          float e0, e1;
          const uint64_t e2 = add2(pack2(x[s][n][2 * a], x[s][n][2 * a + 1]), pack2(-r[n][0], -r[n][1]));
          unpack2(e2, e0, e1);
          float p0 = ex2(e0), p1 = ex2(e1);
          l[n][0] += p0;
          l[n][1] += p1;
          if constexpr (FMT == POD_KV_E4M3_BLOCK) {
            unpack2(add2(add2(e2, pack2(xe[s][a], xe[s][a])), pack2(-rv[n][0], -rv[n][1])), e0, e1);
            p0 = ex2(e0);
            p1 = ex2(e1);
          }
          if constexpr (S::PARTS == 2) {
            uint32_t hi, lo;
            if constexpr (MBF) {
              Pack<M>::split(p0, p1, hi, lo);
            } else {
              hi = Pack<M>::two(p0, p1);
              const float2 h = Pack<M>::unpack(hi);
              lo = Pack<M>::two((p0 - h.x) * 0x1p11f, (p1 - h.y) * 0x1p11f);
            }
            ph[s][n][a] = turn8x8(hi);
            pl[s][n][a] = turn8x8(lo);
          } else {
            ph[s][n][a] = turn8x8(Pack<M>::two(p0, p1));
          }
        }
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int s = 0; s < MT; ++s)
#pragma unroll
      for (int b = 0; b < S::NV; ++b)
#pragma unroll
        for (int w = 0; w < S::WV; ++w) {
          const uint32_t v0w = vr[s][0][b][w], v1w = vr[s][1][b][w], v2w = vr[s][2][b][w], v3w = vr[s][3][b][w];
          if constexpr (FMT == POD_KV_16BIT) {
            const uint32_t a[4] = {prmt(v0w, v1w, 0x5410), prmt(v0w, v1w, 0x7632), prmt(v2w, v3w, 0x5410),
                                   prmt(v2w, v3w, 0x7632)};
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_parts<MBF, S::PARTS>(o[n][b][w], a, ph[s][n], pl[s][n]);
          } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t lo = prmt(v0w, v1w, q ? 0x7362 : 0x5140), hi = prmt(v2w, v3w, q ? 0x7362 : 0x5140);
              const uint32_t a[4] = {e4m3x2_to<__half>((uint16_t)lo), e4m3x2_to<__half>((uint16_t)(lo >> 16)),
                                     e4m3x2_to<__half>((uint16_t)hi), e4m3x2_to<__half>((uint16_t)(hi >> 16))};
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_parts<MBF, S::PARTS>(o[n][b][2 * w + q], a, ph[s][n], pl[s][n]);
            }
          }
        }
    load_v();
  }

  // ---- the warps' sums join
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], d);
      if (g == 0) {
        const int h = n * 8 + 2 * t + c;
        sh.m[0][warp][h] = r[n][c];
        sh.m[1][warp][h] = l[n][c];
        if constexpr (FMT == POD_KV_E4M3_BLOCK) sh.m[2][warp][h] = rv[n][c];
      }
    }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float* dst = sh.o[warp][n * 8 + 2 * t + c];
#pragma unroll
      for (int b = 0; b < S::NV; ++b)
#pragma unroll
        for (int i = 0; i < S::CV / 4; ++i)
          *reinterpret_cast<float4*>(dst + (b * 8 + g) * S::CV + 4 * i) =
              make_float4(o[n][b][2 * i][c], o[n][b][2 * i][2 + c], o[n][b][2 * i + 1][c], o[n][b][2 * i + 1][2 + c]);
    }
  __syncthreads();
}

// The sum of a CTA's n <= 4 pieces at one float4 of a row, normalised, and in `at` the row's
// reference and the sum of its weights;
// `lanes` neighbouring lanes with n pieces each share it. Piece w has its r, l and O's
// reference from r on at stat(w, 0..2) and its O at value(w).
template <int FMT, typename A, typename B>
POD_DEV float4 join(int n, int lanes, float v_scale, float2& at, A stat, B value) {
  float m[kDecodeWarps], mo[kDecodeWarps], l[kDecodeWarps];
  float4 p[kDecodeWarps];
  float top = -INFINITY, topv = -INFINITY;
#pragma unroll
  for (int w = 0; w < kDecodeWarps; ++w) {
    m[w] = -INFINITY;
    mo[w] = l[w] = 0.f;
    p[w] = make_float4(0, 0, 0, 0);
    if (w >= n) continue;
    m[w] = stat(w, 0);
    l[w] = stat(w, 1);
    if constexpr (FMT == POD_KV_E4M3_BLOCK) mo[w] = stat(w, 2);
    p[w] = value(w);
    top = fmaxf(top, m[w]);
  }
  for (int o = 1; o < lanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
  for (int w = 0; w < kDecodeWarps; ++w) {
    m[w] -= top;
    mo[w] += m[w];
    topv = fmaxf(topv, mo[w]);
  }
  if constexpr (FMT == POD_KV_E4M3_BLOCK)
    for (int o = 1; o < lanes; o <<= 1) topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, o));
  float sum = 0.f;
  float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
  for (int w = 0; w < kDecodeWarps; ++w) {
    const float f = ex2(m[w]), fv = FMT == POD_KV_E4M3_BLOCK ? ex2(mo[w] - topv) : f;
    sum += l[w] * f;
    acc.x += p[w].x * fv; acc.y += p[w].y * fv; acc.z += p[w].z * fv; acc.w += p[w].w * fv;
  }
  for (int o = 1; o < lanes; o <<= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
  }
  // (sum == 0: no visible key; a NaN stays one)
  at = make_float2(top, sum);
  const float f = sum == 0.f ? 0.f : v_scale / sum;
  acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
  if constexpr (FMT == POD_KV_E4M3_BLOCK) {
    // O's own reference, in two steps (2^-127, the smallest scale, is 0 to the exponential)
    const float back = ex2(0.5f * topv);
    acc.x = acc.x * back * back; acc.y = acc.y * back * back;
    acc.z = acc.z * back * back; acc.w = acc.w * back * back;
  }
  return acc;
}

// base-2 LSE of a row
POD_DEV float lse_of(float2 at) { return at.y == 0.f ? -INFINITY : at.x + log2f(at.y); }

template <typename T>
POD_DEV void store_out(const DecodeParams& P, int row, int head, int D, int c4, float4 o, float2 at) {
  const float lse = lse_of(at);
  if (P.sinks && lse != -INFINITY) {
    const float f = sink_factor(lse, P.sinks[head]);
    o.x *= f; o.y *= f; o.z *= f; o.w *= f;
  }
  T* dst = static_cast<T*>(P.out) + (long long)row * P.out_stride + (long long)head * D + 4 * c4;
  *reinterpret_cast<uint2*>(dst) = make_uint2(Pack<T>::two(o.x, o.y), Pack<T>::two(o.z, o.w));
  if (c4 == 0 && P.lse) P.lse[(long long)row * P.H + head] = lse;
}

template <typename T, int D, int FMT, int NT>
__global__ void __launch_bounds__(kDecodeThreads, (D == 256 || NT == 2) ? 2 : 3)
    decode_kernel(const __grid_constant__ DecodeParams P) {
  using S = DecodeShape<T, D, FMT, NT>;
  constexpr int HT = S::HT;
  __shared__ DecodeShared<D, HT> sh;
  __shared__ long long sh_scan[kDecodeWarps], sh_rest[kDecodeWarps], sh_first;
  __shared__ int sh_row;

  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int parts = kDecodeWarps / P.hw, unit = S::TK * parts;      // warps of a KV head, keys of a unit

  // ---- this CTA's run of units. The first requests, a thread one, are scanned once; those
  // behind them are summed, and scanned where the run begins among them.
  auto units_of = [&](int r) { return r < P.batch ? (long long)((keys_of(P, r).count + unit - 1) / unit) : 0ll; };
  auto scan = [&](long long n) {                   // the sum up to this thread's, within its warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += y;
    }
    return n;
  };
  long long n = units_of(tid), x = scan(n), rest = 0;
  for (int r = tid + kDecodeThreads; r < P.batch; r += kDecodeThreads) rest += units_of(r);
  if (P.batch > kDecodeThreads)
#pragma unroll
    for (int o = 16; o; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
  if (lane == 31) {
    sh_scan[warp] = x;
    sh_rest[warp] = rest;
  }
  if (tid == 0) sh_row = -1;
  __syncthreads();
  long long total = 0, head = 0;                   // units of a plane, and of the scanned requests
#pragma unroll
  for (int w = 0; w < kDecodeWarps; ++w) {
    head += sh_scan[w];
    total += sh_rest[w];
  }
  total += head;
  if (blockIdx.x == 0 && tid == 0) *P.total = total;
  const long long all = total * P.planes, runs = min((long long)P.grid, all);
  if (blockIdx.x >= runs) return;                  // (as many runs as units at most: none is empty)
  long long u = quotient(all * blockIdx.x, runs);
  const long long u_end = quotient(all * (blockIdx.x + 1), runs), u_start = u;
  int plane = (int)quotient(u, total);
  // the request of the first unit
  const long long at = u - (long long)plane * total;   // unit within the plane
  long long before = 0;                            // units of the requests up to this round
  for (int base = 0;; base += kDecodeThreads) {
    if (base) {
      n = units_of(base + tid);
      x = scan(n);
      __syncthreads();                             // (sh_scan is read)
      if (lane == 31) sh_scan[warp] = x;
      __syncthreads();
    }
    long long off = before;
#pragma unroll
    for (int w = 0; w < kDecodeWarps; ++w) {
      if (w < warp) off += sh_scan[w];
      before += sh_scan[w];
    }
    if (at >= off + x - n && at < off + x) {
      sh_row = base + tid;
      sh_first = off + x - n;
    }
    __syncthreads();
    if (sh_row >= 0 || base + kDecodeThreads >= P.batch) break;
  }
  int row = sh_row;
  long long row_first = sh_first;                  // first unit of the request in its plane

  // ---- segments: the units of one (plane, request)
  while (u < u_end) {
    const Keys K = keys_of(P, row);
    const int units = (K.count + unit - 1) / unit;
    if (units == 0) {                              // (an empty request: the merge kernel's)
      if (++row == P.batch) { row = 0; row_first = 0; ++plane; }
      continue;
    }
    const long long seg0 = (long long)plane * total + row_first;      // of the whole request
    const int ua = (int)(u - seg0), ub = (int)min((long long)units, u_end - seg0);
    const int groups = P.Hk / P.hw, hk0 = plane % groups * P.hw, tile0 = plane / groups * HT;
    const int heads = min(HT, P.G - tile0);        // of every KV head
    if (tid == 0 && plane == 0 && ua == 0) P.first[row] = row_first;
    {
      const int hk = hk0 + warp % P.hw;
      attend<T, D, FMT, NT>(P, K, row, hk, hk * P.G + tile0, heads, ua * unit + warp / P.hw * S::TK, unit,
                            (int)min((long long)K.count, (long long)ub * unit), sh);
    }
    const bool whole = ua == 0 && ub == units;
    const int slot = (int)blockIdx.x * 2 + (u == u_start ? 0 : 1);
    for (int i = tid; i < P.hw * heads * (D / 4); i += kDecodeThreads) {
      const int c4 = i % (D / 4), k = i / (D / 4) / heads, h = i / (D / 4) - k * heads;   // of KV head hk0 + k
      float2 at;
      const float4 o = join<FMT>(parts, 1, P.v_scale, at,
                                 [&](int w, int what) { return sh.m[what][k + w * P.hw][h]; },
                                 [&](int w) { return *reinterpret_cast<const float4*>(&sh.o[k + w * P.hw][h][4 * c4]); });
      if (whole) {
        store_out<T>(P, row, (hk0 + k) * P.G + tile0 + h, D, c4, o, at);
      } else {
        const long long piece = ((long long)slot * P.hw + k) * HT + h;
        *reinterpret_cast<float4*>(P.piece_o + piece * D + 4 * c4) = o;
        if (c4 == 0) P.piece_at[piece] = at;
      }
    }
    __syncthreads();                               // (the buffers are the next segment's)
    u = seg0 + ub;
    row_first += units;
    if (++row == P.batch) { row = 0; row_first = 0; ++plane; }
  }
}

// Short rows: a cluster of CL CTAs for each (plane, request), which share its units and join
// them through each other's shared memory: one launch, no workspace.
template <typename T, int D, int FMT, int NT, int CL>
__global__ void __launch_bounds__(kDecodeThreads, (D == 256 || NT == 2) ? 2 : 3)
    decode_short_kernel(const __grid_constant__ DecodeParams P) {
  using S = DecodeShape<T, D, FMT, NT>;
  constexpr int HT = S::HT;
  __shared__ DecodeShared<D, HT> sh;
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;
  const int item = (int)(blockIdx.x / CL), plane = item / P.batch, row = item - plane * P.batch;
  const Keys K = keys_of(P, row);
  constexpr int U = S::TK * kDecodeWarps;          // keys of a unit
  const int units = (K.count + U - 1) / U;
  const int hk = plane % P.Hk, h0 = hk * P.G + plane / P.Hk * HT;
  const int heads = min(HT, P.G - plane / P.Hk * HT);
  if (plane == 0 && rank == 0 && tid == 0 && P.status && P.lens[row] != K.len) atomicOr(P.status, kStatusSlot);
  const int v0 = units * rank / CL * U, v1 = min(K.count, units * (rank + 1) / CL * U);
  attend<T, D, FMT, NT>(P, K, row, hk, h0, heads, v0 + (tid >> 5) * S::TK, U, v1, sh);
  if (CL > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  // CL neighbouring threads join one float4, each the four pieces of a CTA
  const uint32_t mine = smem_u32(&sh);
  uint32_t base = mine;
  if (CL > 1) asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base) : "r"(mine), "r"(tid % CL));
  const int per = kDecodeThreads / CL;             // float4s of a CTA at a time
  for (int i0 = rank * per; i0 < heads * (D / 4); i0 += per * CL) {
    const int i = i0 + tid / CL, j = min(i, heads * (D / 4) - 1), h = j / (D / 4), c4 = j - h * (D / 4);
    float2 at;
    const float4 o = join<FMT>(
        kDecodeWarps, CL, P.v_scale, at,
        [&](int w, int what) {
          float x;
          const uint32_t a = base + (uint32_t)offsetof_m<D, HT>(what, w, h);
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
          return x;
        },
        [&](int w) {
          float4 x;
          const uint32_t a = base + (uint32_t)(((w * HT + h) * D + 4 * c4) * 4);
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(a) : "memory");
          return x;
        });
    if (i == j && tid % CL == 0) store_out<T>(P, row, h0 + h, D, c4, o, at);
  }
  if (CL > 1)                                      // (nobody leaves while others read its memory)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Rows whose keys were cut: the pieces in the order of the keys, weighted by
// sum * 2^(reference - M). Rows without keys: 0 and -inf. WPR warps work on a (request, head).
template <typename T, int D, int HT, int TK, int WPR>
__global__ void __launch_bounds__(128) decode_merge_kernel(const __grid_constant__ DecodeParams P) {
  constexpr int PL = D / 32 < 4 ? D / 32 : 4, NP = D / (32 * PL);      // elements and chunks of a lane
  __shared__ float sh[WPR > 1 ? WPR : 1][D];
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = WPR > 1 ? (long long)blockIdx.x : (long long)blockIdx.x * 4 + warp;
  if (item >= (long long)P.batch * P.H) return;    // (uniform over the block where its warps meet)
  const int row = (int)quotient(item, P.H), head = (int)(item - (long long)row * P.H);
  const long long total = *P.total, first = P.first[row];           // (beside the length; of no use for an empty row)
  const Keys K = keys_of(P, row);
  const int unit = TK * (kDecodeWarps / P.hw), units = (K.count + unit - 1) / unit;
  T* out = static_cast<T*>(P.out) + (long long)row * P.out_stride + (long long)head * D;
  if (head == 0 && (threadIdx.x & (WPR * 32 - 1)) == 0 && P.status && P.lens[row] != K.len) atomicOr(P.status, kStatusSlot);
  if (units == 0) {
    if (WPR > 1 && warp) return;
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int e = 0; e < PL; e += 2)
        *reinterpret_cast<uint32_t*>(out + (j * 32 + lane) * PL + e) = 0u;
    if (lane == 0 && P.lse) P.lse[item] = -INFINITY;
    return;
  }
  const int hk = head / P.G, gh = head - hk * P.G, h = hk % P.hw * HT + gh % HT, per = P.hw * HT;
  const long long plane = (long long)(gh / HT) * (P.Hk / P.hw) + hk / P.hw, all = total * P.planes;
  const long long runs = min((long long)P.grid, all);
  const long long g0 = plane * total + first, g1 = g0 + units;
  const int c0 = (int)quotient((g0 + 1) * runs - 1, all), c1 = (int)quotient(g1 * runs - 1, all);   // CTAs of the first and last unit
  if (c0 == c1) return;                            // written whole
  const int w0 = WPR > 1 ? warp : 0, n = c1 - c0 + 1;
  // piece k of the row: the CTA's first segment, or its second where the row begins inside its run
  const bool inside = quotient(all * c0, runs) != g0;
  auto at_of = [&](int k) { return P.piece_at[((long long)2 * (c0 + k) + (k == 0 && inside)) * per + h]; };
  // The largest reference, then the weights, a lane a piece; the first pieces are asked for beside
  // the references.
  constexpr int U = WPR > 1 ? 8 : 4;               // pieces in flight
  float x[U][NP][PL];
  auto load = [&](int k0, int end) {               // pieces k0, k0 + WPR, ... (the last one for those past the end)
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = min(k0 + i * WPR, end - 1);
      const float* src = P.piece_o + (((long long)2 * (c0 + k) + (k == 0 && inside)) * per + h) * D + lane * PL;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        if constexpr (PL == 4) *reinterpret_cast<float4*>(x[i][j]) = *reinterpret_cast<const float4*>(src + j * 128);
        else *reinterpret_cast<float2*>(x[i][j]) = *reinterpret_cast<const float2*>(src);
      }
    }
  };
  float top = -INFINITY, sum = 0.f;
  const float2 none = make_float2(-INFINITY, 0.f);
  float2 mine = lane < n ? at_of(lane) : none;
  load(w0, n);
  for (int k = lane; k < n; k += 32) top = fmaxf(top, k == lane ? mine.x : at_of(k).x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float acc[NP][PL];
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int e = 0; e < PL; ++e) acc[j][e] = 0.f;
  for (int k32 = 0; k32 < n; k32 += 32) {
    if (k32) mine = k32 + lane < n ? at_of(k32 + lane) : none;
    const float f = k32 + lane < n ? mine.y * ex2(mine.x - top) : 0.f;
    sum += f;                                      // (of all warps' pieces: every warp has them)
    const int end = min(32, n - k32);
    for (int k0 = w0; k0 < end; k0 += WPR * U) {
      if (k32 + k0 != w0) load(k32 + k0, n);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float w = __shfl_sync(0xffffffffu, f, min(k0 + i * WPR, 31));
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
          for (int e = 0; e < PL; ++e) acc[j][e] += k0 + i * WPR < end ? x[i][j][e] * w : 0.f;
      }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if constexpr (WPR > 1) {
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int e = 0; e < PL; ++e) sh[warp][(j * 32 + lane) * PL + e] = acc[j][e];
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        acc[j][e] = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) acc[j][e] += sh[w][(j * 32 + lane) * PL + e];
      }
  }
  const float lse = lse_of(make_float2(top, sum));
  float f = sum == 0.f ? 0.f : 1.f / sum;
  if (P.sinks && sum != 0.f) f *= sink_factor(lse, P.sinks[head]);
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int e = 0; e < PL; e += 2)
      *reinterpret_cast<uint32_t*>(out + (j * 32 + lane) * PL + e) = Pack<T>::two(acc[j][e] * f, acc[j][e + 1] * f);
  if (lane == 0 && P.lse) P.lse[item] = lse;
}

template <typename T, int D, int FMT, int NT>
cudaError_t launch_decode_nt(DecodeParams& P, cudaStream_t st) {
  using S = DecodeShape<T, D, FMT, NT>;
  const int tiles = (P.G + S::HT - 1) / S::HT;
  constexpr int per_sm = (D == 256 || NT == 2) ? 2 : 3;
  P.grid = 152 * per_sm;
  // A CTA's warps take four KV heads instead of four parts of one head's keys where a head's
  // rows in a page of an NHD cache are few: neighbouring heads' rows are neighbours in memory.
  // (96 block-scaled requests with pages of one slot 334 -> 280 us, of two 273 -> 270, per-tensor
  // scales 304 -> 262; with pages of 16 slots nothing to 2 %; one long request, whose pieces get four
  // times as many, 91 -> 111.)
  P.hw = !P.hnd && P.ps < 8 && P.Hk % 4 == 0 && (long long)P.batch * P.Hk * tiles >= P.grid ? 4 : 1;
  P.planes = P.Hk / P.hw * tiles;
  // Units of the longest row that the table (the list of pages, the window) allows.
  const long long items = (long long)P.batch * P.planes;
  constexpr int U = S::TK * kDecodeWarps;
  const long long keys = P.pages ? (long long)min(P.num_selected, P.width) * P.ps
                                 : min((long long)P.width * P.ps, P.window < 0 ? LLONG_MAX : P.window + 1ll);
  const long long units = (keys + U - 1) / U, pairs = (long long)P.batch * P.Hk * tiles;
  // Short rows: one CTA, or a cluster of two, four or eight, for each (request, plane), while its
  // CTAs get at most eight units each; half the cluster where they would get fewer than two. A
  // cluster's launch costs time that grows with its size, so no more than kShortCtas CTAs come in
  // clusters. (us with 1 / 2 / 4 / 8 CTAs and split over the GPU, bf16, 8 KV heads: 1 request of
  // 256 keys 5.4 / 4.9 / 4.6 / 6.1 / 8.4, of 2048 keys 25.5 / 15.2 / 9.9 / 8.6 / 10.1; 4 of 512
  // 8.7 / 6.9 / 7.1 / 9.2 / 10.8; 8 of 2048 39.7 / 25.3 / 18.7 / 27.3 / 23.3; 16 of 1024
  // 24.1 / 18.0 / 24.0 / 32.8 / 23.0; 32 of 512 17.0 / 22.7 / 27.1 / 47.5 / 23.3; 128 of 64 to
  // 512 31.9 / 41.9 / 71.1 / 169 / 42.0. 128 of 1024: 95.0 by one CTA each, 92.0 split.)
  int cl = 1;
  while (cl < 8 && pairs * cl * 2 <= kShortCtas) cl *= 2;
  if (P.hw == 1 && pairs <= INT_MAX && units <= kShortUnits * cl) {
    while (cl > 1 && units < 2 * cl) cl /= 2;
    const auto kernel = cl == 1 ? decode_short_kernel<T, D, FMT, NT, 1> : cl == 2 ? decode_short_kernel<T, D, FMT, NT, 2>
                      : cl == 4 ? decode_short_kernel<T, D, FMT, NT, 4> : decode_short_kernel<T, D, FMT, NT, 8>;
    return launch_beside(kernel, (unsigned)(pairs * cl), kDecodeThreads, 0, (unsigned)cl, st, P);
  }
  cudaError_t e = launch_beside(decode_kernel<T, D, FMT, NT>, (unsigned)P.grid, kDecodeThreads, 0, 1, st, P);
  if (e != cudaSuccess) return e;
  // A warp for each (request, head), or a block of four where a row may have many pieces (one
  // long request 88 us, 94 by single warps; 32 x 8 (request, KV head) pairs 106 and 103).
  const long long rows = (long long)P.batch * P.H;
  if (items * 4 <= P.grid) return launch_beside(decode_merge_kernel<T, D, S::HT, S::TK, 4>, (unsigned)rows, 128, 0, 1, st, P);
  return launch_beside(decode_merge_kernel<T, D, S::HT, S::TK, 1>, (unsigned)((rows + 3) / 4), 128, 0, 1, st, P);
}

template <typename T, int FMT>
cudaError_t launch_decode(int d, DecodeParams& P, cudaStream_t st) {
  // (16 query heads a KV head: 359 us for 64 ragged requests over bf16, 321 for 96 over
  // block-scaled FP8; as two tiles of eight 457 and 456 before rows were asked for ahead, when one
  // tile took 380 and 350. Heads of 256 go as two tiles, which read the keys twice: 435 and 445 us,
  // of 343 and 229 at the copy rate.)
  const bool wide = P.G > 8;
  switch (d) {
    case 64: return wide ? launch_decode_nt<T, 64, FMT, 2>(P, st) : launch_decode_nt<T, 64, FMT, 1>(P, st);
    case 128: return wide ? launch_decode_nt<T, 128, FMT, 2>(P, st) : launch_decode_nt<T, 128, FMT, 1>(P, st);
    default: return launch_decode_nt<T, 256, FMT, 1>(P, st);   // (O of 16 heads would not fit the registers)
  }
}

}  // namespace
}  // namespace pod
