// pod_select.cu — which pages of a long cache a decode step attends: the bounds of
// every page's keys, and the choice of the pages whose bounds promise a query the most.
//
// Mathematics. With the smallest m_j and the largest M_j of every channel over a
// page's keys, max(q_j m_j, q_j M_j) bounds q_j k_j from above, so its sum over j
// bounds the logit. The score of a page is the sum of these bounds over the G query
// heads of a KV head, and that is one product, whatever G is:
//   sum_g sum_j max(q_gj m_j, q_gj M_j) = sum_j M_j up_j + m_j down_j,
//   up_j = sum_g max(q_gj, 0), down_j = sum_g min(q_gj, 0).
//
// The choice is that of the scores in 64 bits, without computing them so: an fp32
// score is off by at most E = (10 + G) 2^-24 times the sum of its terms' magnitudes (4
// fused steps a lane, 8 at D = 256, six additions, G - 1 in a weight), of which
// a bound is kept per warp. Pages further than 2 E from the last place are decided;
// the others, where they are more than the places left, are scored again in 64
// bits (of which this GPU does two a clock and SM).
#include <cuda_runtime.h>
#include <math.h>

#include <string>

#include "../../include/pod.h"
#include "pod_beside.h"
#include "pod_decode.h"
#include "pod_device.cuh"

void pod_set_last_error(const std::string& msg);

using namespace pod;

namespace {

constexpr int kBoundThreads = 256, kBoundRows = 256;
constexpr int kScoreThreads = 128, kLeastPages = 16;   // pages of a warp at least
constexpr int kBinBits = 10, kBins = 1 << kBinBits, kNear = 256;
constexpr int kPickThreads = 512;                      // at most
constexpr int kHeldPages = kPickThreads * 16;          // pages whose keys a block holds

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static constexpr float kMax = 3.3895313892515355e38f;
  static POD_DEV __nv_bfloat16 down(float x) { return __float2bfloat16_rd(x); }
  static POD_DEV __nv_bfloat16 up(float x) { return __float2bfloat16_ru(x); }
};
template <>
struct Pair<__half> {
  using type = __half2;
  static constexpr float kMax = 65504.f;
  static POD_DEV __half down(float x) { return __float2half_rd(x); }
  static POD_DEV __half up(float x) { return __float2half_ru(x); }
};
// element by element; a NaN loses against a number
template <typename T>
POD_DEV uint32_t min2(uint32_t a, uint32_t b) {
  using P = typename Pair<T>::type;
  const P r = __hmin2(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
POD_DEV uint32_t max2(uint32_t a, uint32_t b) {
  using P = typename Pair<T>::type;
  const P r = __hmax2(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// the larger magnitudes (the signs are of no use)
template <typename T>
POD_DEV uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (Pack<T>::kBF16) asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// ------------------------------------------------------------------ bounds
struct BoundParams {
  const uint8_t* cache;
  const uint8_t* scales;
  void* bounds;
  const int64_t* slots;
  int32_t* status;
  long long rows, num_slots;
  int ps, Hk, hnd, span;
  float k_scale;
};

// x within +-most; a NaN stays one
POD_DEV float within(float x, float most) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-most));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(most));
  return x;
}
// Two values rounded outward to T, within its finite values.
template <typename T>
POD_DEV uint32_t outward2(float x, float y, bool upper) {
  x = within(x, Pair<T>::kMax);
  y = within(y, Pair<T>::kMax);
  T r[2] = {upper ? Pair<T>::up(x) : Pair<T>::down(x), upper ? Pair<T>::up(y) : Pair<T>::down(y)};
  return (uint32_t)*reinterpret_cast<uint16_t*>(&r[0]) | (uint32_t)*reinterpret_cast<uint16_t*>(&r[1]) << 16;
}

// A warp's (page, head) whose exponents lie more than 15 binades apart: in fp32, a lane some
// channels, key by key.
template <typename T, int D>
__device__ __noinline__ void bounds_of_far_scales(const BoundParams& P, const uint8_t* keys, const uint8_t* scales,
                                                  long long row_bytes, int step, int valid, long long to) {
  for (int c = 2 * (threadIdx.x & 31); c < D; c += 64) {
    float lo0 = NAN, lo1 = NAN, hi0 = NAN, hi1 = NAN;
    for (int k = 0; k < valid; ++k) {
      const int e = scales[(long long)k * step];
      const float s = e ? __uint_as_float((uint32_t)e << 23) : 5.877471754111438e-39f;
      const uint32_t a = e4m3x2_to<__half>(*reinterpret_cast<const uint16_t*>(keys + k * row_bytes + c));
      const float2 f = Pack<__half>::unpack(a);
      lo0 = fminf(lo0, f.x * s);
      hi0 = fmaxf(hi0, f.x * s);
      lo1 = fminf(lo1, f.y * s);
      hi1 = fmaxf(hi1, f.y * s);
    }
    T* dst = static_cast<T*>(P.bounds) + to + c;
    *reinterpret_cast<uint32_t*>(dst) = outward2<T>(lo0, lo1, false);
    *reinterpret_cast<uint32_t*>(dst + D) = outward2<T>(hi0, hi1, true);
  }
}

// A block takes `span` rows of the write. A row whose page differs from that of the row
// before owns the page; a warp finds how far its run of rows goes. Then a warp brings in
// the keys of one (page, head) at a time, eight channels a lane, 32 / LPR keys at once, the
// loads of a page of 16 in flight together, and keeps the extremes packed, two 16-bit values a
// register. Codes go to fp16, under block scales relative to the largest exponent of the page's
// keys: exact down to 15 binades below it (pages whose exponents lie further apart take a slow
// way). That is half the instructions of the same in fp32: 38000 pages and heads of block-scaled
// codes 45 -> 18.9 us, of per-tensor ones 15.8, of 16-bit keys 22.9 (at the copy rate 11.7, 11.6,
// 20.8). Over FP8 neither issue slots (64 %) nor memory (38 %) are full: a warp loads a page's
// keys, then works, and 32 warps an SM do not cover that. (Codes 16 a lane, with twice the extremes to join
// across lanes: 1.3 us more; branches around the keys past the last, where NaN stands now, and a
// division a page and head: 1.8. The next page's keys asked for ahead, into registers of their
// own: 2 more; 5 or 6 blocks an SM in 48 or 40 registers a thread: 2.4, 5.)
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kBoundThreads, 4) bounds_kernel(const __grid_constant__ BoundParams P) {
  // eight channels a lane: LPR lanes a key, KPL keys at a time, U of these in flight
  constexpr int E = FMT == POD_KV_16BIT ? 2 : 1, LPR = D / 8, KPL = 32 / LPR, U = 8 / E, R = 4;
  using Chunk = typename std::conditional<E == 2, uint4, uint2>::type;
  using M = typename std::conditional<FMT == POD_KV_16BIT, T, __half>::type;
  __shared__ long long page_of[kBoundRows];
  __shared__ int row_of[kBoundRows], keys_of[kBoundRows];
  __shared__ int owners;
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) owners = 0;
  __syncthreads();
  const long long row0 = (long long)blockIdx.x * P.span;
  if (tid < P.span && row0 + tid < P.rows) {
    const long long r = row0 + tid, s = P.slots[r], b = r ? P.slots[r - 1] : -1;
    if (s >= P.num_slots && P.status) atomicOr(P.status, kStatusSlot);
    if (s >= 0 && s < P.num_slots && (b < 0 || b / P.ps != s / P.ps)) {
      const int at = atomicAdd(&owners, 1);
      row_of[at] = tid;
      page_of[at] = s / P.ps;
    }
  }
  __syncthreads();
  const int n = owners;
  for (int i = warp; i < n; i += kBoundThreads / 32) {
    // the page's rows of the write stand behind the first
    const long long page = page_of[i];
    int valid = 0;
    for (long long a = row0 + row_of[i]; a < P.rows; a += 32) {
      const long long s = a + lane < P.rows ? P.slots[a + lane] : -1;
      const unsigned same = __ballot_sync(0xffffffffu, s >= page * P.ps && s - page * P.ps < P.ps);
      const int run = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
      valid = max(valid, __reduce_max_sync(0xffffffffu, lane < run ? (int)(s - page * P.ps) + 1 : 0));
      if (run < 32) break;
    }
    if (lane == 0) keys_of[i] = valid;
  }
  __syncthreads();
  const int part = lane % LPR, sub = lane / LPR;
  const long long row_bytes = (long long)D * E * (P.hnd ? 1 : P.Hk);          // from a key to the next
  // (page, head) pairs warp, warp + 8, ...: a division once
  constexpr int W = kBoundThreads / 32;
  const int o_step = W / P.Hk, h_step = W - o_step * P.Hk;
  int o = warp / P.Hk, h = warp - o * P.Hk;
  auto next = [&]() {
    o += o_step;
    h += h_step;
    if (h >= P.Hk) { h -= P.Hk; ++o; }
  };
  for (; o < n; next()) {
    const int valid = keys_of[o];
    const long long page = page_of[o];
    const long long row = page * 2 * P.Hk * P.ps + (P.hnd ? (long long)h * P.ps : h);   // of key 0, in rows of D
    const uint8_t* keys = P.cache + row * (D * E) + part * (8 * E);
    const uint8_t* scales = FMT == POD_KV_E4M3_BLOCK ? P.scales + row : nullptr;
    const int step = P.hnd ? 1 : P.Hk;
    uint32_t lo[R], hi[R];
#pragma unroll
    for (int e = 0; e < R; ++e) lo[e] = hi[e] = 0x7fff7fffu;   // (NaN, which stays where no key is a number)
    // the exponents of the page's keys, of 32 at a time, and the first keys' loads beside them
    int eb = 0, top = 0, low = 255;
    if (FMT == POD_KV_E4M3_BLOCK && lane < valid) eb = scales[(long long)lane * step];
    Chunk x[U], no_key;                                  // (NaN, which does not count)
    memset(&no_key, E == 2 ? 0xff : 0x7f, sizeof no_key);
    const uint8_t* at = keys + sub * row_bytes;          // of this lane's next key
    auto load = [&](int k0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[u] = no_key;
        if (k0 + u * KPL + sub < valid) x[u] = __ldcs(reinterpret_cast<const Chunk*>(at));
        at += KPL * row_bytes;
      }
    };
    load(0);
    if constexpr (FMT == POD_KV_E4M3_BLOCK) {
      if (lane < valid) top = low = eb;
      for (int k = 32 + lane; k < valid; k += 32) {
        const int e = scales[(long long)k * step];
        top = max(top, e);
        low = min(low, e);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      low = __reduce_min_sync(0xffffffffu, low);
      if (top - low > 15) {
        bounds_of_far_scales<T, D>(P, keys - part * 8, scales, row_bytes, step, valid, (page * P.Hk + h) * 2 * D);
        continue;
      }
    }
    // 2^(exponent - top), twice: fp16's exponent bias is 15, a normal number down to 2^-14
    auto factor = [&]() { return eb - top < -14 ? 0x02000200u : (uint32_t)(eb - top + 15) * 0x04000400u; };
    uint32_t mine = FMT == POD_KV_E4M3_BLOCK ? factor() : 0u;
    for (int k0 = 0; k0 < valid; k0 += KPL * U) {
      if (k0) load(k0);
      if (FMT == POD_KV_E4M3_BLOCK && k0 && k0 % 32 == 0) {
        eb = k0 + lane < valid ? scales[(long long)(k0 + lane) * step] : top;
        mine = factor();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t s = FMT == POD_KV_E4M3_BLOCK ? __shfl_sync(0xffffffffu, mine, (k0 + u * KPL + sub) & 31) : 0u;
        uint32_t w[R];
        if constexpr (E == 2) {
          w[0] = x[u].x; w[1] = x[u].y; w[2] = x[u].z; w[3] = x[u].w;
        } else {
          w[0] = e4m3x2_to<__half>((uint16_t)x[u].x);
          w[1] = e4m3x2_to<__half>((uint16_t)(x[u].x >> 16));
          w[2] = e4m3x2_to<__half>((uint16_t)x[u].y);
          w[3] = e4m3x2_to<__half>((uint16_t)(x[u].y >> 16));
        }
#pragma unroll
        for (int e = 0; e < R; ++e) {
          if constexpr (FMT == POD_KV_E4M3_BLOCK) {
            const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&w[e]), *reinterpret_cast<const __half2*>(&s));
            w[e] = *reinterpret_cast<const uint32_t*>(&y);
          }
          lo[e] = min2<M>(lo[e], w[e]);
          hi[e] = max2<M>(hi[e], w[e]);
        }
      }
    }
#pragma unroll
    for (int d = LPR; d < 32; d <<= 1)
#pragma unroll
      for (int e = 0; e < R; ++e) {
        lo[e] = min2<M>(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], d));
        hi[e] = max2<M>(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], d));
      }
    const float s = FMT == POD_KV_E4M3 ? P.k_scale
                    : FMT == POD_KV_E4M3_BLOCK ? (top ? __uint_as_float((uint32_t)top << 23) : 5.877471754111438e-39f) : 1.f;
    // the lanes that hold the same channels share their outputs: the smallest values, the largest
    T* dst = static_cast<T*>(P.bounds) + (page * P.Hk + h) * 2 * D + part * 8;
#pragma unroll
    for (int o = 0; o < 2; o += KPL) {
      const int side = o + sub;
      if (KPL > 2 && side >= 2) break;
      uint32_t w[R];
#pragma unroll
      for (int e = 0; e < R; ++e) {
        const float2 f = Pack<M>::unpack(side ? hi[e] : lo[e]);
        w[e] = outward2<T>(FMT == POD_KV_16BIT ? f.x : f.x * s, FMT == POD_KV_16BIT ? f.y : f.y * s, side);
      }
      *reinterpret_cast<uint4*>(dst + side * D) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ------------------------------------------------------------------ scores
struct PickParams {
  const void* q;
  const void* bounds;
  const int32_t* table;
  const int32_t* lens;
  int32_t* pages;
  int32_t* status;
  float* score;                    // [batch, Hk, width]
  float* off;                      // [batch, Hk, chunks]: how far a chunk's scores may be off
  double* again;                   // [batch, Hk, width]: scores computed again
  long long q_stride, table_stride;
  unsigned num_pages;
  int batch, Hk, G, width, per, chunks, ps, k, first, last;   // per: pages of a warp, a chunk
};

POD_DEV int pages_of(const PickParams& P, int row) {
  const int most = P.width * P.ps, len = P.lens[row];
  return (int)(((unsigned)min(max(len, 0), most) + P.ps - 1) / (unsigned)P.ps);
}

// A warp scores `per` pages for one head: a page's bounds are 4 D bytes, 16 a lane. Each
// lane copies its own 16 bytes of eight pages into a ring of its own in shared memory,
// two sets ahead of the one that is summed (asynchronous copies: no registers, and no
// other lane to wait for); the eight sums cross the lanes together (nine shuffles).
// Bound by memory. With the sets held in registers instead: 67 us (one set, 24 warps
// an SM) and 91 us (two sets, 16 warps) where the ring takes 56 (655000
// pages and heads of 128, 333 MB).
constexpr int kRing = 3;
constexpr int kScoreShared = kScoreThreads / 32 * kRing * 8 * 32 * 16;
static_assert(kScoreShared <= 48 * 1024, "what a launch may ask for without an attribute of the kernel");

template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads, 4) score_kernel(const __grid_constant__ PickParams P) {
  constexpr int LPP = D == 64 ? 16 : 32, NC = D == 256 ? 2 : 1, PPL = 32 / LPP, U = 8 / NC, STEP = U * PPL;
  extern __shared__ uint4 ring[];
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const unsigned task = blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5), rest = task / (unsigned)P.Hk;
  const int hk = (int)(task - rest * P.Hk), row = (int)(rest / (unsigned)P.chunks);
  const int chunk = (int)(rest - (unsigned)row * P.chunks);
  if (row >= P.batch) return;
  const int page0 = chunk * P.per;
  // (the table's entries and q do not wait for the length: one trip to memory)
  const int32_t* table = P.table + row * P.table_stride + page0;
  int id = page0 + lane < P.width && lane < P.per ? table[lane] : -1;
  int after = page0 + 32 + lane < P.width && 32 + lane < P.per ? table[32 + lane] : -1;
  const int n = pages_of(P, row), mine = min(P.per, n - page0);
  if (mine <= 0 || n <= P.k) return;                   // (n <= k: all are chosen)
  const int c = lane % LPP;
  const T* bounds = static_cast<const T*>(P.bounds) + (long long)hk * 2 * D + c * 8;
  const long long page_step = (long long)P.Hk * 2 * D;
  float* score = P.score + ((long long)row * P.Hk + hk) * P.width + page0;
  // entries 32 i + lane of the table, one set ahead
  auto checked = [&](int x, int p) {
    if (p >= mine) return -1;
    if ((unsigned)x < P.num_pages) return x;
    if (P.status) atomicOr(P.status, kStatusSlot);
    return -1;
  };
  id = checked(id, lane);                              // of the pages that are asked for
  int asked = 0, next = 0, at = 0;                     // pages asked for; the ring's sets to fill and to read
  uint4* slots = ring + (threadIdx.x >> 5) * (kRing * 256) + lane;
  auto ask = [&]() {
    if (asked < mine) {
      if (asked && asked % 32 == 0) {
        id = checked(after, asked + lane);
        after = asked + 32 + lane < mine ? table[asked + 32 + lane] : -1;
      }
      uint4* to = slots + next * 256;
      next = next + 1 == kRing ? 0 : next + 1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int page = __shfl_sync(0xffffffffu, id, (asked + u * PPL + lane / LPP) & 31);
        const T* from = bounds + max(page, 0) * page_step;
#pragma unroll
        for (int i = 0; i < NC; ++i)
          cp_async16(smem_u32(to + (u * NC + i) * 32), from + i * D, page < 0 ? 0u : 16u);
      }
    }
    cp_async_commit();
    asked += STEP;
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) ask();
  // this lane's channels and its weights: smallest values first, then largest
  float w[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = 0.f;
  {
    const int j0 = c * 8 % D;
    const bool largest = c * 8 >= D;
    const T* q = static_cast<const T*>(P.q) + row * P.q_stride + (long long)hk * P.G * D + j0;
#pragma unroll 8
    for (int g = 0; g < P.G; ++g) {
      const uint4 r = *reinterpret_cast<const uint4*>(q + (long long)g * D);
      const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Pack<T>::unpack(u[e]);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const bool up = NC == 2 ? i == 1 : largest;
          // (comparisons that keep a NaN)
          w[i][2 * e] += up ? (f.x < 0.f ? 0.f : f.x) : (f.x > 0.f ? 0.f : f.x);
          w[i][2 * e + 1] += up ? (f.y < 0.f ? 0.f : f.y) : (f.y > 0.f ? 0.f : f.y);
        }
      }
    }
  }
  uint32_t top[NC][4];                                 // largest magnitudes seen, per channel
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) top[i][e] = 0u;
  for (int p0 = 0; p0 < mine; p0 += STEP) {
    ask();
    cp_async_wait<kRing - 1>();
    const uint4* from = slots + at * 256;
    at = at + 1 == kRing ? 0 : at + 1;
    float s[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) s[u] = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint64_t two = 0;                                // even and odd channels
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint4 x = from[(u * NC + i) * 32];
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Pack<T>::unpack(v[e]);
          two = fma2(pack2(f.x, f.y), pack2(w[i][2 * e], w[i][2 * e + 1]), two);
          top[i][e] = max_abs2<T>(top[i][e], v[e]);
        }
      }
      float a, b;
      unpack2(two, a, b);
      s[u] = a + b;
    }
    // sums over the lanes of a page: halves of the sums go to halves of the lanes
    constexpr int O1 = LPP / 2, O2 = LPP / 4, O3 = LPP / 8;
    float s4[4], s2[2], s1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (U == 8) s4[u] = (lane & O1 ? s[u + 4] : s[u]) + __shfl_xor_sync(0xffffffffu, lane & O1 ? s[u] : s[u + 4], O1);
      else s4[u] = s[u] + __shfl_xor_sync(0xffffffffu, s[u], O1);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
      s2[u] = (lane & O2 ? s4[u + 2] : s4[u]) + __shfl_xor_sync(0xffffffffu, lane & O2 ? s4[u] : s4[u + 2], O2);
    s1 = (lane & O3 ? s2[1] : s2[0]) + __shfl_xor_sync(0xffffffffu, lane & O3 ? s2[0] : s2[1], O3);
#pragma unroll
    for (int o = O3 / 2; o; o >>= 1) s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    const int u = (U == 8 && (lane & O1) ? 4 : 0) + (lane & O2 ? 2 : 0) + (lane & O3 ? 1 : 0);
    const int p = p0 + u * PPL + lane / LPP;
    const bool writes = (lane & (O3 - 1)) == 0 && (U == 8 || !(lane & O1));
    if (writes && p < mine) score[p] = s1;
  }
  // (pages outside the pool: few, and known by now; their sums, 0, are other lanes' stores)
  __syncwarp();
  for (int p = lane; p < mine; p += 32)
    if ((unsigned)table[p] >= P.num_pages) score[p] = -INFINITY;
  float mag = 0.f;
  bool some = false;                                   // a term that is not 0, though its fp32 product may be
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // (0 times an infinity is a NaN, as a term of that kind is)
      const float2 m = Pack<T>::unpack(top[i][e] & 0x7fff7fffu);
      some |= (w[i][2 * e] != 0.f && m.x != 0.f) || (w[i][2 * e + 1] != 0.f && m.y != 0.f);
      mag += fabsf(w[i][2 * e]) * m.x + fabsf(w[i][2 * e + 1]) * m.y;
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) mag += __shfl_xor_sync(0xffffffffu, mag, o);
  some = __any_sync(0xffffffffu, some || mag != mag);
  if (lane == 0)
    // (products of the smallest numbers are off by more than their part: each by up to 2^-150)
    P.off[((long long)row * P.Hk + hk) * P.chunks + chunk] =
        some ? mag * ((float)(4 * NC + 6 + P.G) * 0x1.04p-24f) + 0x1p-140f : 0.f;
}

// ------------------------------------------------------------------ the choice
// keys in the order of the values; every NaN above all numbers, or (fp32, where scores with
// one are computed again) anywhere. fp32 keys lie in [1, kForced): 0 is a page that does not
// compete, kForced one that is chosen whatever its score.
constexpr uint32_t kForced = 0xffffffffu;
POD_DEV uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);         // (-0 is 0)
  return min(max(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), 1u), kForced - 1);
}
POD_DEV float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
POD_DEV uint64_t key_of(double x) {
  if (x != x) return ~0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(x == 0. ? 0. : x);
  return b >> 63 ? ~b : b | 1ull << 63;
}

struct PickShared {
  alignas(16) int bins[kBins];
  unsigned long long lo[32], hi[32];
  int2 sums[32];
  float off[32];
  uint32_t near[kNear];            // keys, or pages
  double exact[kNear];
  bool in[kNear];
  int nears, bin, above, inside;
  uint32_t kth;
};

// Two counts of a warp (the same in its lanes): those of the warps before it, and of all.
POD_DEV int2 warp_sums_before(int x, int y, int2& all, PickShared& S) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) S.sums[warp] = make_int2(x, y);
  __syncthreads();
  const int2 w = lane < warps ? S.sums[lane] : make_int2(0, 0);
  all = make_int2(__reduce_add_sync(0xffffffffu, w.x), __reduce_add_sync(0xffffffffu, w.y));
  return make_int2(__reduce_add_sync(0xffffffffu, lane < warp ? w.x : 0), __reduce_add_sync(0xffffffffu, lane < warp ? w.y : 0));
}

// In which bin, counted from the top, is the need-th largest? `above` keys are larger
// than all bins. Leaves the bin, its keys and the number of keys above it in S. (The first
// warp's work, 32 bins a lane: two barriers less than a scan by the block.)
POD_DEV void find_bin(int need, int above, PickShared& S) {
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int4* fours = reinterpret_cast<const int4*>(S.bins) + lane;      // a lane's stand 32 fours apart
    int total[kBins / 128];
#pragma unroll
    for (int i = 0; i < kBins / 128; ++i) {
      const int4 n = fours[i * 32];
      total[i] = __reduce_add_sync(0xffffffffu, n.x + n.y + n.z + n.w);
    }
    int set = -1;                                    // of 128 bins, the one with the wanted key
#pragma unroll
    for (int i = kBins / 128 - 1; i >= 0; --i) {
      if (set >= 0) continue;
      if (above + total[i] >= need) set = i;
      else above += total[i];
    }
    const int4 n = fours[max(set, 0) * 32];
    const int own = n.x + n.y + n.z + n.w;
    int s = own;                                     // of the fours from this lane's up
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_down_sync(0xffffffffu, s, o);
      if (lane + o < 32) s += y;
    }
    int over = above + s - own;                      // keys above this four
    if (over < need && over + own >= need) {
      int bin = 3, inside = n.w;
      if (over + inside < need) { over += inside; inside = n.z; bin = 2; }
      if (over + inside < need) { over += inside; inside = n.y; bin = 1; }
      if (over + inside < need) { over += inside; inside = n.x; bin = 0; }
      S.bin = (max(set, 0) * 32 + lane) * 4 + bin;
      S.above = over;
      S.inside = inside;
    }
  }
  __syncthreads();
}

// The need-th largest (1 is the largest) of the keys that each() hands out, those that are
// at least `from`, of which there are at least `need`; `above` receives how many are larger.
// The range between the smallest and the largest is cut into bins, then the bin
// with the wanted key again, until a bin is one key.
template <typename F>
POD_DEV uint64_t kth_largest(F each, uint64_t from, int need, int& above, PickShared& S) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x;
  unsigned long long lo = ~0ull, hi = 0;
  each([&](int, uint64_t x) {
    if (x < from) return;
    lo = min(lo, (unsigned long long)x);
    hi = max(hi, (unsigned long long)x);
  });
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  __syncthreads();
  if (lane == 0) {
    S.lo[warp] = lo;
    S.hi[warp] = hi;
  }
  __syncthreads();
  for (int w = 0; w < T / 32; ++w) {
    lo = min(lo, S.lo[w]);
    hi = max(hi, S.hi[w]);
  }
  above = 0;
  while (lo < hi) {
    const int bits = 64 - __clzll((long long)(hi - lo)), shift = max(0, bits - kBinBits);
    for (int i = tid; i < kBins; i += T) S.bins[i] = 0;
    __syncthreads();
    each([&](int, uint64_t x) {
      if (x >= lo && x <= hi) atomicAdd(&S.bins[(x - lo) >> shift], 1);
    });
    find_bin(need, above, S);
    above = S.above;
    lo += (unsigned long long)S.bin << shift;
    hi = lo + min(hi - lo, (1ull << shift) - 1);
    __syncthreads();
  }
  return lo;
}

// A warp's share of a page's bounds, and with it the page's score in 64 bits.
template <typename T, int D>
struct PageBounds {
  T lo[D / 32], hi[D / 32];                            // (converted where they are used, not where they are asked for)
  bool there;
  POD_DEV void load(const PickParams& P, int row, int hk, int i) {
    const unsigned page = (unsigned)P.table[row * P.table_stride + i];
    there = page < P.num_pages;
    if (!there) return;
    const T* m = static_cast<const T*>(P.bounds) + ((long long)page * P.Hk + hk) * 2 * D + (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      lo[j] = m[j * 32];
      hi[j] = m[D + j * 32];
    }
  }
  POD_DEV double score(const double (*weight)[D]) const {
    if (!there) return -INFINITY;
    const int lane = threadIdx.x & 31;
    double s = 0., t = 0.;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      s = fma((double)(float)lo[j], weight[0][j * 32 + lane], s);
      t = fma((double)(float)hi[j], weight[1][j * 32 + lane], t);
    }
    s += t;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
};

// The pages [a, b) whose fp32 keys are in [least, sure], `close` of them, scored again in
// 64 bits; of them `ties` are chosen. Few, whose positions stand in S.near: which of
// them are chosen stands in S.in, and 0 is returned. Many: their scores are kept, the last
// chosen one's key is returned, and in `ties` how many of that score. (A block that comes
// here ends later than the others, so its loads are asked for together.)
template <typename T, int D>
__device__ __noinline__ uint64_t score_again(const PickParams& P, bool few, int row, int hk, int a, int b, uint32_t least,
                                             uint32_t sure, int close, int& ties, PickShared& S) {
  __shared__ double weight[2][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const long long item = (long long)row * P.Hk + hk;
  const T* q = static_cast<const T*>(P.q) + row * P.q_stride + (long long)hk * P.G * D;
  __syncthreads();                                     // (S.near is written)
  PageBounds<T, D> page;
  if (few && warp < close) page.load(P, row, hk, (int)S.near[warp]);
  for (int j = tid; j < D; j += threads) {
    // sums of the heads, exact as pairs of fp32 numbers (a sum and what its rounding left)
    float up = 0.f, up2 = 0.f, down = 0.f, down2 = 0.f;
    for (int g = 0; g < P.G; g += 8) {                 // (eight loads at a time)
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = g + i < P.G ? (float)q[(long long)(g + i) * D + j] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = x[i] < 0.f ? 0.f : x[i], d = x[i] > 0.f ? 0.f : x[i];
        const float su = up + u, sd = down + d, tu = su - up, td = sd - down;
        up2 += (up - (su - tu)) + (u - tu);
        down2 += (down - (sd - td)) + (d - td);
        up = su;
        down = sd;
      }
    }
    // (an infinity leaves a NaN as its remainder)
    weight[0][j] = fabsf(down) < INFINITY ? (double)down + (double)down2 : (double)down;
    weight[1][j] = fabsf(up) < INFINITY ? (double)up + (double)up2 : (double)up;
  }
  __syncthreads();
  if (few) {
    for (int c = warp; c < close; c += threads / 32) {
      if (c != warp) page.load(P, row, hk, (int)S.near[c]);
      const double s = page.score(weight);
      if (lane == 0) S.exact[c] = s;
    }
    __syncthreads();
    for (int c = tid; c < close; c += threads) {
      const uint64_t x = key_of(S.exact[c]);
      const int i = (int)S.near[c];
      int before = 0;
      for (int d = 0; d < close; ++d) {
        const uint64_t y = key_of(S.exact[d]);
        before += y > x || (y == x && (int)S.near[d] < i);
      }
      S.in[c] = before < ties;
    }
    __syncthreads();
    return 0;
  }
  const float* score = P.score + item * P.width;
  double* again = P.again + item * P.width;
  auto is_close = [&](int i) {
    const uint32_t x = key_of(score[i]);
    return x >= least && x <= sure;
  };
  for (int i = a + warp; i < b; i += threads / 32) {
    if (!is_close(i)) continue;
    page.load(P, row, hk, i);
    const double s = page.score(weight);
    if (lane == 0) again[i] = s;
  }
  __syncthreads();
  int larger;
  const uint64_t last = kth_largest(
      [&](auto f) {
        for (int i = a + tid; i < b; i += threads)
          if (is_close(i)) f(i, key_of(again[i]));
      },
      1ull, ties, larger, S);
  ties -= larger;
  return last;
}

// The need-th largest of the competing keys that each() hands out, all of them of finite
// numbers between those of lo and hi: bins over the range of the values, then the keys of
// the wanted bin by their ranks among themselves, where they are few. (S.bins and S.nears are
// zero.)
template <typename F>
POD_DEV uint32_t kth_score(F each, uint32_t lo, uint32_t hi, int need, PickShared& S) {
  const int tid = threadIdx.x, T = blockDim.x;
  if (lo == hi) return lo;
  // (monotone: a difference, a product and a truncation, each rounded in order)
  const float v0 = value_of(lo), scale = (kBins - 1) / fmaxf(value_of(hi) - v0, 1e-30f);
  auto bin_of = [&](uint32_t x) { return min(kBins - 1, (int)((value_of(x) - v0) * scale)); };
  each([&](int, uint32_t x) {
    if (x - 1 < kForced - 1) atomicAdd(&S.bins[bin_of(x)], 1);
  });
  find_bin(need, 0, S);
  const int bin = S.bin, above = S.above, count = S.inside;
  if (count <= kNear) {
    each([&](int, uint32_t x) {
      if (bin_of(x) == bin && x - 1 < kForced - 1) S.near[atomicAdd(&S.nears, 1)] = x;
    });
    __syncthreads();
    for (int i = tid; i < count; i += T) {
      const uint32_t x = S.near[i];
      int larger = above, same = 0;
      for (int j = 0; j < count; ++j) {
        larger += S.near[j] > x;
        same += S.near[j] == x;
      }
      if (larger < need && larger + same >= need) S.kth = x;
    }
    __syncthreads();
    return S.kth;
  }
  int larger;
  return (uint32_t)kth_largest(
      [&](auto f) {
        each([&](int i, uint32_t x) {
          if (bin_of(x) == bin && x - 1 < kForced - 1) f(i, (uint64_t)x);
        });
      },
      1ull, need - above, larger, S);
}

// A block makes one choice. HELD > 0: a lane's keys stay in registers (0: they are read in every
// pass, for more pages than a block can hold). A run of pages is a warp's, so that the chosen
// ones come out in order. Bound by latency: two trips to memory and seven barriers, some 4 us; a
// block with close calls takes 4 more, and among hundreds of blocks some have them.
template <typename T, int D, int HELD>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const __grid_constant__ PickParams P) {
  __shared__ PickShared S;
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
  const long long item = blockIdx.x;
  const int row = (int)(blockIdx.x / (unsigned)P.Hk), hk = (int)(blockIdx.x - (unsigned)row * P.Hk);
  const int n = pages_of(P, row);
  if (hk == 0 && tid == 0 && P.status && (P.lens[row] < 0 || P.lens[row] > P.width * P.ps))
    atomicOr(P.status, kStatusSlot);
  int32_t* out = P.pages + item * P.k;
  if (n <= P.k) {
    for (int i = tid; i < P.k; i += threads) out[i] = i < n ? i : -1;
    return;
  }
  // pages [a, b) compete for `need` places
  const int a = P.first, b = n - P.last, need = P.k - P.first - P.last;
  const float* score = P.score + item * P.width;
  const int run = HELD ? 32 * HELD : ((n + 31) / 32 + warps - 1) / warps * 32;
  const int i0 = min(n, warp * run), i1 = min(n, i0 + run);
  float off = 0.f;
  bool odd = false;                                    // (an infinite or NaN bound or score)
  auto key_at = [&](int i, float x) {
    if (i >= i1) return 0u;
    if (i < a || i >= b) return kForced;
    odd |= !(fabsf(x) < 0x1p120f);
    return key_of(x);
  };
  uint32_t held[HELD ? HELD : 1];
  const float first_off = P.off[item * P.chunks + min(tid, (n + P.per - 1) / P.per - 1)];
  if constexpr (HELD > 0) {
    float x[HELD];                                     // (all loads before the first use)
#pragma unroll
    for (int j = 0; j < HELD; ++j) x[j] = i0 + j * 32 + lane < i1 ? score[i0 + j * 32 + lane] : 0.f;
#pragma unroll
    for (int j = 0; j < HELD; ++j) held[j] = key_at(i0 + j * 32 + lane, x[j]);
  }
  const int offs = (n + P.per - 1) / P.per;
  float e = first_off;
  for (int i = tid; i < offs;) {
    odd |= !(e < 0x1p100f);
    off = fmaxf(off, e);
    if ((i += threads) < offs) e = P.off[item * P.chunks + i];
  }
  auto each = [&](auto f) {                            // (the lanes of a warp together)
    if constexpr (HELD > 0) {
#pragma unroll
      for (int j = 0; j < HELD; ++j) f(i0 + j * 32 + lane, held[j]);
    } else {
      for (int i = i0; i < i1; i += 32) f(i + lane, key_at(i + lane, i + lane < i1 ? score[i + lane] : 0.f));
    }
  };
  // the scores' range, and what they may be off by
  uint32_t lo = 0xffffffffu, hi = 0u;
  each([&](int, uint32_t x) {
    lo = min(lo, x - 1);                               // (0 is not the smallest, kForced not the largest)
    hi = max(hi, x + 1);
  });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  off = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(off)));
  if (lane == 0) {
    S.sums[warp] = make_int2((int)lo, (int)hi);
    S.off[warp] = off;
  }
  for (int i = tid; i < kBins; i += threads) S.bins[i] = 0;
  if (tid == 0) S.nears = 0;
  odd = __syncthreads_or(odd);
  {
    const int w = lane < warps ? lane : 0;
    const int2 range = S.sums[w];
    lo = __reduce_min_sync(0xffffffffu, (uint32_t)range.x) + 1;
    hi = __reduce_max_sync(0xffffffffu, (uint32_t)range.y) - 1;
    off = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(S.off[w])));
  }

  // keys above `sure` are in, those from `least` to it as far as places are left: the
  // lowest positions, or by their scores in 64 bits
  uint32_t sure = kForced - 1, least = need > 0 ? 1u : kForced;
  if (need > 0 && !odd) {
    const uint32_t kth = kth_score(each, lo, hi, need, S);
    const float v = value_of(kth);
    sure = off == 0.f ? kth : key_of(v + 2.5f * off);
    least = off == 0.f ? kth : key_of(v - 2.5f * off);
  }
  int full, close;
  auto count = [&]() {
    full = close = 0;
    each([&](int, uint32_t x) {
      full += x > sure;
      close += x >= least;
    });
    full = __reduce_add_sync(0xffffffffu, full);
    close = __reduce_add_sync(0xffffffffu, close) - full;
  };
  count();
  __syncthreads();                                     // (S.sums is read above)
  int2 all, at = warp_sums_before(full, close, all, S);
  int ties = P.k - all.x;                              // places for the close ones
  uint64_t last64 = 0;
  bool exactly = false;
  if (all.y > ties && (off != 0.f || odd)) {           // (without an error, equal scores are ties)
    const bool few = HELD > 0 && all.y <= kNear;
    if (few) {
      if (tid == 0) S.nears = 0;
      __syncthreads();
      each([&](int i, uint32_t x) {
        if (x >= least && x <= sure) S.near[atomicAdd(&S.nears, 1)] = (uint32_t)i;
      });
    }
    last64 = score_again<T, D>(P, few, row, hk, a, b, least, sure, all.y, ties, S);
    if (few) {                                         // the chosen ones are in, the others out
      if constexpr (HELD > 0) {
#pragma unroll
        for (int j = 0; j < HELD; ++j)
          if (held[j] >= least && held[j] <= sure) {
            held[j] = 0u;
            for (int c = 0; c < all.y; ++c)
              if (S.near[c] == (uint32_t)(i0 + j * 32 + lane)) held[j] = S.in[c] ? kForced : 0u;
          }
      }
      least = sure + 1;
      count();
      __syncthreads();
      at = warp_sums_before(full, close, all, S);
      ties = 0;
    } else {
      exactly = true;
    }
  }
  const unsigned below = (1u << lane) - 1;
  if (!exactly && all.y <= ties) {                     // all close ones are in
    int to = at.x + at.y;
    each([&](int i, uint32_t x) {
      const unsigned m = __ballot_sync(0xffffffffu, x >= least);
      const int slot = to + __popc(m & below);
      if (x >= least && slot < P.k) out[slot] = i;
      to += __popc(m);
    });
    return;
  }
  // some close ones are: by position, or by their scores in 64 bits and then by position
  const double* exact = P.again + item * P.width;
  auto grade = [&](int i, uint32_t x) {                // 2: in, 1: in as far as places are left
    if (x > sure) return 2;
    if (x < least) return 0;
    if (!exactly) return 1;
    const uint64_t y = key_of(exact[i]);
    return y > last64 ? 2 : y == last64 ? 1 : 0;
  };
  if (exactly) {
    full = close = 0;
    each([&](int i, uint32_t x) {
      const int g = grade(i, x);
      full += g == 2;
      close += g == 1;
    });
    full = __reduce_add_sync(0xffffffffu, full);
    close = __reduce_add_sync(0xffffffffu, close);
    __syncthreads();
    at = warp_sums_before(full, close, all, S);
    ties = P.k - all.x;
  }
  int tied_at = at.y, to = at.x + min(at.y, ties);
  each([&](int i, uint32_t x) {
    const int g = grade(i, x);
    const unsigned m1 = __ballot_sync(0xffffffffu, g == 1);
    const bool in = g == 2 || (g == 1 && tied_at + __popc(m1 & below) < ties);
    const unsigned m = __ballot_sync(0xffffffffu, in);
    const int slot = to + __popc(m & below);
    if (in && slot < P.k) out[slot] = i;
    to += __popc(m);
    tied_at += __popc(m1);
  });
}

// ------------------------------------------------------------------ host
pod_status fail(pod_status code, const std::string& msg) {
  pod_set_last_error(msg);
  return code;
}

template <typename T, int D>
cudaError_t launch_bounds(const BoundParams& P, int fmt, cudaStream_t st) {
  const long long blocks = (P.rows + P.span - 1) / P.span;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)blocks;
  return fmt == POD_KV_16BIT ? launch_beside(bounds_kernel<T, D, POD_KV_16BIT>, grid, kBoundThreads, 0, 1, st, P)
         : fmt == POD_KV_E4M3 ? launch_beside(bounds_kernel<T, D, POD_KV_E4M3>, grid, kBoundThreads, 0, 1, st, P)
                              : launch_beside(bounds_kernel<T, D, POD_KV_E4M3_BLOCK>, grid, kBoundThreads, 0, 1, st, P);
}
template <typename T>
cudaError_t launch_bounds_d(const BoundParams& P, int d, int fmt, cudaStream_t st) {
  return d == 64 ? launch_bounds<T, 64>(P, fmt, st)
         : d == 128 ? launch_bounds<T, 128>(P, fmt, st) : launch_bounds<T, 256>(P, fmt, st);
}

template <typename T, int D>
cudaError_t launch_pick(const PickParams& P, cudaStream_t st) {
  const long long warps = (long long)P.batch * P.chunks * P.Hk, per = kScoreThreads / 32;
  const long long blocks = (warps + per - 1) / per, items = (long long)P.batch * P.Hk;
  if (warps > 0x7fffffff) return cudaErrorInvalidConfiguration;      // (counted in 32 bits)
  if (P.width > P.k) {                                 // (else every page is chosen)
    const cudaError_t e = launch_beside(score_kernel<T, D>, (unsigned)blocks, kScoreThreads, kScoreShared, 1, st, P);
    if (e != cudaSuccess) return e;
  }
  // Threads that hold the longest row's keys, eight a lane, or sixteen. (Sixteen a lane and half the
  // threads for shorter rows too: 512 choices of some 1300 pages the same, 256 of them 7 us more.)
  const unsigned grid = (unsigned)items;
  if (P.width <= 256 * 8) return launch_beside(pick_kernel<T, D, 8>, grid, 256, 0, 1, st, P);
  if (P.width <= kPickThreads * 8) return launch_beside(pick_kernel<T, D, 8>, grid, kPickThreads, 0, 1, st, P);
  if (P.width <= kHeldPages) return launch_beside(pick_kernel<T, D, 16>, grid, kPickThreads, 0, 1, st, P);
  return launch_beside(pick_kernel<T, D, 0>, grid, kPickThreads, 0, 1, st, P);
}
template <typename T>
cudaError_t launch_pick_d(const PickParams& P, int d, cudaStream_t st) {
  return d == 64 ? launch_pick<T, 64>(P, st) : d == 128 ? launch_pick<T, 128>(P, st) : launch_pick<T, 256>(P, st);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

namespace pod {

// ------------------------------------------------------------------ checks that the calls share
pod_status check_decode_sizes(const pod_decode_args& a) {
  if (a.dtype != POD_F16 && a.dtype != POD_BF16) return fail(POD_ERR_UNSUPPORTED, "dtype must be fp16 or bf16");
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256)
    return fail(POD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  if (a.num_kv_heads < 1 || a.num_kv_heads > 4096) return fail(POD_ERR_INVALID_ARG, "num_kv_heads must be in [1, 4096]");
  if (a.page_size < 1 || a.num_pages < 1) return fail(POD_ERR_INVALID_ARG, "the page pool is empty");
  if (a.page_size > (1 << 30)) return fail(POD_ERR_INVALID_ARG, "page_size must be at most 2^30");
  // rows of head_dim elements are counted in 32 bits (a pool past this would be 2^38 bytes or more)
  if (a.num_pages > 0xfffffff0ll / (2 * (int64_t)a.page_size * a.num_kv_heads))
    return fail(POD_ERR_INVALID_ARG, "the page pool is too large");
  return POD_OK;
}

pod_status check_decode_cache(const pod_decode_args& a) {
  if (a.kv_format != POD_KV_16BIT && a.kv_format != POD_KV_E4M3 && a.kv_format != POD_KV_E4M3_BLOCK)
    return fail(POD_ERR_INVALID_ARG, "unknown cache format");
  if (a.kv_layout != 0 && a.kv_layout != 1) return fail(POD_ERR_INVALID_ARG, "kv_layout must be 0 (NHD) or 1 (HND)");
  if (!a.kv_cache || reinterpret_cast<uintptr_t>(a.kv_cache) % 32)
    return fail(POD_ERR_INVALID_ARG, "the cache must be a 32-byte aligned pointer");
  if (a.kv_format == POD_KV_E4M3_BLOCK && !a.kv_scales)
    return fail(POD_ERR_INVALID_ARG, "a block-scaled cache needs its scales");
  if (a.kv_format != POD_KV_E4M3_BLOCK && a.kv_scales)
    return fail(POD_ERR_INVALID_ARG, "scales given, but the cache format has none");
  if (a.kv_format == POD_KV_E4M3 && !(a.k_scale > 0.f && isfinite(a.k_scale)))
    return fail(POD_ERR_INVALID_ARG, "k_scale and v_scale must be finite and positive");
  return POD_OK;
}

pod_status check_decode_rows(const pod_decode_args& a) {
  if (a.batch < 0) return fail(POD_ERR_INVALID_ARG, "batch must not be negative");
  if (a.num_qo_heads < 1 || a.num_qo_heads > 65536 || a.num_qo_heads % a.num_kv_heads)
    return fail(POD_ERR_INVALID_ARG, "num_qo_heads must be a multiple of num_kv_heads, at most 65536");
  if (a.table_width < 1 || (int64_t)a.table_width * a.page_size > (1 << 30))
    return fail(POD_ERR_INVALID_ARG, "table_width must be positive, and table_width * page_size at most 2^30");
  if (a.batch > 1 && a.table_stride < a.table_width)
    return fail(POD_ERR_INVALID_ARG, "table_stride must hold table_width entries");
  if (!a.batch) return POD_OK;
  if (!a.block_table || !a.kv_lens) return fail(POD_ERR_INVALID_ARG, "block_table or kv_lens is NULL");
  if (!a.q || reinterpret_cast<uintptr_t>(a.q) % 16 || a.q_stride % 8 ||
      a.q_stride < (int64_t)a.num_qo_heads * a.head_dim)
    return fail(POD_ERR_INVALID_ARG,
                "q must be 16-byte aligned, its row stride a multiple of 8 elements that holds the row's heads");
  return POD_OK;
}

}  // namespace pod

extern "C" {

pod_status pod_page_bounds(const pod_decode_args* a, void* stream) {
  pod_set_last_error("");
  if (!a) return fail(POD_ERR_INVALID_ARG, "args is NULL");
  pod_status st = check_decode_sizes(*a);
  if (st == POD_OK) st = check_decode_cache(*a);
  if (st != POD_OK) return st;
  if (a->rows < 0 || a->rows > 0x7fffffff) return fail(POD_ERR_INVALID_ARG, "rows must be in [0, 2^31)");
  if (!a->bounds || reinterpret_cast<uintptr_t>(a->bounds) % 16)
    return fail(POD_ERR_INVALID_ARG, "bounds must be a 16-byte aligned pointer");
  if (!a->rows) return POD_OK;
  if (!a->slots) return fail(POD_ERR_INVALID_ARG, "slots is NULL");
  BoundParams P = {};
  P.cache = static_cast<const uint8_t*>(a->kv_cache);
  P.scales = a->kv_scales;
  P.bounds = a->bounds;
  P.slots = a->slots;
  P.status = a->status;
  P.rows = a->rows;
  P.num_slots = a->num_pages * a->page_size;
  P.ps = a->page_size;
  P.Hk = a->num_kv_heads;
  P.hnd = a->kv_layout;
  P.k_scale = a->k_scale;
  // few rows a block where there are few, so that every SM gets some
  const int64_t span = (a->rows + 152 * 4 - 1) / (152 * 4);
  P.span = (int)(span < kBoundRows ? span : kBoundRows);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = a->dtype == POD_BF16 ? launch_bounds_d<__nv_bfloat16>(P, a->head_dim, a->kv_format, s)
                                             : launch_bounds_d<__half>(P, a->head_dim, a->kv_format, s);
  if (e != cudaSuccess) return fail(POD_ERR_CUDA, std::string("page bounds launch: ") + cudaGetErrorString(e));
  return POD_OK;
}

size_t pod_select_pages_workspace_size(int32_t batch, int32_t num_kv_heads, int32_t table_width) {
  if (batch < 0 || num_kv_heads < 1 || table_width < 1) return 0;
  const size_t items = (size_t)batch * num_kv_heads;
  const size_t chunks = ((size_t)table_width + kLeastPages - 1) / kLeastPages;
  return round256(items * table_width * sizeof(double)) + round256(items * table_width * sizeof(float)) +
         round256(items * chunks * sizeof(float));
}

pod_status pod_select_pages(const pod_decode_args* a, void* stream) {
  pod_set_last_error("");
  if (!a) return fail(POD_ERR_INVALID_ARG, "args is NULL");
  pod_status st = check_decode_sizes(*a);
  if (st == POD_OK) st = check_decode_rows(*a);
  if (st != POD_OK) return st;
  if (a->num_selected < 1 || a->keep_first < 0 || a->keep_last < 0 ||
      (int64_t)a->keep_first + a->keep_last > a->num_selected)
    return fail(POD_ERR_INVALID_ARG, "num_selected must be positive, keep_first and keep_last at most that together");
  if (!a->batch) return POD_OK;
  if (!a->bounds || reinterpret_cast<uintptr_t>(a->bounds) % 16)
    return fail(POD_ERR_INVALID_ARG, "bounds must be a 16-byte aligned pointer");
  if (!a->pages) return fail(POD_ERR_INVALID_ARG, "pages is NULL");
  if (!a->workspace || reinterpret_cast<uintptr_t>(a->workspace) % 256 ||
      a->workspace_bytes < pod_select_pages_workspace_size(a->batch, a->num_kv_heads, a->table_width))
    return fail(POD_ERR_WORKSPACE, "the workspace is missing, too small or not 256-byte aligned");
  PickParams P = {};
  P.q = a->q;
  P.bounds = a->bounds;
  P.table = a->block_table;
  P.lens = a->kv_lens;
  P.pages = a->pages;
  P.status = a->status;
  P.q_stride = a->q_stride;
  P.table_stride = a->table_stride;
  P.num_pages = (unsigned)a->num_pages;
  P.batch = a->batch;
  P.Hk = a->num_kv_heads;
  P.G = a->num_qo_heads / a->num_kv_heads;
  P.width = a->table_width;
  // Pages of a warp: few where the SMs would not all be busy otherwise, more where that makes
  // the weights less often (16 / 64 a warp: 2 rows of 8 heads and some 250 pages 9.2 / 11.3 us, 64
  // rows of 1300 pages 93 / 69).
  const int64_t pages = (int64_t)a->batch * a->num_kv_heads * a->table_width;
  P.per = pages <= 152 * 16 * 32 ? kLeastPages : 64;
  P.chunks = (a->table_width + P.per - 1) / P.per;
  P.ps = a->page_size;
  P.k = a->num_selected;
  P.first = a->keep_first;
  P.last = a->keep_last;
  const size_t entries = (size_t)P.batch * P.Hk * P.width;
  char* w = static_cast<char*>(a->workspace);
  P.again = reinterpret_cast<double*>(w);
  w += round256(entries * sizeof(double));
  P.score = reinterpret_cast<float*>(w);
  w += round256(entries * sizeof(float));
  P.off = reinterpret_cast<float*>(w);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = a->dtype == POD_BF16 ? launch_pick_d<__nv_bfloat16>(P, a->head_dim, s)
                                             : launch_pick_d<__half>(P, a->head_dim, s);
  if (e != cudaSuccess) return fail(POD_ERR_CUDA, std::string("page selection launch: ") + cudaGetErrorString(e));
  return POD_OK;
}

}  // extern "C"
