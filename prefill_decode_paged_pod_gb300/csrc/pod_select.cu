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
// score is off by at most E = (24 + G) 2^-24 times the sum of its terms' magnitudes (8
// or 16 fused steps a lane, five additions across lanes, G - 1 in a weight), of which
// a bound is kept per 32 pages. Pages further than 2 E from the last place are decided;
// the others, where they are more than the places left, are scored again in 64
// bits (of which this GPU does two a clock and SM).
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>

#include <string>

#include "../../include/pod.h"
#include "pod_decode.h"
#include "pod_device.cuh"

void pod_set_last_error(const std::string& msg);

using namespace pod;

namespace {

constexpr int kBoundThreads = 256, kBoundRows = 128;
constexpr int kScoreThreads = 256, kScorePages = 32;   // pages of a warp
constexpr int kPickThreads = 256, kBins = 1024;
constexpr int kKeysInShared = 8192;                    // pages whose scores a block holds

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static constexpr uint32_t kInf = 0x7f807f80u;
  static constexpr float kMax = 3.3895313892515355e38f;
  static POD_DEV __nv_bfloat16 down(float x) { return __float2bfloat16_rd(x); }
  static POD_DEV __nv_bfloat16 up(float x) { return __float2bfloat16_ru(x); }
};
template <>
struct Pair<__half> {
  using type = __half2;
  static constexpr uint32_t kInf = 0x7c007c00u;
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

// A block takes `span` rows of the write; a row whose page differs from that of
// the row before owns the page, and a warp brings in the keys of one (page, head): eight
// 16-byte loads a lane in flight, 32 / LPR keys each. Read once: bound by memory.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kBoundThreads) bounds_kernel(const __grid_constant__ BoundParams P) {
  constexpr int E = FMT == POD_KV_16BIT ? 2 : 1, LPR = D * E / 16, KPL = 32 / LPR, U = 8;
  constexpr int N = 16 / E;                            // elements of a lane's chunk
  using M = typename std::conditional<FMT == POD_KV_16BIT, T, __half>::type;
  __shared__ long long own[kBoundRows];
  __shared__ int owners;
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) owners = 0;
  __syncthreads();
  const long long row0 = (long long)blockIdx.x * P.span;
  if (tid < P.span && row0 + tid < P.rows) {
    const long long r = row0 + tid, s = P.slots[r];
    if (s >= P.num_slots && P.status) atomicOr(P.status, kStatusSlot);
    if (s >= 0 && s < P.num_slots) {
      const long long b = r ? P.slots[r - 1] : -1;
      if (b < 0 || b / P.ps != s / P.ps) own[atomicAdd(&owners, 1)] = r;
    }
  }
  __syncthreads();
  const int tasks = owners * P.Hk;
  for (int i = warp; i < tasks; i += kBoundThreads / 32) {
    const long long r = own[i / P.Hk];
    const int h = i - i / P.Hk * P.Hk;
    const long long page = P.slots[r] / P.ps;
    // the page's rows of the write stand behind r
    int valid = 0;
    for (long long a = r; a < P.rows; a += 32) {
      const long long s = a + lane < P.rows ? P.slots[a + lane] : -1;
      const unsigned same = __ballot_sync(0xffffffffu, s >= 0 && s / P.ps == page);
      const int run = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
      valid = max(valid, __reduce_max_sync(0xffffffffu, lane < run ? (int)(s - page * P.ps) + 1 : 0));
      if (run < 32) break;
    }
    const long long row = (page * 2 * P.Hk * P.ps + (P.hnd ? (long long)h * P.ps : h));   // of key 0, in rows of D
    const int step = P.hnd ? 1 : P.Hk;
    const int part = lane % LPR, sub = lane / LPR;
    uint32_t lo2[4], hi2[4];                           // packed extremes (not with block scales)
    float lo[N], hi[N];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo2[e] = Pair<M>::kInf;
      hi2[e] = Pair<M>::kInf | 0x80008000u;
    }
    uint32_t lo3[4], hi3[4];                           // (the upper half of a chunk of 16 codes)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo3[e] = lo2[e];
      hi3[e] = hi2[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      lo[e] = INFINITY;
      hi[e] = -INFINITY;
    }
    for (int k0 = 0; k0 < valid; k0 += KPL * U) {
      uint4 x[U];
      int eb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * KPL + sub;
        if (k < valid) {
          const long long at = row + (long long)k * step;
          x[u] = __ldcs(reinterpret_cast<const uint4*>(P.cache + at * (D * E)) + part);
          if (FMT == POD_KV_E4M3_BLOCK) eb[u] = P.scales[at];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + u * KPL + sub >= valid) continue;
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (FMT == POD_KV_16BIT) {
            lo2[e] = min2<M>(lo2[e], w[e]);
            hi2[e] = max2<M>(hi2[e], w[e]);
          } else {
            const uint32_t a = e4m3x2_to<__half>((uint16_t)w[e]), b = e4m3x2_to<__half>((uint16_t)(w[e] >> 16));
            if constexpr (FMT == POD_KV_E4M3) {
              lo2[e] = min2<M>(lo2[e], a);
              hi2[e] = max2<M>(hi2[e], a);
              lo3[e] = min2<M>(lo3[e], b);
              hi3[e] = max2<M>(hi3[e], b);
            } else {
              const float s = eb[u] ? __uint_as_float((uint32_t)eb[u] << 23) : 5.877471754111438e-39f;
              const float2 fa = Pack<__half>::unpack(a), fb = Pack<__half>::unpack(b);
              const float y[4] = {fa.x * s, fa.y * s, fb.x * s, fb.y * s};
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                lo[4 * e + c] = fminf(lo[4 * e + c], y[c]);
                hi[4 * e + c] = fmaxf(hi[4 * e + c], y[c]);
              }
            }
          }
        }
      }
    }
    // packed extremes as values
    if constexpr (FMT != POD_KV_E4M3_BLOCK) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo2[e] = min2<M>(lo2[e], __shfl_xor_sync(0xffffffffu, lo2[e], o));
          hi2[e] = max2<M>(hi2[e], __shfl_xor_sync(0xffffffffu, hi2[e], o));
          if constexpr (FMT == POD_KV_E4M3) {
            lo3[e] = min2<M>(lo3[e], __shfl_xor_sync(0xffffffffu, lo3[e], o));
            hi3[e] = max2<M>(hi3[e], __shfl_xor_sync(0xffffffffu, hi3[e], o));
          }
        }
      const float s = FMT == POD_KV_E4M3 ? P.k_scale : 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = Pack<M>::unpack(lo2[e]), b = Pack<M>::unpack(hi2[e]);
        if constexpr (FMT == POD_KV_16BIT) {
          lo[2 * e] = a.x; lo[2 * e + 1] = a.y;
          hi[2 * e] = b.x; hi[2 * e + 1] = b.y;
        } else {
          const float2 c = Pack<M>::unpack(lo3[e]), d = Pack<M>::unpack(hi3[e]);
          lo[4 * e] = a.x * s; lo[4 * e + 1] = a.y * s; lo[4 * e + 2] = c.x * s; lo[4 * e + 3] = c.y * s;
          hi[4 * e] = b.x * s; hi[4 * e + 1] = b.y * s; hi[4 * e + 2] = d.x * s; hi[4 * e + 3] = d.y * s;
        }
      }
    } else {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
          hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
        }
    }
    T* dst = static_cast<T*>(P.bounds) + (page * P.Hk + h) * 2 * D + part * N;
    auto put = [&](T* to, const float* v, bool upper) {
      T y[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float c = fminf(fmaxf(v[e], -Pair<T>::kMax), Pair<T>::kMax);
        y[e] = upper ? Pair<T>::up(c) : Pair<T>::down(c);
      }
#pragma unroll
      for (int e = 0; e < N; e += 8) {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          w[c] = (uint32_t)*reinterpret_cast<uint16_t*>(&y[e + 2 * c]) |
                 (uint32_t)*reinterpret_cast<uint16_t*>(&y[e + 2 * c + 1]) << 16;
        *reinterpret_cast<uint4*>(to + e) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    };
    if (sub == 0) put(dst, lo, false);
    if (sub == KPL - 1) put(dst + D, hi, true);
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
  int batch, Hk, G, width, chunks, ps, k, first, last;
};

POD_DEV int pages_of(const PickParams& P, int row) {
  const int most = P.width * P.ps, len = P.lens[row];
  return (min(max(len, 0), most) + P.ps - 1) / P.ps;
}

// A warp scores 32 pages for one head: a page's bounds are 4 D bytes, 16 a lane, eight
// loads in flight; the eight sums cross the lanes together (nine shuffles). Bound by memory.
template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const __grid_constant__ PickParams P) {
  constexpr int LPP = D == 64 ? 16 : 32, NC = D == 256 ? 2 : 1, PPL = 32 / LPP, U = 8;
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long task = (long long)blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
  const int hk = (int)(task % P.Hk);
  const long long rest = task / P.Hk;
  const int chunk = (int)(rest % P.chunks);
  const int row = (int)(rest / P.chunks);
  if (row >= P.batch) return;
  const int n = pages_of(P, row), page0 = chunk * kScorePages;
  if (page0 >= n || n <= P.k) return;                  // (then all are chosen)
  int id = -1;
  if (page0 + lane < n) {
    id = P.table[row * P.table_stride + page0 + lane];
    if ((unsigned)id >= P.num_pages) {
      id = -1;
      if (P.status) atomicOr(P.status, kStatusSlot);
    }
  }
  // this lane's channels and its weights: smallest values first, then largest
  const int c = lane % LPP;
  float w[NC][8], mag = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = 0.f;
  {
    const int j0 = c * 8 % D;
    const bool largest = c * 8 >= D;
    const T* q = static_cast<const T*>(P.q) + row * P.q_stride + (long long)hk * P.G * D + j0;
#pragma unroll 4
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
  const T* bounds = static_cast<const T*>(P.bounds) + (long long)hk * 2 * D + c * 8;
  float* score = P.score + ((long long)row * P.Hk + hk) * P.width;
  uint32_t top[NC];                                    // largest magnitudes seen
#pragma unroll
  for (int i = 0; i < NC; ++i) top[i] = 0u;
  for (int p0 = 0; p0 < kScorePages && page0 + p0 < n; p0 += U * PPL) {
    uint4 x[U][NC];
    int at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = __shfl_sync(0xffffffffu, id, p0 + u * PPL + lane / LPP);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        x[u][i] = make_uint4(0, 0, 0, 0);
        if (at[u] >= 0)
          x[u][i] = __ldcs(reinterpret_cast<const uint4*>(bounds + (long long)at[u] * P.Hk * 2 * D + i * D));
      }
    }
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint32_t v[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Pack<T>::unpack(v[e]);
          s[u] = fmaf(f.x, w[i][2 * e], s[u]);
          s[u] = fmaf(f.y, w[i][2 * e + 1], s[u]);
          top[i] = max2<T>(top[i], v[e] & 0x7fff7fffu);
        }
      }
    }
    // sums over the lanes of a page: halves of the eight go to halves of the lanes
    constexpr int O1 = LPP / 2, O2 = LPP / 4, O3 = LPP / 8;
    float s4[4], s2[2], s1;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      s4[u] = (lane & O1 ? s[u + 4] : s[u]) + __shfl_xor_sync(0xffffffffu, lane & O1 ? s[u] : s[u + 4], O1);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      s2[u] = (lane & O2 ? s4[u + 2] : s4[u]) + __shfl_xor_sync(0xffffffffu, lane & O2 ? s4[u] : s4[u + 2], O2);
    s1 = (lane & O3 ? s2[1] : s2[0]) + __shfl_xor_sync(0xffffffffu, lane & O3 ? s2[0] : s2[1], O3);
#pragma unroll
    for (int o = O3 / 2; o; o >>= 1) s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    const int u = (lane & O1 ? 4 : 0) + (lane & O2 ? 2 : 0) + (lane & O3 ? 1 : 0);
    const int p = p0 + u * PPL + lane / LPP;
    const int mine = __shfl_sync(0xffffffffu, id, p);
    if ((lane & (O3 - 1)) == 0 && page0 + p < n) score[page0 + p] = mine < 0 ? -INFINITY : s1;
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const float2 m = Pack<T>::unpack(top[i]);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += fabsf(w[i][e]);
    // (0 times an infinity is a NaN, as a term of that kind is)
    mag += sum * fmaxf(m.x, m.y);
  }
#pragma unroll
  for (int o = LPP / 2; o; o >>= 1) mag += __shfl_xor_sync(0xffffffffu, mag, o);
  if (PPL == 2) mag = mag + __shfl_xor_sync(0xffffffffu, mag, 16);
  if (lane == 0)
    // (products of the smallest numbers are off by more than their part)
    P.off[((long long)row * P.Hk + hk) * P.chunks + chunk] =
        mag == 0.f ? 0.f : mag * ((24.f + P.G) * 0x1.04p-24f) + 0x1p-140f;
}

// ------------------------------------------------------------------ the choice
// keys in the order of the values; every NaN above all numbers
POD_DEV uint32_t key_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
POD_DEV float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
POD_DEV uint64_t key_of(double x) {
  if (x != x) return ~0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(x == 0. ? 0. : x);
  return b >> 63 ? ~b : b | 1ull << 63;
}

struct PickShared {
  int bins[kBins];
  int sums[kPickThreads / 32 + 1];
  unsigned long long lo[kPickThreads / 32], hi[kPickThreads / 32];
  int bin, above;
};

POD_DEV int block_sum_before(int x, int& all, PickShared& S) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) S.sums[warp] = s;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kPickThreads / 32; ++w) {
    before += w < warp ? S.sums[w] : 0;
    all += S.sums[w];
  }
  return before + s - x;
}

// The need-th largest (1 is the largest) of the keys key(i), i in [a, b), that are in
// [lo, hi], of which there are at least `need`; `above` receives how many are larger.
// The range between the smallest and the largest is cut into 1024 bins, then the bin
// with the wanted key again, until a bin is one key.
template <typename K, typename F>
POD_DEV K kth_largest(F key, int a, int b, K from, K to, int need, int& above, PickShared& S) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned long long lo = ~0ull, hi = 0;
  for (int i = a + tid; i < b; i += kPickThreads) {
    const K x = key(i);
    if (x < from || x > to) continue;
    lo = min(lo, (unsigned long long)x);
    hi = max(hi, (unsigned long long)x);
  }
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
#pragma unroll
  for (int w = 0; w < kPickThreads / 32; ++w) {
    lo = min(lo, S.lo[w]);
    hi = max(hi, S.hi[w]);
  }
  above = 0;
  while (lo < hi) {
    const int bits = 64 - __clzll((long long)(hi - lo)), shift = max(0, bits - 10);
    for (int i = tid; i < kBins; i += kPickThreads) S.bins[i] = 0;
    __syncthreads();
    for (int i = a + tid; i < b; i += kPickThreads) {
      const unsigned long long x = key(i);
      if (x >= lo && x <= hi) atomicAdd(&S.bins[(x - lo) >> shift], 1);
    }
    __syncthreads();
    // from the top: a thread's four bins, the sum of those above them
    constexpr int PER = kBins / kPickThreads;
    int mine[PER], sum = 0, all;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      mine[i] = S.bins[kBins - 1 - (tid * PER + i)];
      sum += mine[i];
    }
    int before = above + block_sum_before(sum, all, S);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (before < need && before + mine[i] >= need) {
        S.bin = kBins - 1 - (tid * PER + i);
        S.above = before;
      }
      before += mine[i];
    }
    __syncthreads();
    above = S.above;
    lo += (unsigned long long)S.bin << shift;
    hi = lo + min(hi - lo, (1ull << shift) - 1);
    __syncthreads();
  }
  return (K)lo;
}

template <typename T, int D>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const __grid_constant__ PickParams P) {
  extern __shared__ uint32_t sh_keys[];
  __shared__ PickShared S;
  __shared__ double sh_w[2][D];
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long item = blockIdx.x;
  const int row = (int)(item / P.Hk), hk = (int)(item - (long long)row * P.Hk);
  const int n = pages_of(P, row);
  if (hk == 0 && tid == 0 && P.status && (P.lens[row] < 0 || P.lens[row] > P.width * P.ps))
    atomicOr(P.status, kStatusSlot);
  int32_t* out = P.pages + item * P.k;
  if (n <= P.k) {
    for (int i = tid; i < P.k; i += kPickThreads) out[i] = i < n ? i : -1;
    return;
  }
  // pages [a, b) compete for `need` places
  const int a = P.first, b = n - P.last, need = P.k - P.first - P.last;
  const float* score = P.score + item * P.width;
  double* again = P.again + item * P.width;
  float off = 0.f;
  bool odd = false;                                    // (an infinite or NaN bound)
  for (int i = tid; i < (n + kScorePages - 1) / kScorePages; i += kPickThreads) {
    const float e = P.off[item * P.chunks + i];
    odd |= !(e < 0x1p100f);
    off = fmaxf(off, e);
  }
  const bool held = n <= kKeysInShared;
  if (held)
    for (int i = tid; i < n; i += kPickThreads) sh_keys[i] = key_of(score[i]);
#pragma unroll
  for (int o = 16; o; o >>= 1) off = fmaxf(off, __shfl_xor_sync(0xffffffffu, off, o));
  if (lane == 0) S.sums[warp] = __float_as_int(off);
  odd = __syncthreads_or(odd);
#pragma unroll
  for (int w = 0; w < kPickThreads / 32; ++w) off = fmaxf(off, __int_as_float(S.sums[w]));
  auto key = [&](int i) { return held ? sh_keys[i] : key_of(score[i]); };

  // keys above `sure` are in, those from `least` to it compete on, by their score in 64
  // bits where `exactly`
  uint32_t sure = 0xffffffffu, least = 0xffffffffu;
  uint64_t last64 = 0;
  int ties = 0;
  bool exactly = false;
  if (need > 0) {
    int above;
    const uint32_t kth = kth_largest<uint32_t>(key, a, b, 0u, 0xffffffffu, need, above, S);
    const float v = value_of(kth);
    sure = least = kth;
    if (off != 0.f || odd) {
      if (odd || !(fabsf(v) < 0x1p120f)) {
        sure = 0xffffffffu;
        least = 0u;
      } else {
        sure = key_of(v + 2.5f * off);
        least = key_of(v - 2.5f * off);
      }
    }
    int in = 0, close = 0;
    for (int i = a + tid; i < b; i += kPickThreads) {
      const uint32_t x = key(i);
      in += x > sure;
      close += x >= least && x <= sure;
    }
    int all;
    block_sum_before(in | close << 16, all, S);
    // (counts past 16 bits: summed apart)
    if (b - a >= 32768) {
      block_sum_before(in, in, S);
      block_sum_before(close, close, S);
    } else {
      in = all & 0xffff;
      close = all >> 16;
    }
    ties = need - in;                                  // places for the close ones
    if (close > ties && (off != 0.f || odd)) {
      exactly = true;
      // the weights, then a warp a page
      const T* q = static_cast<const T*>(P.q) + row * P.q_stride + (long long)hk * P.G * D;
      for (int j = tid; j < D; j += kPickThreads) {
        double up = 0., down = 0.;
        for (int g = 0; g < P.G; ++g) {
          const double x = (double)(float)q[(long long)g * D + j];
          up += x < 0. ? 0. : x;
          down += x > 0. ? 0. : x;
        }
        sh_w[0][j] = down;
        sh_w[1][j] = up;
      }
      __syncthreads();
      for (int i = a + warp; i < b; i += kPickThreads / 32) {
        const uint32_t x = key(i);
        if (x < least || x > sure) continue;
        const unsigned page = (unsigned)P.table[row * P.table_stride + i];
        double s = 0.;
        if (page < P.num_pages) {
          const T* m = static_cast<const T*>(P.bounds) + ((long long)page * P.Hk + hk) * 2 * D;
#pragma unroll 4
          for (int j = lane; j < D; j += 32)
            s += (double)(float)m[j] * sh_w[0][j] + (double)(float)m[D + j] * sh_w[1][j];
#pragma unroll
          for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        } else {
          s = -INFINITY;
        }
        if (lane == 0) again[i] = s;
      }
      __syncthreads();
      auto key64 = [&](int i) {
        const uint32_t x = key(i);
        return x >= least && x <= sure ? key_of(again[i]) : 0ull;
      };
      int larger;
      last64 = kth_largest<uint64_t>(key64, a, b, 1ull, ~0ull, ties, larger, S);
      ties -= larger;
    }                                                  // (without an error, equal scores are ties)
  }
  // ---- in order: a run of pages a thread
  const int per = (n + kPickThreads - 1) / kPickThreads, i0 = min(n, tid * per), i1 = min(n, i0 + per);
  auto grade = [&](int i) {                            // 2: in, 1: in as far as places are left
    if (i < a || i >= b) return 2;
    if (need == 0) return 0;
    const uint32_t x = key(i);
    if (x > sure) return 2;
    if (x < least) return 0;
    if (!exactly) return 1;
    const uint64_t y = key_of(again[i]);
    return y > last64 ? 2 : y == last64 ? 1 : 0;
  };
  int full = 0, tied = 0, all;
  for (int i = i0; i < i1; ++i) {
    const int g = grade(i);
    full += g == 2;
    tied += g == 1;
  }
  int tied_at = block_sum_before(tied, all, S);
  const int taken = min(max(ties - tied_at, 0), tied);
  int to = block_sum_before(full + taken, all, S);
  for (int i = i0; i < i1; ++i) {
    const int g = grade(i);
    if ((g == 2 || (g == 1 && tied_at < ties)) && to < P.k) out[to++] = i;
    tied_at += g == 1;
  }
}

// ------------------------------------------------------------------ host
pod_status fail(pod_status code, const std::string& msg) {
  pod_set_last_error(msg);
  return code;
}

template <typename... A, typename... B>
cudaError_t launch_beside(void (*kernel)(A...), unsigned grid, unsigned threads, unsigned shared, cudaStream_t st,
                          const B&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int D>
cudaError_t launch_bounds(const BoundParams& P, int fmt, cudaStream_t st) {
  const long long blocks = (P.rows + P.span - 1) / P.span;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)blocks;
  return fmt == POD_KV_16BIT ? launch_beside(bounds_kernel<T, D, POD_KV_16BIT>, grid, kBoundThreads, 0, st, P)
         : fmt == POD_KV_E4M3 ? launch_beside(bounds_kernel<T, D, POD_KV_E4M3>, grid, kBoundThreads, 0, st, P)
                              : launch_beside(bounds_kernel<T, D, POD_KV_E4M3_BLOCK>, grid, kBoundThreads, 0, st, P);
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
  if (blocks > 0x7fffffff || items > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (P.width > P.k) {                                 // (else every page is chosen)
    const cudaError_t e = launch_beside(score_kernel<T, D>, (unsigned)blocks, kScoreThreads, 0, st, P);
    if (e != cudaSuccess) return e;
  }
  const unsigned shared = 4u * (unsigned)(P.width < kKeysInShared ? P.width : kKeysInShared);
  return launch_beside(pick_kernel<T, D>, (unsigned)items, kPickThreads, shared, st, P);
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
  // rows of head_dim elements are counted in 32 bits (a pool past this would be 2^38 bytes or more)
  if (a.num_pages > 0xfffffff0ll / (2 * (int64_t)a.page_size * a.num_kv_heads))
    return fail(POD_ERR_INVALID_ARG, "the page pool is too large");
  return POD_OK;
}

pod_status check_decode_cache(const pod_decode_args& a) {
  if (a.kv_format != POD_KV_16BIT && a.kv_format != POD_KV_E4M3 && a.kv_format != POD_KV_E4M3_BLOCK)
    return fail(POD_ERR_INVALID_ARG, "unknown cache format");
  if (a.kv_layout != 0 && a.kv_layout != 1) return fail(POD_ERR_INVALID_ARG, "kv_layout must be 0 (NHD) or 1 (HND)");
  if (!a.kv_cache || reinterpret_cast<uintptr_t>(a.kv_cache) % 16)
    return fail(POD_ERR_INVALID_ARG, "the cache must be a 16-byte aligned pointer");
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
  const size_t chunks = ((size_t)table_width + kScorePages - 1) / kScorePages;
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
  P.chunks = (a->table_width + kScorePages - 1) / kScorePages;
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
