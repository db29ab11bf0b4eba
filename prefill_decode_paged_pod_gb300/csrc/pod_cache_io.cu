// pod_cache_io.cu — the operators around the paged cache: per-head RMS norm of
// queries and keys with the position rotation, the write of keys and values
// into the cache (16-bit, E4M3 with per-tensor scales, E4M3 with a power-of-two
// scale per token and KV head), and the read of cache rows back as 16-bit
// values.
//
// Mathematics. A head row x of d elements becomes
//   y = x * (mean(x^2) + eps)^(-1/2) * w, then the pairs (j, j + R/2) or
//   (2j, 2j + 1), j < R/2, turn by the angle pos / rope_scale * theta^(-2j/R).
// The angle is kept in turns as a 64-bit fixed-point fraction: the per-turn
// frequency F = theta^(-2j/R) / (2 pi rope_scale) * 2^64 is an integer, and
// pos * F modulo 2^64 is the exact fraction of a turn for that F (whole turns
// drop out by themselves, for negative positions too). Its error is pos * 2^-56
// of a turn, so far positions cost no 64-bit floating point, of which this GPU
// has little. Everything else runs in fp32 and is rounded once, at the store.
//
// A power-of-two block scale 2^e is the smallest with amax <= 448 * 2^e. E4M3
// is a floating-point format, so a power of two costs no significant bit
// against the exact quotient amax / 448 (at most one of its 17 binades), the
// product with it is exact, and it is stored in one byte (exponent + 127).
//
// Work split. A head row is read by d/8 lanes with one 16-byte load each; the
// lane groups of a block walk the (token, head) tasks of a few tokens, four
// loads in flight a thread. The rotation's partner elements come by shuffle,
// cos and sin from a table that the block computes once per token. All of it
// is bound by HBM for long calls and by the launch for short ones.
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <string>

#include "../../include/pod.h"
#include "pod_device.cuh"

void pod_set_last_error(const std::string& msg);

using namespace pod;

namespace {

constexpr int kIoThreads = 256;
constexpr int kMaxTok = 8;        // tokens per block
constexpr int kUnroll = 4;        // head rows in flight per lane group
constexpr int kStatusSlot = 4;    // status bit: a slot outside the pool

enum { FMT_NONE = -1, FMT_16 = POD_KV_16BIT, FMT_SCALED = POD_KV_E4M3, FMT_BLOCK = POD_KV_E4M3_BLOCK };

struct IoParams {
  const void *q, *k, *v;
  void *q_out, *k_out;
  const void *qw, *kw;
  const int32_t* pos;
  const int64_t* slots;
  void* cache;
  uint8_t* scales;
  int32_t* status;
  long long q_stride, k_stride, v_stride, qo_stride, ko_stride;   // elements per token
  long long num_slots;
  int rows, H, Hk, ps, hnd, R, interleaved;
  int tok, heads_per_block;
  float eps, k_scale, v_scale;
};
struct IoFreq {
  uint64_t f[128];
};

// Element offset of (slot, K half, head 0) in the cache, and the steps to the
// next head and to the V half.
struct SlotMap {
  long long head, half;
};
POD_DEV SlotMap slot_steps(int ps, int Hk, int D, int hnd) {
  SlotMap m;
  m.head = hnd ? (long long)ps * D : D;
  m.half = (long long)ps * Hk * D;
  return m;
}
POD_DEV long long slot_base(long long slot, int ps, int Hk, int D, int hnd) {
  const long long page = slot / ps;
  const int in = (int)(slot - page * ps);
  return (page * 2 * ps * Hk + (hnd ? (long long)in : (long long)in * Hk)) * D;
}

// exponent byte of the smallest power of two 2^e with amax <= 448 * 2^e
// (448 = 1.75 * 2^8), from the bits of the non-negative fp32 amax
POD_DEV int block_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -127) + 127;
}
// 2^(127 - byte): the factor that takes a value to its code's range
POD_DEV float inv_scale_of(int byte) {
  return byte == 254 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)(254 - byte) << 23);
}
// 2^(byte - 127) (2^-127 is subnormal)
POD_DEV float scale_of(int byte) {
  return byte == 0 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)byte << 23);
}

template <typename T>
POD_DEV void unpack8(const uint4& r, float* x) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Pack<T>::unpack(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <typename T>
POD_DEV uint4 pack8(const float* x) {
  return make_uint4(Pack<T>::two(x[0], x[1]), Pack<T>::two(x[2], x[3]), Pack<T>::two(x[4], x[5]),
                    Pack<T>::two(x[6], x[7]));
}
POD_DEV uint2 codes8(const float* x) {
  return make_uint2(f32x2_to_e4m3x2(x[0], x[1]) | (f32x2_to_e4m3x2(x[2], x[3]) << 16),
                    f32x2_to_e4m3x2(x[4], x[5]) | (f32x2_to_e4m3x2(x[6], x[7]) << 16));
}

// One pass over q, k and (with a cache) v. FUSED: norm and rotation of q and
// k; without it the rows are only written.
template <typename T, int D, int FMT, bool FUSED>
__global__ void __launch_bounds__(kIoThreads) cache_io_kernel(const __grid_constant__ IoParams P,
                                                              const __grid_constant__ IoFreq F) {
  constexpr int LPR = D / 8;                     // lanes per head row
  constexpr int NG = kIoThreads / LPR;           // head rows per pass of the block
  constexpr bool CACHE = FMT != FMT_NONE;
  __shared__ float4 cs[FUSED ? kMaxTok * D / 4 : 1];
  __shared__ long long base[kMaxTok];
  const int tid = threadIdx.x, lane = tid % LPR;
  const int tok0 = blockIdx.x * P.tok, ntok = min(P.tok, P.rows - tok0);
  const int half = P.R >> 1;

  if (CACHE && tid < ntok) {
    const long long s = P.slots[tok0 + tid];
    long long b = -1;
    if (s >= 0 && s < P.num_slots) b = slot_base(s, P.ps, P.Hk, D, P.hnd);
    else if (s >= P.num_slots && P.status && blockIdx.y == 0) atomicOr(P.status, kStatusSlot);
    base[tid] = b;
  }
  if (FUSED) {
    // (cos, sin) of pair j of a token, stored so that the lanes of a head row
    // read neighbouring 16-byte chunks: chunk c of lane l holds its pairs 2c, 2c+1
    float2* t2 = reinterpret_cast<float2*>(cs);
    const int per = P.interleaved ? 4 : 8;       // pairs a lane reads
    const int nl = P.R ? half / per : 1;         // lanes that hold distinct pairs
    for (int i = tid; i < ntok * half; i += kIoThreads) {
      const int t = i / half, j = i - t * half;
      const uint64_t ph = (uint64_t)(int64_t)P.pos[tok0 + t] * F.f[j];
      const float fr = (float)(int32_t)(ph >> 32) * 4.656612873077393e-10f;   // half turns: 2^-31
      float sn, c;
      sincospif(fr, &sn, &c);
      const int l = j / per, i8 = j - l * per;
      t2[t * half + ((i8 >> 1) * nl + l) * 2 + (i8 & 1)] = make_float2(c, sn);
    }
  }
  if (CACHE || FUSED) __syncthreads();

  const int HT = P.H + P.Hk + (CACHE ? P.Hk : 0);
  const int h0 = blockIdx.y * P.heads_per_block, nh = min(P.heads_per_block, HT - h0);
  const int n = ntok * nh;
  const T* __restrict__ q = static_cast<const T*>(P.q);
  const T* __restrict__ k = static_cast<const T*>(P.k);
  const T* __restrict__ v = static_cast<const T*>(P.v);
  const SlotMap sm = slot_steps(P.ps, P.Hk, D, P.hnd);
  const int e0 = lane * 8;

  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (FUSED) {
    if (P.qw) wq = *reinterpret_cast<const uint4*>(static_cast<const T*>(P.qw) + e0);
    if (P.kw) wk = *reinterpret_cast<const uint4*>(static_cast<const T*>(P.kw) + e0);
  }
  // a task index advances by NG: (token, head) advance by these steps
  const int dt = NG / nh, dh = NG - dt * nh;
  int idx = tid / LPR, t = idx / nh, h = idx - t * nh;
  for (int first = 0; first < n; first += NG * kUnroll) {
    uint4 raw[kUnroll];
    int tk[kUnroll], hd[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      raw[u] = make_uint4(0, 0, 0, 0);
      tk[u] = -1;
      hd[u] = h0 + h;
      if (idx < n) {
        tk[u] = t;
        const long long r = tok0 + t;
        const int hh = h0 + h;
        const T* src = hh < P.H ? q + r * P.q_stride + hh * D
                       : hh < P.H + P.Hk ? k + r * P.k_stride + (hh - P.H) * D
                                         : v + r * P.v_stride + (hh - P.H - P.Hk) * D;
        raw[u] = __ldcs(reinterpret_cast<const uint4*>(src + e0));   // read once
      }
      idx += NG;
      t += dt;
      h += dh;
      if (h >= nh) { h -= nh; ++t; }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (first + u * NG >= n) break;            // (uniform over the block)
      const bool live = tk[u] >= 0;
      const int hh = hd[u];
      const bool is_q = hh < P.H, is_k = !is_q && hh < P.H + P.Hk;
      float x[8];
      unpack8<T>(raw[u], x);
      if (FUSED) {
        // the shuffles run for every row of the warp, their results are used
        // by the q and k rows
        const bool norm = is_q ? P.qw != nullptr : (is_k && P.kw != nullptr);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, LPR);
        if (norm) {
          const float rs = rsqrtf(ss * (1.f / D) + P.eps);
          float w[8];
          unpack8<T>(is_q ? wq : wk, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * rs * w[i];
        }
        if (P.R) {
          const bool rot = (is_q || is_k) && live && e0 < P.R;
          const float4* tc = cs + (live ? tk[u] : 0) * (half / 2);
          if (P.interleaved) {
            if (rot) {
              const int nl = half / 4;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float4 a = tc[c * nl + lane];
                const float x0 = x[4 * c], x1 = x[4 * c + 1], x2 = x[4 * c + 2], x3 = x[4 * c + 3];
                x[4 * c] = x0 * a.x - x1 * a.y;
                x[4 * c + 1] = x1 * a.x + x0 * a.y;
                x[4 * c + 2] = x2 * a.z - x3 * a.w;
                x[4 * c + 3] = x3 * a.z + x2 * a.w;
              }
            }
          } else {
            const int nl = half / 8;             // lanes in the first half of the pairs
            const bool low = lane < nl;
            const int partner = rot ? (low ? lane + nl : lane - nl) : lane;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner, LPR);
            if (rot) {
              const int l = low ? lane : lane - nl;
              const float sg = low ? -1.f : 1.f;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float4 a = tc[c * nl + l];
                x[2 * c] = fmaf(x[2 * c], a.x, sg * y[2 * c] * a.y);
                x[2 * c + 1] = fmaf(x[2 * c + 1], a.z, sg * y[2 * c + 1] * a.w);
              }
            }
          }
        }
      }
      int ebyte = 0;
      if (FMT == FMT_BLOCK) {
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(x[i]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o, LPR));
        ebyte = block_exp(am);
      }
      if (!live) continue;
      const long long r = tok0 + tk[u];
      if (is_q) {
        *reinterpret_cast<uint4*>(static_cast<T*>(P.q_out) + r * P.qo_stride + hh * D + e0) = pack8<T>(x);
      } else if (!CACHE) {
        *reinterpret_cast<uint4*>(static_cast<T*>(P.k_out) + r * P.ko_stride + (hh - P.H) * D + e0) =
            pack8<T>(x);
      } else {
        const long long b = base[tk[u]];
        if (b >= 0) {
          const int hk = is_k ? hh - P.H : hh - P.H - P.Hk;
          const long long off = b + hk * sm.head + (is_k ? 0 : sm.half);
          if (FMT == FMT_16) {
            *reinterpret_cast<uint4*>(static_cast<T*>(P.cache) + off + e0) =
                FUSED && is_k ? pack8<T>(x) : raw[u];
          } else {
            if (FMT == FMT_SCALED) {
              const float s = is_k ? P.k_scale : P.v_scale;
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], s);
            } else {
              const float s = inv_scale_of(ebyte);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] *= s;
              if (lane == 0) P.scales[off / D] = (uint8_t)ebyte;
            }
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(P.cache) + off + e0) = codes8(x);
          }
        }
      }
    }
  }
}

// Cache rows back as 16-bit values: out[row][K, V][Hk][D]. A lane takes 16
// bytes of cache: 16 codes, or 8 values of a 16-bit cache. Finite values past
// the largest of T saturate. A negative slot gives a row of zeros.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kIoThreads) cache_read_kernel(const __grid_constant__ IoParams P) {
  constexpr int EPL = FMT == FMT_16 ? 8 : 16;    // elements per lane
  constexpr int LPR = D / EPL, NG = kIoThreads / LPR;
  __shared__ long long base[kMaxTok];
  const int tid = threadIdx.x, lane = tid % LPR, e0 = lane * EPL;
  const int tok0 = blockIdx.x * P.tok, ntok = min(P.tok, P.rows - tok0);
  if (tid < ntok) {
    const long long s = P.slots[tok0 + tid];
    long long b = -1;
    if (s >= 0 && s < P.num_slots) b = slot_base(s, P.ps, P.Hk, D, P.hnd);
    else if (s >= P.num_slots && P.status && blockIdx.y == 0) atomicOr(P.status, kStatusSlot);
    base[tid] = b;
  }
  __syncthreads();
  const int HT = 2 * P.Hk;
  const int h0 = blockIdx.y * P.heads_per_block, nh = min(P.heads_per_block, HT - h0);
  const int n = ntok * nh;
  const SlotMap sm = slot_steps(P.ps, P.Hk, D, P.hnd);
  const int dt = NG / nh, dh = NG - dt * nh;
  int idx = tid / LPR, t = idx / nh, h = idx - t * nh;
  const float big = Pack<T>::kBF16 ? 3.3895313892515355e38f : 65504.f;
  for (int first = 0; first < n; first += NG * kUnroll) {
    uint4 raw[kUnroll];
    int eb[kUnroll], tk[kUnroll], hd[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      raw[u] = make_uint4(0, 0, 0, 0);
      eb[u] = 127;
      tk[u] = idx < n ? t : -1;
      hd[u] = h0 + h;
      if (idx < n && base[t] >= 0) {
        const int hh = h0 + h;
        const bool is_v = hh >= P.Hk;
        const long long off = base[t] + (is_v ? hh - P.Hk : hh) * sm.head + (is_v ? sm.half : 0);
        raw[u] = __ldcs(reinterpret_cast<const uint4*>(
            static_cast<const uint8_t*>(P.cache) + (off + e0) * (FMT == FMT_16 ? 2 : 1)));
        if (FMT == FMT_BLOCK) eb[u] = P.scales[off / D];
      }
      idx += NG;
      t += dt;
      h += dh;
      if (h >= nh) { h -= nh; ++t; }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (tk[u] < 0) continue;
      T* dst = static_cast<T*>(P.k_out) + ((long long)(tok0 + tk[u]) * HT + hd[u]) * D + e0;
      if (FMT == FMT_16) {
        __stcs(reinterpret_cast<uint4*>(dst), raw[u]);
      } else {
        const float s = FMT == FMT_BLOCK ? scale_of(eb[u]) : (hd[u] >= P.Hk ? P.v_scale : P.k_scale);
        const uint32_t c[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
        float x[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t h2 = e4m3x2_to<__half>((uint16_t)(c[i >> 1] >> (16 * (i & 1))));
          const float2 f = Pack<__half>::unpack(h2);
          // (a NaN code stays NaN: the comparisons are false)
          float a = f.x * s, b = f.y * s;
          a = a > big ? big : a < -big ? -big : a;
          b = b > big ? big : b < -big ? -big : b;
          x[2 * i] = a;
          x[2 * i + 1] = b;
        }
        __stcs(reinterpret_cast<uint4*>(dst), pack8<T>(x));
        __stcs(reinterpret_cast<uint4*>(dst) + 1, pack8<T>(x + 8));
      }
    }
  }
}

// ------------------------------------------------------------------ host
pod_status fail(pod_status code, const std::string& msg) {
  pod_set_last_error(msg);
  return code;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Tokens per block and heads per block: a block should have a few head rows
// for each lane group, and a short call should still reach every SM.
void shape_of(IoParams& P, int heads, int ng, dim3* grid) {
  const long long total = (long long)P.rows * heads;
  const long long want = 152 * 4;                             // blocks that fill the GPU
  long long per = (total + want - 1) / want;                  // head rows per block
  per = per < ng ? ng : per > ng * 16 ? ng * 16 : per;
  int tok = (int)(per / heads);
  tok = tok < 1 ? 1 : tok > kMaxTok ? kMaxTok : tok;
  int split = 1;
  if (tok == 1) split = (int)((heads + per - 1) / per);
  P.tok = tok;
  P.heads_per_block = (heads + split - 1) / split;
  *grid = dim3((unsigned)((P.rows + tok - 1) / tok),
               (unsigned)((heads + P.heads_per_block - 1) / P.heads_per_block));
}

// Frequencies in turns as 64-bit fractions. They depend on the rotation's
// settings only; the last settings' table is kept per host thread (computing
// it takes longer than a short launch).
const IoFreq& freq_of(int R, float scale, float theta) {
  struct Kept {
    int R = -1;
    float scale = 0.f, theta = 0.f;
    IoFreq f;
  };
  static thread_local Kept kept;
  if (kept.R != R || kept.scale != scale || kept.theta != theta) {
    memset(&kept.f, 0, sizeof(kept.f));
    for (int j = 0; j < R / 2; ++j) {
      const double turns = pow((double)theta, -2.0 * j / R) / (2.0 * 3.14159265358979323846 * scale);
      kept.f.f[j] = (uint64_t)ldexp(turns - floor(turns), 64);
    }
    kept.R = R;
    kept.scale = scale;
    kept.theta = theta;
  }
  return kept.f;
}

template <typename T, int D, int FMT>
cudaError_t launch_io(IoParams& P, bool fused, const IoFreq& f, cudaStream_t st) {
  dim3 grid;
  shape_of(P, P.H + P.Hk + (FMT == FMT_NONE ? 0 : P.Hk), kIoThreads / (D / 8), &grid);
  if (fused)
    cache_io_kernel<T, D, FMT, true><<<grid, kIoThreads, 0, st>>>(P, f);
  else if constexpr (FMT != FMT_NONE)
    cache_io_kernel<T, D, FMT, false><<<grid, kIoThreads, 0, st>>>(P, f);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_fmt(IoParams& P, int fmt, bool fused, const IoFreq& f, cudaStream_t st) {
  switch (fmt) {
    case FMT_16: return launch_io<T, D, FMT_16>(P, fused, f, st);
    case FMT_SCALED: return launch_io<T, D, FMT_SCALED>(P, fused, f, st);
    case FMT_BLOCK: return launch_io<T, D, FMT_BLOCK>(P, fused, f, st);
    default: return launch_io<T, D, FMT_NONE>(P, fused, f, st);
  }
}
template <typename T>
cudaError_t launch_d(IoParams& P, int d, int fmt, bool fused, const IoFreq& f, cudaStream_t st) {
  return d == 64 ? launch_fmt<T, 64>(P, fmt, fused, f, st)
         : d == 128 ? launch_fmt<T, 128>(P, fmt, fused, f, st)
                    : launch_fmt<T, 256>(P, fmt, fused, f, st);
}
template <typename T, int D>
cudaError_t launch_read(IoParams& P, int fmt, cudaStream_t st) {
  dim3 grid;
  shape_of(P, 2 * P.Hk, kIoThreads / (D / (fmt == FMT_16 ? 8 : 16)), &grid);
  if (fmt == FMT_16) cache_read_kernel<T, D, FMT_16><<<grid, kIoThreads, 0, st>>>(P);
  else if (fmt == FMT_SCALED) cache_read_kernel<T, D, FMT_SCALED><<<grid, kIoThreads, 0, st>>>(P);
  else cache_read_kernel<T, D, FMT_BLOCK><<<grid, kIoThreads, 0, st>>>(P);
  return cudaGetLastError();
}

pod_status check_rows(const char* what, const void* p, int64_t stride, int64_t heads, int d) {
  if (!p) return fail(POD_ERR_INVALID_ARG, std::string(what) + " is NULL");
  if (!aligned16(p)) return fail(POD_ERR_INVALID_ARG, std::string(what) + " must be 16-byte aligned");
  if (stride < heads * d || stride % 8 != 0)
    return fail(POD_ERR_INVALID_ARG, std::string(what) +
                                         ": the row stride must be a multiple of 8 elements and "
                                         "hold the row's heads");
  return POD_OK;
}

pod_status check_common(const pod_io_args& a) {
  if (a.rows < 0 || a.rows > 0x7fffffff) return fail(POD_ERR_INVALID_ARG, "rows must be in [0, 2^31)");
  if (a.dtype != POD_F16 && a.dtype != POD_BF16) return fail(POD_ERR_UNSUPPORTED, "dtype must be fp16 or bf16");
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256)
    return fail(POD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  return POD_OK;
}

// norm and rotation: settings, q, weights
pod_status check_rope(const pod_io_args& a) {
  const int R = a.rotary_dim;
  if (a.num_qo_heads < 0 || a.num_qo_heads > 65536) return fail(POD_ERR_INVALID_ARG, "no heads, or too many");
  if (R < 0 || R > a.head_dim || R % 16 != 0)
    return fail(POD_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 in [0, head_dim]");
  if (R && a.rows && !a.positions) return fail(POD_ERR_INVALID_ARG, "positions is NULL");
  if (R && !(a.rope_scale > 0.f && a.rope_theta > 0.f && isfinite(a.rope_scale) && isfinite(a.rope_theta)))
    return fail(POD_ERR_INVALID_ARG, "rope_scale and rope_theta must be finite and positive");
  if (!(a.eps >= 0.f) || !isfinite(a.eps)) return fail(POD_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (a.rows && a.num_qo_heads) {
    pod_status st = check_rows("q", a.q, a.q_stride, a.num_qo_heads, a.head_dim);
    if (st == POD_OK) st = check_rows("q_out", a.q_out, a.q_out_stride, a.num_qo_heads, a.head_dim);
    if (st != POD_OK) return st;
  }
  if (!aligned16(a.q_weight) || !aligned16(a.k_weight))
    return fail(POD_ERR_INVALID_ARG, "the norm weights must be 16-byte aligned");
  return POD_OK;
}

pod_status check_cache(const pod_io_args& a) {
  const int fmt = a.kv_format;
  if (fmt != FMT_16 && fmt != FMT_SCALED && fmt != FMT_BLOCK)
    return fail(POD_ERR_INVALID_ARG, "unknown cache format");
  if (a.kv_layout != 0 && a.kv_layout != 1) return fail(POD_ERR_INVALID_ARG, "kv_layout must be 0 (NHD) or 1 (HND)");
  if (a.num_kv_heads < 1 || a.num_kv_heads > 4096) return fail(POD_ERR_INVALID_ARG, "num_kv_heads must be in [1, 4096]");
  if (a.page_size < 1 || a.num_pages < 1) return fail(POD_ERR_INVALID_ARG, "the page pool is empty");
  // (the element offset of the pool's end has to fit 63 bits)
  if (a.num_pages > (1ll << 50) / ((int64_t)a.page_size * a.num_kv_heads))
    return fail(POD_ERR_INVALID_ARG, "the page pool is too large");
  if (!a.kv_cache || !aligned16(a.kv_cache))
    return fail(POD_ERR_INVALID_ARG, "the cache must be a 16-byte aligned pointer");
  if (fmt == FMT_BLOCK && !a.kv_scales) return fail(POD_ERR_INVALID_ARG, "a block-scaled cache needs its scales");
  if (fmt != FMT_BLOCK && a.kv_scales) return fail(POD_ERR_INVALID_ARG, "scales given, but the cache format has none");
  if (fmt == FMT_SCALED && !(a.k_scale > 0.f && a.v_scale > 0.f && isfinite(a.k_scale) && isfinite(a.v_scale)))
    return fail(POD_ERR_INVALID_ARG, "k_scale and v_scale must be finite and positive");
  return POD_OK;
}

// the rows of a write
pod_status check_written(const pod_io_args& a) {
  if (!a.rows) return POD_OK;
  if (!a.slots) return fail(POD_ERR_INVALID_ARG, "slots is NULL");
  const pod_status st = check_rows("k", a.k, a.k_stride, a.num_kv_heads, a.head_dim);
  return st != POD_OK ? st : check_rows("v", a.v, a.v_stride, a.num_kv_heads, a.head_dim);
}

IoParams params_of(const pod_io_args& a, bool fused, bool cache) {
  IoParams P = {};
  P.rows = (int)a.rows;
  P.k = a.k; P.k_stride = a.k_stride;
  P.k_out = a.k_out; P.ko_stride = a.k_out_stride;
  P.Hk = a.num_kv_heads; P.ps = 1;
  if (fused) {
    P.q = a.q; P.q_out = a.q_out; P.q_stride = a.q_stride; P.qo_stride = a.q_out_stride;
    P.qw = a.q_weight; P.kw = a.k_weight; P.pos = a.positions;
    P.H = a.num_qo_heads; P.R = a.rotary_dim; P.interleaved = a.interleaved != 0; P.eps = a.eps;
  }
  if (cache) {
    P.v = a.v; P.v_stride = a.v_stride;
    P.slots = a.slots; P.cache = a.kv_cache; P.scales = a.kv_scales; P.status = a.status;
    P.num_slots = a.num_pages * a.page_size;
    P.ps = a.page_size; P.hnd = a.kv_layout;
    P.k_scale = a.k_scale; P.v_scale = a.v_scale;
  }
  return P;
}

pod_status run_io(IoParams& P, const pod_io_args& a, int fmt, bool fused, void* stream, const char* what) {
  if (P.rows == 0) return POD_OK;
  const IoFreq& f = freq_of(P.R, a.rope_scale, a.rope_theta);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = a.dtype == POD_BF16 ? launch_d<__nv_bfloat16>(P, a.head_dim, fmt, fused, f, st)
                                            : launch_d<__half>(P, a.head_dim, fmt, fused, f, st);
  if (e != cudaSuccess) return fail(POD_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
  return POD_OK;
}

}  // namespace

#define POD_TRY(x)                      \
  do {                                  \
    const pod_status st_ = (x);         \
    if (st_ != POD_OK) return st_;      \
  } while (0)

extern "C" {

pod_status pod_qk_norm_rope(const pod_io_args* a, void* stream) {
  pod_set_last_error("");
  if (!a) return fail(POD_ERR_INVALID_ARG, "args is NULL");
  POD_TRY(check_common(*a));
  if (a->num_kv_heads < 0 || a->num_kv_heads > 4096 || a->num_qo_heads + (int64_t)a->num_kv_heads < 1)
    return fail(POD_ERR_INVALID_ARG, "no heads, or too many");
  POD_TRY(check_rope(*a));
  if (a->rows && a->num_kv_heads) {
    POD_TRY(check_rows("k", a->k, a->k_stride, a->num_kv_heads, a->head_dim));
    POD_TRY(check_rows("k_out", a->k_out, a->k_out_stride, a->num_kv_heads, a->head_dim));
  }
  IoParams P = params_of(*a, true, false);
  return run_io(P, *a, FMT_NONE, true, stream, "norm and rotation launch");
}

pod_status pod_append_kv(const pod_io_args* a, void* stream) {
  pod_set_last_error("");
  if (!a) return fail(POD_ERR_INVALID_ARG, "args is NULL");
  POD_TRY(check_common(*a));
  POD_TRY(check_cache(*a));
  POD_TRY(check_written(*a));
  IoParams P = params_of(*a, false, true);
  return run_io(P, *a, a->kv_format, false, stream, "cache write launch");
}

pod_status pod_norm_rope_append(const pod_io_args* a, void* stream) {
  pod_set_last_error("");
  if (!a) return fail(POD_ERR_INVALID_ARG, "args is NULL");
  POD_TRY(check_common(*a));
  POD_TRY(check_cache(*a));
  POD_TRY(check_rope(*a));
  POD_TRY(check_written(*a));
  IoParams P = params_of(*a, true, true);
  return run_io(P, *a, a->kv_format, true, stream, "norm, rotation and cache write launch");
}

pod_status pod_gather_kv(const pod_io_args* a, void* stream) {
  pod_set_last_error("");
  if (!a) return fail(POD_ERR_INVALID_ARG, "args is NULL");
  POD_TRY(check_common(*a));
  POD_TRY(check_cache(*a));
  if (a->rows == 0) return POD_OK;
  if (!a->slots) return fail(POD_ERR_INVALID_ARG, "slots is NULL");
  POD_TRY(check_rows("k_out", a->k_out, 2ll * a->num_kv_heads * a->head_dim, 2ll * a->num_kv_heads, a->head_dim));
  IoParams P = params_of(*a, false, true);
  cudaStream_t st = (cudaStream_t)stream;
  const int fmt = a->kv_format, d = a->head_dim;
  cudaError_t e;
  if (a->dtype == POD_BF16)
    e = d == 64 ? launch_read<__nv_bfloat16, 64>(P, fmt, st)
        : d == 128 ? launch_read<__nv_bfloat16, 128>(P, fmt, st)
                   : launch_read<__nv_bfloat16, 256>(P, fmt, st);
  else
    e = d == 64 ? launch_read<__half, 64>(P, fmt, st)
        : d == 128 ? launch_read<__half, 128>(P, fmt, st)
                   : launch_read<__half, 256>(P, fmt, st);
  if (e != cudaSuccess) return fail(POD_ERR_CUDA, std::string("cache read launch: ") + cudaGetErrorString(e));
  return POD_OK;
}

}  // extern "C"
