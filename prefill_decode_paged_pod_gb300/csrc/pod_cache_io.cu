// pod_cache_io.cu — the operators around the paged cache: per-head RMS norm of
// queries and keys with the position rotation, the write of keys and values
// into the cache (16-bit, E4M3 with per-tensor scales, E4M3 with a power-of-two
// scale per token and KV head), and the read of cache rows back as 16-bit
// values.
//
// Mathematics. A head row x of d elements becomes
//   y = x * (mean(x^2) + eps)^(-1/2) * w, then the pairs (j, j + R/2) or
//   (2j, 2j + 1), j < R/2, turn by the angle pos / rope_scale * theta^(-2j/R).
// Rows and weights may have any magnitude of their type (see io_pass).
// The angle is kept in turns as a 64-bit fixed-point fraction: the per-turn
// frequency F = theta^(-2j/R) / (2 pi rope_scale) * 2^64 is an integer, and
// pos * F modulo 2^64 is the exact fraction of a turn for that F (whole turns
// drop out by themselves, for negative positions too). F is off by a unit, so the
// angle by pos * 2^-64 of a turn: far positions cost no 64-bit floating point, of
// which this GPU has little. Everything else runs in fp32 and is rounded once, at
// the store.
//
// A power-of-two block scale 2^e is the smallest with amax <= 448 * 2^e. E4M3
// is a floating-point format, so a power of two costs no significant bit
// against the exact quotient amax / 448 (at most one of its 17 binades), the
// product with it is exact, and it is stored in one byte (exponent + 127).
//
// Work split. A head row is read by d/16 lanes with two 16-byte loads each. Where
// the halves of the head are paired, a lane takes the 16-byte chunks c and
// c + R/16, so it holds both elements of its 8 pairs; the chunks past the rotated
// part go two neighbours to a lane. A block works on queries, keys or values
// only: some heads of some tokens, two head rows in flight a lane group, the
// first of them asked for before the block makes its tables (cos and sin once
// per token, the norm weights) in shared memory. fp32 arithmetic is paired
// (f32x2). A first form held one 16-byte chunk a lane and turned pairs by
// shuffles: 230 instructions per 8 elements, and bound by them (below, in
// brackets).
//
// Measured on a GB300, back to back in a graph over several inputs, with the share of
// the measured copy rate: norm and rotation of 8796 rows of 64/8 heads of 128, bf16:
// 58.8 us, 83 % (84); 4096 rows of 64/8 heads normed, turned and written: 30.7 us, 82 %
// (45); 16384 rows of 8 heads written with block scales: 18.8 us, 81 % (26.6); 65536
// rows read back: 63.7 us, 95 %. Calls of a few hundred rows take 4 to 5 us, the
// launch and two dependent trips to memory.
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <string>

#include "../../include/pod.h"
#include "pod_beside.h"
#include "pod_device.cuh"
#include "pod_turns.h"

void pod_set_last_error(const std::string& msg);

using namespace pod;

namespace {

constexpr int kIoThreads = 256;
constexpr int kMaxTok = 16;       // tokens per block
constexpr int kUnroll = 4;        // cache rows in flight per lane group (read)
constexpr int kTasks = 2;         // head rows in flight per lane group (write)
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
  // how each kind of row (queries, keys, values; reads: keys then values) is cut
  // into blocks: tokens and heads of a block, head ranges per token group, first
  // block of the grid
  struct Cut {
    int tok, heads, ranges, first;
  } cut[3];
  float eps, k_scale, v_scale;
  float k_inv, v_inv;            // reciprocals, rounded to nearest; 0: divide
};
template <int D>
struct IoFreq {                  // (a kernel parameter: no longer than it has to be)
  uint64_t f[D / 2];
};

// The kernels are launched beside the one before (programmatic stream
// serialization) and wait for it here; so may the next. One call after another:
// 16384 block-scaled rows written 20.1 -> 18.2 us, 4096 rows normed and written 32.7
// -> 30.8, 65536 read 66.5 -> 64.3.
POD_DEV void after_the_last_kernel() {
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}

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
  const long long page = (ps & (ps - 1)) == 0 ? slot >> (__ffs(ps) - 1) : slot / ps;
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
// 2^(127 - byte): the factor that takes a value to its code's range (block_exp ends at
// 247, an infinite amax)
POD_DEV float inv_scale_of(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }
// 2^(byte - 127) (2^-127 is subnormal)
POD_DEV float scale_of(int byte) {
  return byte == 0 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)byte << 23);
}

template <typename T>
POD_DEV uint4 pack8(const float* x) {
  return make_uint4(Pack<T>::two(x[0], x[1]), Pack<T>::two(x[2], x[3]), Pack<T>::two(x[4], x[5]),
                    Pack<T>::two(x[6], x[7]));
}
// 8 values of a 16-byte chunk as 4 fp32 pairs, and back
template <typename T>
POD_DEV void unpack8(const uint4& r, uint64_t* x) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Pack<T>::unpack(u[i]);
    x[i] = pack2(f.x, f.y);
  }
}
template <typename T>
POD_DEV uint4 pack8(const uint64_t* x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2(x[i], a, b);
    u[i] = Pack<T>::two(a, b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
POD_DEV uint2 codes8(const uint64_t* x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2(x[i], a, b);
    u[i] = f32x2_to_e4m3x2(a, b);
  }
  return make_uint2(u[0] | (u[1] << 16), u[2] | (u[3] << 16));
}

// x / s rounded to nearest, from y = 1 / s rounded to nearest (Markstein: q = x y
// is within an ulp of the quotient, and q + (x - q s) y rounds it correctly).
// Quotients past 2^100, where the remainder may overflow, stay as q, for they
// saturate either way, and so do zeros, for their sign. The host gives y = 0 for
// scales whose products could leave the normal range: then divide.
POD_DEV uint64_t div2(uint64_t x, float s, float y) {
  float a, b;
  if (y == 0.f) {
    unpack2(x, a, b);
    return pack2(__fdiv_rn(a, s), __fdiv_rn(b, s));
  }
  const uint64_t y2 = pack2(y, y), q = mul2(x, y2);
  const uint64_t r = fma2(fma2(q, pack2(-s, -s), x), y2, q);
  float qa, qb;
  unpack2(q, qa, qb);
  unpack2(r, a, b);
  auto in = [](float v) { return (__float_as_uint(v) & 0x7fffffffu) - 1u < 0x71800000u - 1u; };   // (0, 2^100)
  return pack2(in(qa) ? a : qa, in(qb) ? b : qb);
}

enum { IO_Q, IO_K, IO_V, IO_KV };

// The tables of a block: cos and sin of its tokens, and the norm weights, chunked
// so that the lanes of a head row read neighbouring 16 bytes.
template <int D>
struct IoTables {
  float4 cs[kMaxTok * D / 4];    // [token][4 (2 interleaved, per chunk)][lane]: c, c', s, s'
  float4 w[4][D / 16];           // [quarter of a lane's 16 elements][lane]
};

// The block's tokens: where their rows go, and cos and sin of their positions.
// Returns whether this thread's norm weight is out of the ordinary: neither 0 nor
// within 2^+-30.
template <typename T, int D, bool CACHE, bool TURN, int FD>
POD_DEV bool io_tables(const IoParams& P, const IoFreq<FD>& F, IoTables<TURN ? D : 16>& S, long long* base, int tok0,
                       int ntok, const T* weight, bool report) {
  const int tid = threadIdx.x;
  bool far_weight = false;
  if (CACHE && tid < ntok) {
    const long long s = P.slots[tok0 + tid];
    long long b = -1;
    if (s >= 0 && s < P.num_slots) b = slot_base(s, P.ps, P.Hk, D, P.hnd);
    else if (s >= P.num_slots && P.status && report) atomicOr(P.status, kStatusSlot);
    base[tid] = b;
  }
  if constexpr (TURN) {
    const int half = P.R >> 1, turning = P.R >> 4;
    float* cs = reinterpret_cast<float*>(S.cs);
    for (int i = tid; i < ntok * half; i += kIoThreads) {
      const int t = i / half, j = i - t * half;
      const uint64_t ph = (uint64_t)(int64_t)P.pos[tok0 + t] * F.f[j];
      // the nearest quarter turn, and what is left of the angle: at most an eighth of
      // a turn, so that its rounding to fp32 is below that of cos and sin
      const int quarter = (int)((ph + (1ull << 61)) >> 62);
      const float fr = (float)(int)((long long)(ph - ((uint64_t)quarter << 62)) >> 30) * 0x1p-33f;   // half turns
      float s0, c0;
      sincospif(fr, &s0, &c0);
      const float c = __uint_as_float(__float_as_uint(quarter & 1 ? s0 : c0) ^ (uint32_t)((quarter + 1) & 2) << 30);
      const float sn = __uint_as_float(__float_as_uint(quarter & 1 ? c0 : s0) ^ (uint32_t)(quarter & 2) << 30);
      // a lane's 8 pairs: j = 8 lane + 0..7 in either pairing
      const int l = j >> 3, i8 = j & 7;
      float* at = cs + 4 * (t * (half / 2) + (i8 >> 1) * turning + l) + (i8 & 1);
      at[0] = c;
      at[2] = sn;
    }
    if (weight && tid < D) {
      // element e lies in chunk e / 8: which lane takes it, and as which of its 16?
      const int e = tid, c = e >> 3;
      int l = c >> 1, second = c & 1;
      if (!P.interleaved && c < 2 * turning) {
        second = c >= turning;
        l = second ? c - turning : c;
      }
      const int k = second * 8 + (e & 7);
      const float w = (float)weight[e];
      reinterpret_cast<float*>(&S.w[k >> 2][l])[k & 3] = w;
      far_weight = w != 0.f && !(fabsf(w) >= 0x1p-30f && fabsf(w) <= 0x1p30f);
    }
  }
  return far_weight;
}

// Sum of the squares of a head row, of which each of LPR lanes holds 16 elements.
template <int LPR>
POD_DEV float squares(const uint64_t* x) {
  uint64_t q2 = mul2(x[0], x[0]), q3 = mul2(x[1], x[1]);
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    q2 = fma2(x[i], x[i], q2);
    q3 = fma2(x[i + 1], x[i + 1], q3);
  }
  float a, b;
  unpack2(add2(q2, q3), a, b);
  float ss = a + b;
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, LPR);
  return ss;
}
// Largest magnitude of a head row; NaN does not count.
template <int LPR>
POD_DEV float largest(const uint64_t* x) {
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    unpack2(x[i], a, b);
    am = fmaxf(am, fmaxf(fabsf(a), fabsf(b)));
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o, LPR));
  return am;
}

// One block's tasks: some heads of one kind (IO_KV: K heads, then V heads) for
// some tokens. The rows of the first tasks are asked for before the tables are
// made.
template <typename T, int D, int FMT, int KIND, bool FUSED>
POD_DEV void io_pass(const IoParams& P, const IoFreq<FUSED ? D : 2>& F, const IoParams::Cut& cut) {
  constexpr int LPR = D / 16, NG = kIoThreads / LPR;
  constexpr bool TURN = FUSED && (KIND == IO_Q || KIND == IO_K);
  constexpr bool TO_CACHE = FMT != FMT_NONE && KIND != IO_Q;
  __shared__ IoTables<TURN ? D : 16> S;
  __shared__ long long base[kMaxTok];            // cache offset of the tokens' slots, -1: none
  const int blk = (int)blockIdx.x - cut.first, group = blk / cut.ranges;
  const int heads = KIND == IO_Q ? P.H : KIND == IO_KV ? 2 * P.Hk : P.Hk;
  const int tok0 = group * cut.tok, ntok = min(cut.tok, P.rows - tok0);
  const int h0 = (blk - group * cut.ranges) * cut.heads, h1 = min(h0 + cut.heads, heads);
  const int nh = h1 - h0, n = ntok * nh;
  const int lane = threadIdx.x % LPR;
  const int half = P.R >> 1, turning = P.R >> 4;           // lanes that turn pairs
  // this lane's two chunks
  const bool turns = FUSED && lane < turning;
  const bool split = turns && !P.interleaved;
  const int ca = split ? lane : 2 * lane, cb = split ? lane + turning : 2 * lane + 1;
  const SlotMap sm = slot_steps(P.ps, P.Hk, D, P.hnd);
  const T* weight = static_cast<const T*>(KIND == IO_Q ? P.qw : P.kw);
  const int dt = NG / nh, dh = NG - dt * nh;
  bool far_weights = false;                                // (of the block)
  int idx = threadIdx.x / LPR, t = idx / nh, h = idx - t * nh;
  for (int first = 0; first < n; first += NG * kTasks) {
    uint4 ra[kTasks], rb[kTasks];
    int tk[kTasks], hd[kTasks];
#pragma unroll
    for (int u = 0; u < kTasks; ++u) {
      ra[u] = rb[u] = make_uint4(0, 0, 0, 0);
      tk[u] = -1;
      hd[u] = h0 + h;
      if (idx < n) {
        tk[u] = t;
        const long long r = tok0 + t;
        const int hh = h0 + h;
        const T* src;
        if constexpr (KIND == IO_Q) src = static_cast<const T*>(P.q) + r * P.q_stride + hh * D;
        else if constexpr (KIND == IO_K) src = static_cast<const T*>(P.k) + r * P.k_stride + hh * D;
        else if constexpr (KIND == IO_V) src = static_cast<const T*>(P.v) + r * P.v_stride + hh * D;
        else
          src = hh < P.Hk ? static_cast<const T*>(P.k) + r * P.k_stride + hh * D
                          : static_cast<const T*>(P.v) + r * P.v_stride + (hh - P.Hk) * D;
        ra[u] = __ldcs(reinterpret_cast<const uint4*>(src) + ca);       // read once
        rb[u] = __ldcs(reinterpret_cast<const uint4*>(src) + cb);
      }
      idx += NG;
      t += dt;
      h += dh;
      if (h >= nh) { h -= nh; ++t; }
    }
    if (first == 0) {
      const bool far = io_tables<T, D, TO_CACHE, TURN>(P, F, S, base, tok0, ntok, weight, h0 == 0 && KIND != IO_V);
      if constexpr (TURN && Pack<T>::kBF16) far_weights = __syncthreads_or(far);
      else __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kTasks; ++u) {
      if (first + u * NG >= n) break;                      // (uniform over the block)
      const bool live = tk[u] >= 0;
      constexpr bool COPY = FMT == FMT_16 && !TURN;        // values go as they are
      uint64_t x[8];                                       // 4 pairs of chunk a, 4 of chunk b
      if constexpr (!COPY) {
        unpack8<T>(ra[u], x);
        unpack8<T>(rb[u], x + 4);
      }
      if constexpr (TURN) {
        if (weight) {
          float mean = squares<LPR>(x) * (1.f / D) + P.eps;
          // Squares, or products with the weights, that may leave fp32's range: the row
          // by a power of two that brings its largest element, or the root of eps where
          // that is more, near 1, which the norm undoes. (Zeros under an eps, the usual
          // padding, are not of these, and no fp16 row is.)
          const bool far = far_weights || !(mean >= 0x1p-64f && mean <= 0x1p64f);
          if (Pack<T>::kBF16 && __any_sync(0xffffffffu, far)) {
            const int ex = (int)(__float_as_uint(largest<LPR>(x)) >> 23) - 127;
            const int half_eps = P.eps == 0.f ? -127 : ((int)(__float_as_uint(P.eps) >> 23) - 127) >> 1;
            const int e = far ? min(max(max(ex, half_eps), -126), 126) : 0;
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);
            const uint64_t f2 = pack2(f, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], f2);
            mean = squares<LPR>(x) * (1.f / D) + P.eps * f * f;
          }
          const float rs = __frsqrt_rn(mean);
          const uint64_t rs2 = pack2(rs, rs);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 w = S.w[i][lane];
            x[2 * i] = mul2(mul2(x[2 * i], pack2(w.x, w.y)), rs2);   // (the first product is exact)
            x[2 * i + 1] = mul2(mul2(x[2 * i + 1], pack2(w.z, w.w)), rs2);
          }
        }
        if (turns) {
          const float4* tc = S.cs + (live ? tk[u] : 0) * (half / 2);
          if (split) {
            // pairs (chunk a, chunk b), element by element
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 c = tc[i * turning + lane];
              const uint64_t c2 = pack2(c.x, c.y), s2 = pack2(c.z, c.w), n2 = pack2(-c.z, -c.w);
              const uint64_t a = x[i], b = x[4 + i];
              x[i] = fma2(a, c2, mul2(b, n2));
              x[4 + i] = fma2(b, c2, mul2(a, s2));
            }
          } else {
            // neighbouring elements
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 c = tc[i * turning + lane];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float a, b;
                unpack2(x[2 * i + k], a, b);
                const float cc = k ? c.y : c.x, ss = k ? c.w : c.z;
                x[2 * i + k] = pack2(fmaf(a, cc, -b * ss), fmaf(b, cc, a * ss));
              }
            }
          }
        }
      }
      int ebyte = 0;
      if constexpr (TO_CACHE && FMT == FMT_BLOCK) {
        ebyte = block_exp(largest<LPR>(x));
      }
      if (!live) continue;
      const long long r = tok0 + tk[u];
      if constexpr (!TO_CACHE) {
        T* dst = KIND == IO_Q ? static_cast<T*>(P.q_out) + r * P.qo_stride + hd[u] * D
                              : static_cast<T*>(P.k_out) + r * P.ko_stride + hd[u] * D;
        reinterpret_cast<uint4*>(dst)[ca] = pack8<T>(x);
        reinterpret_cast<uint4*>(dst)[cb] = pack8<T>(x + 4);
      } else {
        const long long b = base[tk[u]];
        if (b < 0) continue;
        const bool is_v = KIND == IO_V || (KIND == IO_KV && hd[u] >= P.Hk);
        const int hk = KIND == IO_KV && is_v ? hd[u] - P.Hk : hd[u];
        const long long off = b + hk * sm.head + (is_v ? sm.half : 0);
        if constexpr (FMT == FMT_16) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(P.cache) + off);
          if constexpr (COPY) {
            dst[ca] = ra[u];
            dst[cb] = rb[u];
          } else {
            dst[ca] = pack8<T>(x);
            dst[cb] = pack8<T>(x + 4);
          }
        } else {
          if constexpr (FMT == FMT_SCALED) {
            const float s = is_v ? P.v_scale : P.k_scale, y = is_v ? P.v_inv : P.k_inv;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = div2(x[i], s, y);
          } else {
            const float s = inv_scale_of(ebyte);
            const uint64_t s2 = pack2(s, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], s2);
            if (lane == 0) P.scales[off / D] = (uint8_t)ebyte;
          }
          const uint2 qa = codes8(x), qb = codes8(x + 4);
          uint8_t* dst = static_cast<uint8_t*>(P.cache) + off;
          if (split) {
            *reinterpret_cast<uint2*>(dst + 8 * ca) = qa;
            *reinterpret_cast<uint2*>(dst + 8 * cb) = qb;
          } else {
            *reinterpret_cast<uint4*>(dst + 8 * ca) = make_uint4(qa.x, qa.y, qb.x, qb.y);
          }
        }
      }
    }
  }
}

// One launch over q, k and (with a cache) v; a block works on one of them.
// FUSED: norm and rotation of q and k; without it the rows are only written.
template <typename T, int D, int FMT, bool FUSED>
__global__ void __launch_bounds__(kIoThreads) cache_io_kernel(const __grid_constant__ IoParams P,
                                                              const __grid_constant__ IoFreq<FUSED ? D : 2> F) {
  after_the_last_kernel();
  if constexpr (FUSED) {
    if ((int)blockIdx.x < P.cut[1].first)
      io_pass<T, D, FMT, IO_Q, true>(P, F, P.cut[0]);
    else if (FMT == FMT_NONE || (int)blockIdx.x < P.cut[2].first)
      io_pass<T, D, FMT, IO_K, true>(P, F, P.cut[1]);
    else
      io_pass<T, D, FMT == FMT_NONE ? FMT_16 : FMT, IO_V, true>(P, F, P.cut[2]);
  } else {
    io_pass<T, D, FMT, IO_KV, false>(P, F, P.cut[0]);
  }
}

// Cache rows back as 16-bit values: out[row][K, V][Hk][D]. A lane takes 16
// bytes of cache: 16 codes, or 8 values of a 16-bit cache. Finite values past
// the largest of T saturate. A negative slot gives a row of zeros.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kIoThreads, 4) cache_read_kernel(const __grid_constant__ IoParams P) {
  after_the_last_kernel();
  constexpr int EPL = FMT == FMT_16 ? 8 : 16;    // elements per lane
  constexpr int LPR = D / EPL, NG = kIoThreads / LPR;
  __shared__ long long base[kMaxTok];
  const int tid = threadIdx.x, lane = tid % LPR, e0 = lane * EPL;
  const IoParams::Cut& cut = P.cut[0];
  const int group = (int)blockIdx.x / cut.ranges, h0 = ((int)blockIdx.x - group * cut.ranges) * cut.heads;
  const int tok0 = group * cut.tok, ntok = min(cut.tok, P.rows - tok0);
  if (tid < ntok) {
    const long long s = P.slots[tok0 + tid];
    long long b = -1;
    if (s >= 0 && s < P.num_slots) b = slot_base(s, P.ps, P.Hk, D, P.hnd);
    else if (s >= P.num_slots && P.status && h0 == 0) atomicOr(P.status, kStatusSlot);
    base[tid] = b;
  }
  __syncthreads();
  const int HT = 2 * P.Hk;
  const int nh = min(cut.heads, HT - h0), n = ntok * nh;
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

// How `heads` rows a token are cut into blocks of about `tasks` head rows: whole
// tokens, or a range of one token's heads. Returns the number of blocks.
long long cut_of(IoParams::Cut& c, long long first, int rows, int heads, long long tasks) {
  if (tasks < 1) tasks = 1;
  long long tok = tasks / heads;
  tok = tok < 1 ? 1 : tok > kMaxTok ? kMaxTok : tok;
  const long long ranges = heads > tasks ? (heads + tasks - 1) / tasks : 1;
  c.tok = (int)tok;
  c.heads = (int)((heads + ranges - 1) / ranges);
  c.ranges = (heads + c.heads - 1) / c.heads;
  c.first = (int)first;
  return (rows + tok - 1) / tok * c.ranges;
}

// Head rows of a block: one round of its lane groups for short calls, so that
// every SM gets some, up to `most` where that still leaves several blocks per SM
// (the tables of a block then serve more rows).
long long tasks_of(const IoParams& P, long long heads, int round, int most) {
  const long long total = (long long)P.rows * heads, wave = 152 * 4;
  long long t = (total + wave - 1) / wave;
  return t < round ? round : t > most * round ? most * round : t;
}

template <typename T, int D, int FMT>
cudaError_t launch_io(IoParams& P, bool fused, const Turns& f, cudaStream_t st) {
  constexpr int round = kIoThreads / (D / 16) * kTasks;
  constexpr bool cache = FMT != FMT_NONE;
  const long long tasks = tasks_of(P, P.H + P.Hk + (cache ? P.Hk : 0), round, fused ? 4 : 2);
  long long blocks = 0;
  if (fused) {
    if (P.H) blocks += cut_of(P.cut[0], blocks, P.rows, P.H, tasks);
    P.cut[1].first = P.cut[2].first = (int)blocks;
    if (P.Hk) blocks += cut_of(P.cut[1], blocks, P.rows, P.Hk, tasks);
    if (cache) blocks += cut_of(P.cut[2], blocks, P.rows, P.Hk, tasks);
  } else {
    blocks = cut_of(P.cut[0], 0, P.rows, 2 * P.Hk, tasks);
  }
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)blocks;
  if (fused) {
    IoFreq<D> fd;
    memcpy(&fd, f.f, sizeof(fd));
    return launch_beside(cache_io_kernel<T, D, FMT, true>, grid, kIoThreads, 0, 1, st, P, fd);
  } else if constexpr (cache) {
    return launch_beside(cache_io_kernel<T, D, FMT, false>, grid, kIoThreads, 0, 1, st, P, IoFreq<2>{});
  }
  return cudaErrorInvalidValue;                  // (a write without a cache is not asked for)
}
template <typename T, int D>
cudaError_t launch_fmt(IoParams& P, int fmt, bool fused, const Turns& f, cudaStream_t st) {
  switch (fmt) {
    case FMT_16: return launch_io<T, D, FMT_16>(P, fused, f, st);
    case FMT_SCALED: return launch_io<T, D, FMT_SCALED>(P, fused, f, st);
    case FMT_BLOCK: return launch_io<T, D, FMT_BLOCK>(P, fused, f, st);
    default: return launch_io<T, D, FMT_NONE>(P, fused, f, st);
  }
}
template <typename T>
cudaError_t launch_d(IoParams& P, int d, int fmt, bool fused, const Turns& f, cudaStream_t st) {
  return d == 64 ? launch_fmt<T, 64>(P, fmt, fused, f, st)
         : d == 128 ? launch_fmt<T, 128>(P, fmt, fused, f, st)
                    : launch_fmt<T, 256>(P, fmt, fused, f, st);
}
template <typename T, int D>
cudaError_t launch_read(IoParams& P, int fmt, cudaStream_t st) {
  const int round = kIoThreads / (D / (fmt == FMT_16 ? 8 : 16)) * kUnroll;
  const long long blocks = cut_of(P.cut[0], 0, P.rows, 2 * P.Hk, tasks_of(P, 2 * P.Hk, round, 2));
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)blocks;
  return fmt == FMT_16 ? launch_beside(cache_read_kernel<T, D, FMT_16>, grid, kIoThreads, 0, 1, st, P)
         : fmt == FMT_SCALED ? launch_beside(cache_read_kernel<T, D, FMT_SCALED>, grid, kIoThreads, 0, 1, st, P)
                             : launch_beside(cache_read_kernel<T, D, FMT_BLOCK>, grid, kIoThreads, 0, 1, st, P);
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
    // products of scales within 2^+-60 and fp32 values that matter stay normal
    auto inv = [](float s) { return s > 8.7e-19f && s < 1.15e18f ? 1.f / s : 0.f; };
    P.k_inv = inv(a.k_scale);
    P.v_inv = inv(a.v_scale);
  }
  return P;
}

pod_status run_io(IoParams& P, const pod_io_args& a, int fmt, bool fused, void* stream, const char* what) {
  if (P.rows == 0) return POD_OK;
  // (the frequencies depend on the rotation's settings only; a write has R = 0)
  static thread_local KeptTurns kept;
  const Turns& f = kept.of(P.R, a.rope_scale, a.rope_theta);
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
