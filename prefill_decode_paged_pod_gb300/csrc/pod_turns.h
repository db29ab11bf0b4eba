// pod_turns.h — frequencies of the position rotation, in turns (host only).
//
// F[j] = theta^(-2j/R) / (2 pi rope_scale) * 2^64 modulo 2^64, j < R/2: a position
// times F[j] modulo 2^64 is its angle as a 64-bit fraction of a turn. A position has up
// to 31 bits, so a frequency of 53 would leave 22 of the angle (1.3e-7 rad off at
// 2^31, theta = 1e4); these are computed as pairs of doubles (about 100 bits) and
// are off by one unit of 2^-64 at most, as long as a frequency is below 2^30 turns.
#pragma once
#include <math.h>
#include <stdint.h>
#include <string.h>

namespace pod {

struct Turns {
  uint64_t f[128];
};

namespace turns_detail {
struct DD {
  double hi, lo;
};
inline DD two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
inline DD mul(DD a, DD b) {
  const double p = a.hi * b.hi;
  return two_sum(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
inline DD div(DD a, double s) {
  const double q = a.hi / s;
  return two_sum(q, (fma(-q, s, a.hi) + a.lo) / s);
}
// the fraction of a, in units of 2^-64
inline uint64_t fraction(DD a) {
  const double h = ldexp(a.hi - floor(a.hi), 64), r = a.lo - nearbyint(a.lo);
  const double low = ldexp(r, 64) + (h - floor(h));     // (h has a fraction only below 2^53)
  return (uint64_t)h + (fabs(low) < 0x1p63 ? (uint64_t)(int64_t)nearbyint(low) : 1ull << 63);
}
}  // namespace turns_detail

// R a multiple of 16 up to 256; scale and theta finite and positive.
inline void make_turns(int R, float scale, float theta, Turns* out) {
  using namespace turns_detail;
  memset(out, 0, sizeof(*out));
  if (R == 0) return;
  const double th2 = (double)theta * theta;             // exact
  // y = theta^(-2/R), the root of y^R theta^2 = 1: a double, and one Newton step
  const double y0 = pow((double)theta, -2.0 / R);
  DD p = {1.0, 0.0}, sq = {y0, 0.0};
  for (int n = R; n; n >>= 1, sq = mul(sq, sq))
    if (n & 1) p = mul(p, sq);
  p = mul(p, {th2, 0.0});
  const DD y = two_sum(y0, -y0 * ((p.hi - 1.0) + p.lo) / R);
  const DD inv_2pi = {0.15915494309189535, -9.839338337591243e-18};
  DD turn = div(inv_2pi, (double)scale);
  for (int j = 0; j < R / 2; ++j, turn = mul(turn, y)) out->f[j] = fraction(turn);
}

// The tables of the last few settings: making one takes longer than a short launch
// does. R = 0 needs none and displaces none.
class KeptTurns {
 public:
  const Turns& of(int R, float scale, float theta) {
    static const Turns none = {};
    if (R == 0) return none;
    for (const Entry& e : kept_)
      if (e.R == R && e.scale == scale && e.theta == theta) return e.turns;
    Entry& e = kept_[made_++ % kEntries];
    make_turns(R, scale, theta, &e.turns);
    e.R = R;
    e.scale = scale;
    e.theta = theta;
    return e.turns;
  }
  unsigned made() const { return made_; }

 private:
  static constexpr unsigned kEntries = 4;
  struct Entry {
    int R = 0;
    float scale = 0.f, theta = 0.f;
    Turns turns;
  };
  Entry kept_[kEntries];
  unsigned made_ = 0;
};

}  // namespace pod
