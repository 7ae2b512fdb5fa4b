// rope_turns.h -- frequencies of the rotation on the host, to more digits than a
// double has: a position near 2^31 multiplies what is wrong with them.
//
// A value is hi + lo, lo below half a unit of hi.  Sums and products are the
// error-free ones (Knuth's two-sum; a product and its rest by a fused
// multiply-add); exp is the Taylor series of expm1 at x / 2^9, doubled nine times
// by e -> 2 e + e^2, and log one Newton step on it from the double's.
#pragma once

#include <cmath>

namespace vattn {
namespace host {

struct Twofold {
  double hi, lo;
};

inline Twofold two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
inline Twofold add(Twofold a, Twofold b) {
  const Twofold s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + (a.lo + b.lo));
}
inline Twofold mul(Twofold a, Twofold b) {
  const double p = a.hi * b.hi, e = std::fma(a.hi, b.hi, -p);
  return two_sum(p, e + (a.hi * b.lo + a.lo * b.hi));
}
inline Twofold divide(Twofold a, double b) {
  const double q = a.hi / b;
  return two_sum(q, (std::fma(-q, b, a.hi) + a.lo) / b);
}

constexpr Twofold kLn2Twofold{0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56};
constexpr Twofold kTurnTwofold{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)

inline Twofold exp_twofold(Twofold x) {
  const double k = std::nearbyint(x.hi / kLn2Twofold.hi);
  Twofold r = add(x, mul({-k, 0.0}, kLn2Twofold));
  r = {r.hi * 0x1p-9, r.lo * 0x1p-9};  // |r| < 2^-10
  Twofold e{0.0, 0.0};
  for (int n = 10; n >= 1; --n)  // r (1 + r / 2 (1 + r / 3 (...))), cut below 2^-125
    e = divide(mul(r, add({1.0, 0.0}, e)), n);
  for (int i = 0; i < 9; ++i) e = add({2.0 * e.hi, 2.0 * e.lo}, mul(e, e));
  e = add({1.0, 0.0}, e);
  const int n = static_cast<int>(std::fmax(std::fmin(k, 4000.0), -4000.0));
  return {std::ldexp(e.hi, n), std::ldexp(e.lo, n)};
}

// f[i] = base^(-2 i / rope_dims) / (2 pi), i < rope_dims / 2: turns a position.
inline void rope_turns(double base, int rope_dims, double* hi, float* lo) {
  const int half = rope_dims / 2;
  if (half == 0) return;
  int e = 0;
  const double m = std::frexp(base, &e), y = std::log(m);
  // log(base) = e log(2) + y + log(m exp(-y)), the last of them some 2^-53
  const Twofold rest = add(mul({m, 0.0}, exp_twofold({-y, 0.0})), {-1.0, 0.0});
  const Twofold ln = add(mul({static_cast<double>(e), 0.0}, kLn2Twofold), add({y, 0.0}, rest));
  const Twofold step = exp_twofold(divide({-2.0 * ln.hi, -2.0 * ln.lo}, rope_dims));
  Twofold f = kTurnTwofold;
  for (int i = 0; i < half; ++i, f = mul(f, step)) {
    hi[i] = f.hi;
    lo[i] = std::fabs(f.hi) < 0x1p60 ? static_cast<float>(f.lo) : 0.0f;  // (of 2^53 turns hi has no fraction)
  }
}

}  // namespace host
}  // namespace vattn
