// rope_table.cuh -- rotary frequencies as 64-bit fractions of a turn (host).
//
// Positions reach 2^31, so a turn fraction has to be right to 2^-65, which a double
// (2^-56 at a sixth of a turn) is not: angles would be off by 2^-25 turns there.  The
// frequencies are formed in pairs of doubles (about 106 bits; sums by Knuth's and
// products by Dekker's exact transformation, the latter with fma), from powers that
// need no logarithm:
//   theta^(-2 i / rot) = q^i,  q = theta^(-1 / (rot / 2)), a root, by Newton steps;
//   the changed base theta * factor^(rot / (rot - 2)) has the root
//   theta^(-1 / n) * factor^(-1 / (n - 1)), n = rot / 2.
// The same on every machine: no long double, and no product and sum that a compiler may fuse.
#pragma once

#include <cmath>
#include <cstdint>

#include "../../include/csa2.h"

namespace csa2 {

constexpr int kMaxRot = 256;
constexpr int kMaxPairs = kMaxRot / 2;

// By value into the kernels (constant bank): the turn fraction of every pair.
struct RopeTable {
  uint64_t turn[kMaxPairs];    // f_i / (2 pi) * 2^64, to the nearest
  float mscale;                // multiplies cosine and sine
  int pairs;
};

struct Wide {
  double hi, lo;
};
inline Wide wide_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
inline Wide wide_product(double a, double b) {
  const double p = a * b;
  return {p, std::fma(a, b, -p)};
}
inline Wide operator+(Wide a, Wide b) {
  const Wide s = wide_sum(a.hi, b.hi), t = wide_sum(a.lo, b.lo), u = wide_sum(s.hi, s.lo + t.hi);
  return wide_sum(u.hi, u.lo + t.lo);
}
inline Wide operator-(Wide a) { return {-a.hi, -a.lo}; }
inline Wide operator*(Wide a, Wide b) {
  const Wide p = wide_product(a.hi, b.hi);
  return wide_sum(p.hi, std::fma(a.hi, b.lo, std::fma(a.lo, b.hi, p.lo)));
}
inline Wide operator/(Wide a, Wide b) {
  // two quotients, each of what the ones before leave
  const double q0 = a.hi / b.hi;
  const Wide r0 = a + -(b * Wide{q0, 0.0});
  const double q1 = r0.hi / b.hi;
  const Wide r1 = r0 + -(b * Wide{q1, 0.0});
  return wide_sum(q0, q1) + Wide{r1.hi / b.hi, 0.0};
}

// x^(-1 / n) for x >= 1, n >= 1.
inline Wide wide_root(double x, int n) {
  // x = 2^(k n) v with v in [1, 2^n): no power below leaves the range of doubles
  const int k = std::ilogb(x) / n;
  const double v = std::ldexp(x, -k * n);
  Wide y = {std::pow(v, -1.0 / n), 0.0};
  for (int step = 0; step < 2; ++step) {               // errors 2^-50, then 2^-94 or less
    Wide p = {1.0, 0.0}, square = y;
    for (int e = n; e > 0; e >>= 1) {
      if (e & 1) p = p * square;
      square = square * square;
    }
    const Wide rest = Wide{1.0, 0.0} + -(p * Wide{v, 0.0});
    y = y + y * rest / Wide{double(n), 0.0};
  }
  return {std::ldexp(y.hi, -k), std::ldexp(y.lo, -k)};
}

// The frequencies of `r`.  The caller has checked `r`.
inline RopeTable make_rope_table(const csa2_rope& r) {
  constexpr Wide kPerTwoPi = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};
  const Wide one = {1.0, 0.0};
  RopeTable t;
  t.mscale = r.mscale;
  t.pairs = r.rot / 2;
  Wide q = wide_root(r.theta, t.pairs);
  if (r.scaling == CSA2_ROPE_BASE && r.rot > 2) q = q * wide_root(r.factor, t.pairs - 1);
  Wide power = one;
  for (int i = 0; i < t.pairs; ++i) {
    Wide f = power;
    power = power * q;
    if (r.scaling == CSA2_ROPE_LINEAR) f = f / Wide{r.factor, 0.0};
    if (r.scaling == CSA2_ROPE_PARTS) {
      // turns the pair makes over the original context: above turns_hi the
      // frequency stays, below turns_lo it is divided, linear between
      const Wide turns = f * kPerTwoPi * Wide{r.orig_ctx, 0.0};
      const Wide ramp = wide_sum(r.turns_hi, -r.turns_lo), into = turns + Wide{-r.turns_lo, 0.0};
      Wide keep = {0.0, 0.0};
      if (into.hi >= ramp.hi) keep = one;              // or within 2^-52 of the end: as good
      else if (into.hi > 0.0) keep = into / ramp;
      f = f * keep + f / Wide{r.factor, 0.0} * (one + -keep);
    }
    // f <= 1: below a sixth of a turn; the two parts as integers
    const Wide turn = f * kPerTwoPi;
    const double hi = std::ldexp(turn.hi, 64), whole = std::floor(hi);
    t.turn[i] = uint64_t(whole) + uint64_t(int64_t(std::floor((hi - whole) + std::ldexp(turn.lo, 64) + 0.5)));
  }
  return t;
}

}  // namespace csa2
