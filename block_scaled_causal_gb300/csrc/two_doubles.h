// Sums of two doubles, hi + lo with |lo| <= ulp(hi) / 2: 106 bits on the host, where 53 are too few.  The error-free sum is Knuth's,
// the error-free product a fused multiply-add's; results are within a few 2^-104 of the terms' magnitudes.
#pragma once
#include <cmath>
#include <cstdint>

namespace bsc {

struct Two {
  double hi, lo;
  Two(double h, double l = 0.0) : hi(h), lo(l) {}
};
inline Two sum_of(double a, double b) {
  const double s = a + b, c = s - a;
  return {s, (a - (s - c)) + (b - c)};
}
inline Two operator+(Two x, Two y) {
  const Two s = sum_of(x.hi, y.hi);
  return sum_of(s.hi, s.lo + (x.lo + y.lo));
}
inline Two operator-(Two x, Two y) { return x + Two(-y.hi, -y.lo); }
inline Two operator*(Two x, Two y) {
  const double p = x.hi * y.hi;
  return sum_of(p, std::fma(x.hi, y.hi, -p) + (x.hi * y.lo + x.lo * y.hi));
}
inline Two operator/(Two x, Two y) {
  const double q = x.hi / y.hi;
  const Two r = x - y * q;
  const double q2 = r.hi / y.hi;
  return sum_of(q, q2) + Two((r - y * q2).hi / y.hi);
}
inline Two power(Two x, int n) {
  Two p(1.0);
  for (; n; n >>= 1, x = x * x)
    if (n & 1) p = p * x;
  return p;
}
// b^(-1/n) for b > 0 and n from 2 to 128: Newton's x += x (1 - b x^n) / n, from 53 bits.  b is brought into [1/2, 2^n) first, by a
// power of 2^n, so that no step leaves the range.
inline Two inverse_root(double b, int n) {
  int e;
  const double m = std::frexp(b, &e);
  const int rest = ((e % n) + n) % n, whole = (e - rest) / n;
  const Two y(std::ldexp(m, rest));
  Two x(std::pow(y.hi, -1.0 / n));
  for (int i = 0; i < 2; ++i) x = x + x * (Two(1.0) - y * power(x, n)) / Two(n);
  return {std::ldexp(x.hi, -whole), std::ldexp(x.lo, -whole)};
}
// The fraction of x in units of 2^-64, modulo 2^64.
inline unsigned long long fraction_64(Two x) {
  Two f = sum_of(x.hi - std::rint(x.hi), x.lo - std::rint(x.lo));
  f = sum_of(f.hi - std::rint(f.hi), f.lo);                     // |f| <= 1/2 and a little
  const double a = std::ldexp(f.hi, 64), whole = std::rint(a), rest = std::rint((a - whole) + std::ldexp(f.lo, 64));
  const uint64_t u = whole >= 0x1p63 ? 1ull << 63 : (uint64_t)(int64_t)whole;
  return u + (uint64_t)(int64_t)rest;
}

}  // namespace bsc
