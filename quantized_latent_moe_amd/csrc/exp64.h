// exp in 64 bits of the routing by scores: no GPU header, so that it can be
// compiled and compared by itself.
#pragma once

namespace latmoe {

// exp(x), |x| <= 700, within 5e-16 of itself (2^-50.8): x = n ln 2 + r, and the
// polynomial of degree 10 through exp at the Chebyshev points of
// |r| <= ln 2 / 2, which is within 3.3e-16.  ln 2 is in two parts: n times the
// first is subtracted without rounding, and what that lacks of ln 2, 2.3e-17,
// would be n times as much in r (2^-45 at |x| = 700).  Coefficients from the
// highest degree down to 1.
constexpr int kExp64Coefficients = 10;
constexpr double kExp64[kExp64Coefficients] = {
    2.7626357241447223e-07, 2.764018079620985e-06, 2.4801504346997686e-05, 0.00019841170270440067,
    0.0013888888932488599,  0.008333333385667782,  0.04166666666657314,    0.16666666666554406,
    0.5000000000000006,     1.0000000000000067};

// Real is double; constexpr templates are host and device code to a HIP compiler.
template <class Real>
constexpr Real exp64_power(Real x) {
  return __builtin_rint(x * 0x1.71547652b82fep+0);
}
template <class Real>
constexpr Real exp64_rest(Real x, Real n) {
  return __builtin_fma(n, -0x1.abc9e3b39803fp-56, __builtin_fma(n, -0x1.62e42fefa39efp-1, x));
}
// exp(r); exp(x) is 2^n times it.
template <class Real>
constexpr Real exp64_series(const Real* c, Real r) {
  Real p = __builtin_fma(c[0], r, c[1]);
#pragma unroll
  for (int i = 2; i < kExp64Coefficients; ++i) p = __builtin_fma(p, r, c[i]);
  return __builtin_fma(p, r, 1.0);
}

}  // namespace latmoe
