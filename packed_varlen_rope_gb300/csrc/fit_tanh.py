"""Coefficients of the tanh approximations of the capped attention scores (csrc/score_rule.cuh).

tanh(u) = u P(u^2), odd polynomials that interpolate it at Chebyshev nodes (its nearest singularity
is i pi/2, so they converge fast):

* near: degree 7 on |u| <= 0.8, interpolating tanh itself: absolute error below 6.7e-6, which moves a
  score capped at 50 by less than 3.4e-4, a tenth of what rounding the weight to bf16 may do (2^-8);
* small: degree 5 on |u| <= 0.5, the same way: below 5.6e-6;
* large: degree 11 on |u| <= 1, interpolating tanh(u)/u in u^2: relative error below 6.1e-7, for caps
  so large that scores far below them have to keep theirs.

Run: python fit_tanh.py  (prints the coefficients of P, lowest degree first, and the errors).
"""
from __future__ import annotations

import numpy as np

NEAR, SMALL = 0.8, 0.5


def near(degree: int = 3, end: float = NEAR):
    """P of the absolute fit, in u^2."""
    n = 2 * degree + 3                                                   # zeros of the next odd term
    k = np.arange(n)
    u = end * np.cos((2 * k + 1) * np.pi / (2 * n))
    odd = np.vander(u * u, degree + 1, increasing=True) * u[:, None]
    return np.linalg.lstsq(odd, np.tanh(u), rcond=None)[0]


def small():
    return near(2, SMALL)


def target(z):
    """tanh(sqrt z) / sqrt z in binary64 (its series near 0)."""
    u = np.sqrt(z)
    return np.where(z < 1e-8, 1.0 - z / 3.0, np.tanh(u) / np.where(u > 0, u, 1.0))


def large(degree: int = 5):
    """P of the relative fit, in z = u^2 on [0, 1]."""
    k = np.arange(degree + 1)
    x = np.cos((2 * k + 1) * np.pi / (2 * (degree + 1)))
    cheb = np.polynomial.chebyshev.chebfit(x, target((x + 1) / 2), degree)
    p = np.polynomial.Polynomial(np.polynomial.chebyshev.cheb2poly(cheb))
    return p(np.polynomial.Polynomial([-1.0, 2.0])).coef                 # x = 2 z - 1


def near_error(coef, n=40001, end: float = NEAR):
    u = np.linspace(0.0, end, n)
    return float(np.max(np.abs(u * np.polynomial.polynomial.polyval(u * u, coef) - np.tanh(u))))


def large_error(coef, n=40001):
    z = np.linspace(0.0, 1.0, n)
    return float(np.max(np.abs(np.polynomial.polynomial.polyval(z, coef) / target(z) - 1.0)))


if __name__ == "__main__":
    for name, c, e in (("near", near(), near_error(near())), ("small", small(), near_error(small(), end=SMALL)),
                       ("large", large(), large_error(large()))):
        print("%s: error %.3g" % (name, e))
        print("    " + ", ".join("%.9ef" % v for v in c))
