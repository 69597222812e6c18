"""Coefficients of the tanh approximation of the capped attention scores (csrc/score_rule.cuh).

tanh(u) = u P(u^2) on |u| <= 1: tanh(u)/u is a smooth function of z = u^2 (its nearest
singularity is z = -(pi/2)^2), so a Chebyshev interpolant in z on [0, 1] converges fast.
Degree 4 leaves a relative error below 7.2e-6, which moves a score capped at 50 by less than
2.8e-4, an eighth of what rounding the weight to bf16 may do (2^-9).  Run: python fit_tanh.py
[degree]  (prints the coefficients of P, lowest degree first, and the error of the fit).
"""
from __future__ import annotations

import numpy as np


def target(z):
    """tanh(sqrt z) / sqrt z in binary64 (its series near 0)."""
    u = np.sqrt(z)
    return np.where(z < 1e-8, 1.0 - z / 3.0, np.tanh(u) / np.where(u > 0, u, 1.0))


def fit(degree: int):
    k = np.arange(degree + 1)
    x = np.cos((2 * k + 1) * np.pi / (2 * (degree + 1)))     # Chebyshev nodes
    cheb = np.polynomial.chebyshev.chebfit(x, target((x + 1) / 2), degree)
    p = np.polynomial.Polynomial(np.polynomial.chebyshev.cheb2poly(cheb))
    return p(np.polynomial.Polynomial([-1.0, 2.0])).coef     # in z, x = 2 z - 1


def max_error(coef, n=20001):
    """Largest relative error on [0, 1]."""
    z = np.linspace(0.0, 1.0, n)
    return float(np.max(np.abs(np.polynomial.polynomial.polyval(z, coef) / target(z) - 1.0)))


if __name__ == "__main__":
    import sys

    degree = int(sys.argv[1]) if len(sys.argv) > 1 else 4
    c = fit(degree)
    print("degree %d: largest relative error %.3g for |u| <= 1" % (degree, max_error(c)))
    for v in c:
        print("    %.9ef," % v)
