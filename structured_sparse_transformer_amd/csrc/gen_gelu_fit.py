"""Fit of the polynomial behind the products' GELU (sp24_epilogue.hpp).

The logarithm of the normal distribution's tail, log Phi(-a) for a >= 0, is
smooth and nearly quadratic.  A polynomial of degree 6 is fitted to it on
[0, 6] by least squares, reweighted toward the largest errors (Lawson's
iteration), so that Phi(-a) is off by at most REL relative, or a Phi(-a) by ABS
absolute, whichever is more, times the printed factor.  Prints its coefficients
times log2 e, lowest degree first, as fp32 literals, and the largest a up to
which it falls.

Run: python gen_gelu_fit.py   (needs numpy and scipy)
"""
import numpy as np
from scipy.special import log_ndtr, ndtr

DEGREE, END, REL, ABS = 6, 6.0, 1e-6, 3e-9


def allowed(a):
    return np.maximum(REL, ABS / (a * ndtr(-a) + 1e-300))


def fit(nodes=4000, rounds=500):
    a = (0.5 - 0.5 * np.cos(np.pi * (np.arange(nodes) + 0.5) / nodes)) * END
    V = np.polynomial.chebyshev.chebvander(2 * a / END - 1, DEGREE)
    y, scale, w, best = log_ndtr(-a), 1 / allowed(a), np.ones(nodes), None
    for _ in range(rounds):
        s = np.sqrt(w) * scale
        c, *_ = np.linalg.lstsq(V * s[:, None], y * s, rcond=None)
        err = np.abs((V @ c - y) * scale)
        if best is None or err.max() < best[0]:
            best = err.max(), c
        w = w * (err / err.max()) ** 0.5 + 1e-14
        w /= w.mean()
    p = np.polynomial.polynomial.Polynomial(np.polynomial.chebyshev.cheb2poly(best[1]))
    return p(np.polynomial.polynomial.Polynomial([-1.0, 2.0 / END])).coef


if __name__ == "__main__":
    c32 = (fit() * np.log2(np.e)).astype(np.float32)
    p = lambda a: np.polynomial.polynomial.polyval(a, c32.astype(np.float64)) * np.log(2.0)  # noqa: E731
    a = np.linspace(0.0, END, 200001)
    far = np.abs(p(a) - log_ndtr(-a)) / allowed(a)
    big = np.linspace(0.0, 20.0, 20001)
    falls = big[np.argmax(np.diff(p(big)) >= 0)]
    print(", ".join(np.format_float_scientific(v, unique=True) + "f" for v in c32))
    print(f"largest error over what is allowed, with fp32 coefficients: {far.max():.2f}; falls up to {falls:.2f}, to e^{p(falls):.1f}")
