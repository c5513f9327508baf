"""The products' activations, emulated in fp32 on the CPU over every fp16
argument: GELU by its fitted tail (csrc/sp24_epilogue.hpp), its slope, and the
forms through 1 / (1 + 2^z), against float64.  The hardware's 2^y and reciprocal
may be off by 1 ulp: both signs are tried."""
import os
import re

import numpy as np
import pytest
from scipy.special import erfc, ndtr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "structured_sparse_transformer_amd", "csrc", "sp24_epilogue.hpp")).read()
F = np.float32


def every_fp16():
    x = np.arange(65536, dtype=np.uint32).astype(np.uint16).view(np.float16).astype(np.float32)
    return x[np.isfinite(x)]


def table():
    text = re.search(r"kTail\[7\] = \{([^}]*)\}", SOURCE).group(1)
    return [F(v.strip().rstrip("f")) for v in text.split(",")]


def fma(a, b, c):
    a, b, c = (np.asarray(v, dtype=np.float64) for v in (a, b, c))
    return (a * b + c).astype(F)   # one rounding, but for 2^-53


def exp2(y, ulps):
    e = np.exp2(y.astype(np.float64)).astype(F)
    return e if ulps == 0 else np.nextafter(e, F(np.inf) if ulps > 0 else F(0))


def tail(a, ulps):
    c = table()
    p = np.full_like(a, c[6])
    for k in range(5, -1, -1):
        p = fma(p, a, c[k])
    return exp2(p, ulps)


@pytest.mark.parametrize("ulps", [-1, 0, 1])
def test_gelu(ulps):
    x = every_fp16()
    a = np.minimum(np.abs(x), F(10))
    got = fma(-a, tail(a, ulps), np.where(x < 0, F(0), x)).astype(np.float64)
    want = x.astype(np.float64) * 0.5 * erfc(-x.astype(np.float64) / np.sqrt(2))
    # 1.4e-6 relative and a Phi(-a) within 4e-9 by the fit, |P| 2^-23 by the exponent's roundings (7 of them)
    far = np.abs(got - want) - 4e-9
    assert (far <= (1.5e-6 + 4e-6) * np.abs(want) + 2.0 ** -24 * np.abs(x)).all()
    # the result rounded to fp16 is off by half a step and a hundredth
    with np.errstate(over="ignore"):
        h = got.astype(np.float16).astype(np.float64)
    fine = np.isfinite(h)
    assert (np.abs(h - want)[fine] <= (2.0 ** -11 * 1.02) * np.abs(want)[fine] + 2.0 ** -25 + 5e-9).all()


@pytest.mark.parametrize("ulps", [-1, 0, 1])
def test_gelu_slope(ulps):
    x = every_fp16()
    a = np.minimum(np.abs(x), F(10))
    pdf = exp2(fma(a * a, F(-0.5) * F(1.44269504), F(-1.32574806)), ulps)
    left = (-a.astype(np.float64) * pdf + tail(a, ulps)).astype(F)
    got = np.where(x < 0, left, F(1) - left).astype(np.float64)
    xd = x.astype(np.float64)
    want = ndtr(xd) + xd * np.exp(-xd * xd / 2) / np.sqrt(2 * np.pi)
    assert np.abs(got - want).max() <= 1.5e-6


def test_limits():
    a = np.array([10.0], dtype=F)
    assert 0 <= tail(a, 0)[0] * 10 < 1e-21       # where it is held
    assert (np.diff(tail(np.linspace(0, 10, 10001).astype(F), 0)) <= 0).all()
    assert abs(float(tail(np.zeros(1, F), 0)[0]) - 0.5) < 1e-6


def test_the_constants():
    number = lambda name: float(re.search(name + r" = (-?[0-9.e+-]+)f", SOURCE).group(1))  # noqa: E731
    assert abs(number("kLog2") - np.log2(np.e)) < 1e-7 and abs(number("kLog2InvSqrt2Pi") - np.log2(1 / np.sqrt(2 * np.pi))) < 1e-7
    assert abs(number("kTanhK") - 2 * np.sqrt(2 / np.pi)) < 1e-7 and abs(number("kTanhC") - 0.044715) < 1e-9
