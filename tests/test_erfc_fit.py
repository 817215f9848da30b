"""The fit of erfc that the layer's GELU uses, evaluated on the CPU in fp32, one
rounding an operation, against math.erfc: its coefficients are read from the source.

t = 1 / (1 + a / 2), erfc(a) = t exp(-a^2 + P(t)).  The bound is the source's, (2 + 1.4 a^2)
2^-22: the fit itself 4.1e-7 = 1.7 2^-22 near 0, falling with a; the argument -a^2 + P
rounded at 2^-24 of at most a^2 + 1.3, its error that of the exponential; the rest of
it is the fast exponential's, 0.58 a^2 2^-22, which is exact here.
"""
import math
import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_quantized_02_b200",
                      "csrc", "wq_epilogue.cuh")


def coefficients():
    text = open(SOURCE).read()
    body = text[text.index("float epi_erfc(float a)"):]
    body = body[:body.index("return")]
    first = re.search(r"float p = (-?[0-9.]+)f;", body).group(1)
    rest = re.findall(r"p = fmaf\(p, t, (-?[0-9.]+)f\);", body)
    return [np.float32(c) for c in [first] + rest]


def fma32(a, b, c):
    """Products of two fp32 numbers are exact in binary64; the sum's second rounding is
    far below fp32's."""
    return np.float32(np.float64(a) * np.float64(b) + np.float64(c))


def erfc32(a, coef):
    t = np.float32(1.0) / fma32(np.float32(0.5), a, np.float32(1.0))
    p = np.full_like(a, coef[0])
    for c in coef[1:]:
        p = fma32(p, t, c)
    return np.float64(t) * np.exp(np.float64(fma32(-a, a, p)))


@pytest.mark.parametrize("lo,hi", [(0.0, 0.1), (0.1, 1.0), (1.0, 3.0), (3.0, 6.0), (6.0, 9.0)])
def test_relative_error(lo, hi):
    coef = coefficients()
    assert len(coef) == 10
    a = np.linspace(lo, hi, 20001).astype(np.float32)
    ref = np.array([math.erfc(float(v)) for v in a])
    err = np.abs(erfc32(a, coef) - ref) / ref
    assert (err <= (2 + 1.4 * np.float64(a) ** 2) * 2.0 ** -22).all(), float(err.max())
    assert err.max() <= 1e-5  # at 9, where the argument is 81
