"""What the integer kernels' guard accepts of sums that an epilogue multiplies or
that go out in fp32, on the CPU, from the contract in include/wq.h: a token row is
held in integers of 22 bits below its largest, R is the sum of what that rounds
off in units of 2^-21 of the largest's power of two, and a sum is accepted where

    2^-e R max|w| <= rel |v|   (rel = 2^-9 with mul, 2^-21 in fp32), or
    R <= max(4, K / 1024).

Checked: no ordinary row reaches the second limit (so that no output of it is
formed again), rows with an outlier of 2^10 do, and what is accepted is within the
stated error.
"""
import numpy as np
import pytest

import oracle
import wq_inputs as gen
from wqtest_helpers import i8_fixed_point


def rounded(x_bits):
    xq, e = i8_fixed_point(x_bits, with_exponents=True)
    x = oracle.bf16_to_f64(x_bits)
    return x, xq, np.abs(np.ldexp(x - xq, e[:, None])).sum(1), e


def few(K):
    return max(4, K // 1024)


@pytest.mark.parametrize("K", [256, 1024, 5120, 17408, 65536])
def test_ordinary_rows_are_accepted_whole(K):
    _, _, R, _ = rounded(gen.x_bf16(32, K))
    assert R.max() <= few(K)


@pytest.mark.parametrize("K,outlier,whole", [(5120, 5, True), (5120, 10, False), (17408, 5, True), (17408, 9, False)])
def test_rows_with_an_outlier(K, outlier, whole):
    x = oracle.bf16_to_f64(gen.x_bf16(4, K)).astype(np.float32)
    x[:, 7] = 2.0 ** outlier
    _, _, R, _ = rounded(gen.f32_to_bf16_bits(x))
    assert (R <= few(K)).all() if whole else (R > few(K)).all()


@pytest.mark.parametrize("rel", [2.0 ** -9, 2.0 ** -21])
@pytest.mark.parametrize("outlier", [None, 4, 8, 10, 13])
def test_accepted_sums_are_within_the_stated_error(outlier, rel):
    K, N = 2048, 512
    rng = np.random.default_rng(5)
    q = rng.integers(-127, 128, (N, K)).astype(np.float64)
    q[:, 7] = 0
    s = rng.uniform(0.5, 1.5, N) / (73 * np.sqrt(K))
    w, wmax = q * s[:, None], 128 * s
    xf = oracle.bf16_to_f64(gen.x_bf16(4, K)).astype(np.float32)
    if outlier is not None:
        xf[:, 7] = 2.0 ** outlier
    x, xq, R, e = rounded(gen.f32_to_bf16_bits(xf))
    v, fixed = x @ w.T, xq @ w.T
    bound = np.where(R <= few(K), 0.0, np.ldexp(R, -e))[:, None] * wmax
    taken = bound <= rel * np.abs(fixed)
    stated = np.maximum(rel * np.abs(fixed), few(K) * 2.0 ** -21 * np.abs(x).max(1)[:, None] * wmax)
    assert (np.abs(fixed - v)[taken] <= stated[taken]).all()
    if outlier in (None, 4):
        assert taken.all()
    if outlier == 13 and rel < 2.0 ** -20:
        assert not taken.any()
