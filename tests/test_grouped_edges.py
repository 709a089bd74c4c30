"""Edges of the 8-bit and expert-grouped operators without a GPU."""

from fractions import Fraction

import numpy as np

import oracle


def test_offset_scale_ref_against_fractions():
    rng = np.random.default_rng(1)
    xb = oracle.f32_to_bf16_bits((rng.standard_normal((3, 256)) * 10.0 ** rng.integers(-3, 4, (3, 256))).astype(np.float32))
    d = rng.uniform(-1, 1, (4, 2)).astype(np.float32)
    d16 = oracle.f32_to_bf16_bits(d)
    x = oracle.bf16_bits_to_f64(xb)
    for scales, value in ((d, d.astype(np.float64)), (d16, oracle.bf16_bits_to_f64(d16))):
        got = oracle.offset_scale_ref(xb, scales)
        for m in range(3):
            for n in range(4):
                want = sum(abs(Fraction(x[m, k]) * Fraction(value[n, k // 128])) for k in range(256))
                assert abs(Fraction(got[m, n]) - want) <= want * 258 * Fraction(1, 2 ** 53)
    xb[1, 7] = 0x7F80
    got = oracle.offset_scale_ref(xb, d)
    assert np.isnan(got[1]).all() and not np.isnan(got[[0, 2]]).any()


def test_rounding_of_a_group_formed_with_an_offset():
    """sum q x as 16 ((-1.5 sum x) + sum (1.5 + q / 16) x) in fp32, one addition after the other: its error
    stays within OFFSET_TOL of sum |x|, and passes any share of sum |q x| where the large x have codes 0."""
    rng = np.random.default_rng(2)
    f = np.float32
    worst = worst_q = 0.0
    for trial in range(200):
        x = oracle.bf16_bits_to_f64(oracle.f32_to_bf16_bits(
            (rng.standard_normal(128) * 10.0 ** rng.uniform(0, 6 if trial % 2 else 0.1, 128)).astype(np.float32)))
        q = rng.integers(-8, 8, 128)
        if trial % 4 == 1:
            q[np.abs(x) > np.quantile(np.abs(x), 0.3)] = 0
        start = v = f(0)
        for k in rng.permutation(128):
            start = f(start - f(1.5) * f(x[k]))
        v = start
        for k in rng.permutation(128):
            v = f(v + f(1.5 + q[k] / 16.0) * f(x[k]))
        exact = sum(Fraction(int(a)) * Fraction(b) for a, b in zip(q, x))
        err = float(abs(16 * Fraction(float(v)) - exact))
        worst = max(worst, err / np.abs(x).sum())
        worst_q = max(worst_q, err / (2e-3 * np.abs(q * x).sum() + 1e-6))
    assert worst <= oracle.OFFSET_TOL
    assert worst_q > 1.0  # the term is there for a reason
