"""Edges of the 8-bit and expert-grouped operators without a GPU."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_ARG = range(6)


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


def test_calls_of_too_many_threads_are_refused(w4):
    """A grid of 2^32 threads or more cannot be launched: refused as a shape before anything else is looked
    at, and never while (M / 16 + min(experts, M)) * (N + 63) < 2^30."""
    lib = w4.library()
    names = ("w4_linear_grouped", "w4_linear_grouped_f32_s16", "w4_linear_grouped_w8a8", "w4_linear_grouped_w8a8_f32")

    def call(name, M, N, E):
        x, off, K = 0x10000000, 0x20000000, 128
        args = [x, x, M, K, off, E] if "w8a8" in name else [x, M, K, off, E]
        return getattr(lib, name)(*args, None, x, N, x, None)  # no codes: an error of its own once the shape is taken

    for name in names:
        # 6144 (8-bit: 5632) row tiles of 16 rows
        w8 = "w8a8" in name
        M, E = (24576, 4096) if w8 else (32768, 4096)
        per = 4 if w8 else 2  # threads per row tile and output
        tiles = M // 16 + E
        N = (1 << 32) // (per * tiles) // 64 * 64
        assert call(name, M, N + 128, E) == ERR_SHAPE
        assert call(name, M, N - 128, E) == ERR_NULL
    rng = np.random.default_rng(5)
    for _ in range(3000):
        M, E = int(2 ** rng.uniform(0, 18)), int(2 ** rng.uniform(0, 12))
        most = min(((1 << 30) - 1) // (M // 16 + min(E, M)) - 63, (1 << 23) - 16)
        N = int(most * rng.choice([1.0, rng.uniform(0, 1)]))
        if N > 0:
            assert call(names[_ % 4], M, N, E) == ERR_NULL, (M, N, E)
    for _ in range(3000):  # dense 8-bit products: up to 400 GB of y
        M = int(2 ** rng.uniform(0, 18))
        N = min(int(2e11 / M), (1 << 24) - 16)
        assert lib.w4_linear_w8a8(0x10000000, 0x10000000, M, 128, None, 0x10000000, N, 0x10000000, None) == ERR_NULL, (M, N)


@pytest.mark.parametrize("shape", [(1, 16, 128), (3, 16, 128), (128,)])
def test_w8linear_takes_one_matrix(w4, shape):
    with pytest.raises(TypeError, match="2-D"):
        w4.W8Linear.from_float(torch.zeros(shape))
