"""Microscaled 4-bit floating point (MXFP4) and its product (oracle).

The format is that of the OCP Microscaling Formats specification, v1.0: blocks of
32 consecutive inputs, E2M1 elements and one E8M0 scale per block.  Readings:

* the scale is 2^(floor(log2 max|v|) - 2), the exponent of E2M1's largest power of
  two being 2, and at least 2^-127; a block of zeros has the byte 0;
* an element is the E2M1 nearest to v / scale, ties to the even code, magnitudes
  above 6 becoming 6; the sign of a zero is kept;
* a NaN or an infinity in a block gives the scale byte 255 (NaN) and codes 0.

Evaluated in float64, where v / scale (a power of two) is exact.
"""

import numpy as np

MX_BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# Each 128 products that the matrix unit adds to a sum cost at most 2^-22 of the sum of their
# magnitudes and the sum's; so does each sum of a part of K (at most 8 parts).  Products and
# sums below 2^-126 may be lost: 2^-120 per input covers 64 such losses.
MX4_STEP, MX4_LOST = 2.0 ** -22, 2.0 ** -120


def mx4_tolerance(absdot, K):
    """How far an fp32 accumulation may be from the exact product, given sum_k |x^ w^|."""
    return (K // 128 + 8) * MX4_STEP * absdot + K * MX4_LOST


def mx4_quantize_ref(v):
    """v: [rows, K] float32 (or float64 holding bf16/fp32 values) -> codes uint8 [rows, K] (0 .. 15), scales
    uint8 [rows, K / 32]."""
    v = np.asarray(v).astype(np.float64)
    rows, K = v.shape
    b = v.reshape(rows, K // MX_BLOCK, MX_BLOCK)
    finite = np.isfinite(b).all(axis=2)
    b = np.where(finite[..., None], b, 0.0)
    top = np.abs(b).max(axis=2)
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1 - 2, -127)
    e = np.maximum(e, -127)
    a = np.ldexp(np.abs(b), -e[..., None])
    # the nearest code: the first that is not below a, or the one before it
    hi = np.minimum(np.searchsorted(E2M1, a), 7)
    lo = np.maximum(hi - 1, 0)
    down, up = a - E2M1[lo], E2M1[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 6.0, 7, code)
    code = code + 8 * np.signbit(b)
    code = np.where(finite[..., None], code, 0)
    scale = np.where(finite, e + 127, 255)
    return code.astype(np.uint8).reshape(rows, K), scale.astype(np.uint8)


def mx4_values_ref(codes, scales):
    """float64 values of codes [rows, K] under scales [rows, K / 32] (NaN for a scale of 255)."""
    c = np.asarray(codes).astype(np.int64)
    m = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.asarray(scales).astype(np.int64)
    d = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return m * np.repeat(d, MX_BLOCK, axis=1)


def mx4_bytes_ref(codes):
    """Codes [rows, K] -> two per byte, the even input in the low four bits."""
    c = np.asarray(codes)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def mx4_linear_ref(xc, xs, wc, ws):
    """(y, sum_k |x^ w^|) in float64, [M, N]; NaN in rows of x and w that hold a NaN scale."""
    x, w = mx4_values_ref(xc, xs), mx4_values_ref(wc, ws)
    bad = np.isnan(x).any(axis=1)[:, None] | np.isnan(w).any(axis=1)[None, :]
    x, w = np.nan_to_num(x, nan=0.0), np.nan_to_num(w, nan=0.0)
    y, a = x @ w.T, np.abs(x) @ np.abs(w).T
    y[bad] = np.nan
    a[bad] = np.nan
    return y, a


def pack_mx4_ref(codes, scales):
    """Codes [N, K] and scales [N, K / 32] -> native (q, s) byte by byte from the layout's definition."""
    b = mx4_bytes_ref(codes)
    N, K = b.shape[0], 2 * b.shape[1]
    P, C, R = -(-K // 256), -(-K // 512), -(-N // 16)
    q = np.zeros(R * P * 2048, np.uint8)
    n, j = np.meshgrid(np.arange(N), np.arange(K // 2), indexing="ij")
    k = 2 * j
    lane = n % 16 + 16 * (k % 256 // 64)
    q[(((n // 16) * P + k // 256) * 2 + k % 64 // 32) * 1024 + 16 * lane + k % 32 // 2] = b
    s = np.zeros(R * C * 256, np.uint8)
    n, j = np.meshgrid(np.arange(N), np.arange(K // 32), indexing="ij")
    k = 32 * j
    lane = n % 16 + 16 * (k % 256 // 64)
    s[((n // 16) * C + k // 512) * 256 + 4 * lane + 2 * (k % 512 // 256) + k % 64 // 32] = scales
    return q, s
