"""8-bit codes with one scale per row, and their product (oracle).

The quantizer is the group-quantization equation of the Qwen3.5-4B quantization
study, section 1 (z = 0), with a whole row as the group and 127 as the largest
code.  Readings as for the 4-bit codes: d = fl32(max|w| / 127); the code is
fl32(w / d) rounded to the nearest integer, ties away from zero, clamped to
[-127, 127]; a row holding a NaN or an infinity gets d = NaN (0x7FC00000) and
codes 0; d == 0 gives codes 0.  The same rule serves weights (a scale per
output channel) and activations (a scale per token).

The product sx[m] d[n] sum_k xq[m,k] q[n,k] is evaluated in integers and
float64: the integer sum is exact, and the scales are widened.
"""

import numpy as np

from .rtn import NAN_BITS, _round_half_away

QMAX8 = 127
# The kernel rounds the exact sum to fp32 and multiplies by two fp32 scales:
# three roundings of at most 2^-24 each; (1 + 2^-24)^3 - 1 < 3.000001 * 2^-24.
W8A8_REL = 3.000001 * 2.0 ** -24


def rtn_rows_ref(W):
    """W: float32 [N, K] -> (q int8 [N, K], d float32 [N])."""
    W = np.asarray(W)
    if W.dtype != np.float32 or W.ndim != 2:
        raise TypeError("W must be a 2-D float32 array")
    finite = np.isfinite(W).all(axis=1)
    with np.errstate(all="ignore"):
        d = (np.abs(W).max(axis=1) / np.float32(QMAX8)).astype(np.float32)
    d[~finite] = np.array([NAN_BITS], dtype=np.uint32).view(np.float32)[0]
    usable = finite & (d != 0)
    safe = np.where(usable, d, np.float32(1.0)).astype(np.float32)
    with np.errstate(all="ignore"):
        t = (W / safe[:, None]).astype(np.float32)
    q = np.clip(_round_half_away(t), -QMAX8, QMAX8)
    q[~usable] = 0
    return q.astype(np.int8), d


def w8a8_linear_ref(xq, sx, q, d):
    """sx[m] d[n] sum_k xq[m,k] q[n,k] in float64, [M, N] (NaN where a scale is NaN)."""
    # float64 holds every partial sum exactly (below 2^53)
    s = np.asarray(xq).astype(np.float64) @ np.asarray(q).astype(np.float64).T
    return s * np.asarray(sx).astype(np.float64)[:, None] * np.asarray(d).astype(np.float64)[None, :]


def pack_w8_ref(q):
    """int8 [N, K] -> native tiles, byte by byte from the layout's definition."""
    q = np.asarray(q)
    N, K = q.shape
    out = np.zeros(((N + 15) // 16) * 16 * K, np.int8)
    n, k = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    at = ((n // 16) * (K // 64) + k // 64) * 1024 + ((k // 16) % 4 * 16 + n % 16) * 16 + k % 16
    out[at.ravel()] = q.ravel()
    return out
