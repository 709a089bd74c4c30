"""Edges of the expert-grouped operators on an MI355X: routing that leaves most rows to few
experts, every pair of scale and output type, rows that do not disturb each other, inputs that
dominate a row where the weight's code is 0, and launches of more threads than one grid takes.
"""

import numpy as np
import pytest
import torch

import oracle
import workloads
from tests.test_gpu_int8_grouped import (BF16, F32, SIZES, _bits, _codes, _dev, _int8_experts, _offsets, _say, _w4_experts,
                                         _w4_ref, _w8a8_exact, check_w4, check_w8a8, same_bits)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------
# 8-bit experts with uneven routing
# ----------------------------------------------------------------------------

# More than 64 MiB of codes and at most 12 rows per expert on average: experts with one tile of 16
# rows and experts with several read their weights by different loads in one launch.
@pytest.mark.parametrize("N,K,sizes", [
    (5120, 2560, [70, 1, 3, 0, 2, 1, 16, 3]), (5120, 2560, [0, 0, 96, 0, 0, 0, 0, 0]), (5120, 2560, [12] * 8),
    (5121, 2688, [17, 15, 0, 33, 0, 1, 0, 0]), (250, 4096, [0] * 40 + [17, 3] + [0] * 38), (3000, 896, [0] * 62 + [2, 1])])
def test_grouped_w8a8_few_rows_uneven(w4, gpu, N, K, sizes):
    _say(f"grouped_linear_w8a8 uneven N={N} K={K} sizes={sizes[:8]}")
    E, off = len(sizes), _offsets(sizes)
    M = int(off[-1])
    assert E * N * K >= 64 << 20 and M <= 12 * min(E, M)
    rng = np.random.default_rng(N + M)
    xq, sx = _codes(rng, M, K), rng.uniform(1e-3, 0.1, M).astype(np.float32)
    q, d = _int8_experts(K + M, E, N, K)
    txq, tsx, td, toff = _dev(gpu, xq, sx, d, off)
    tc = torch.from_numpy(q).to(gpu)
    tq = torch.stack([w4.pack_w8(tc[e]) for e in range(E)])
    for out_dtype in (BF16, F32):
        y = w4.grouped_linear_w8a8(txq, tsx, toff, tq, td, N, out_dtype=out_dtype)
        for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
            if a < b:
                check_w8a8(y[a:b], _w8a8_exact(txq[a:b], tsx[a:b], tc[e], td[e]), f"expert {e}")
                dense = w4.linear_w8a8(txq[a:b], tsx[a:b].clone(), tq[e], td[e].clone(), N, out_dtype=out_dtype)
                assert same_bits(dense, y[a:b])
