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


# ----------------------------------------------------------------------------
# 4-bit products: inputs that dominate a row
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("scale_dtype", [F32, BF16])
@pytest.mark.parametrize("big", [1e3, 1e6, 1e8])
@pytest.mark.parametrize("rows", [1, 4, 16, [5, 0, 3], [40, 20, 36], [200, 0, 150]])
def test_dominant_inputs_at_zero_codes(w4, gpu, rows, big, scale_dtype):
    """Inputs far above the rest of their row that meet codes 0 add nothing to sum |w_hat x|; what they
    leave is within OFFSET_TOL of sum |d x|, in the dense kernels (a number of rows, each path) and in
    the three grouped ones (the experts' rows)."""
    _say(f"dominant inputs {big:g} rows={rows} scales {scale_dtype}")
    N, K = 48, 640
    sizes = rows if isinstance(rows, list) else [rows]
    E, M, off = len(sizes), sum(sizes), _offsets(sizes)
    rng = np.random.default_rng(M)
    W = (rng.standard_normal((E, N, K)) * 0.02).astype(np.float32)
    x = rng.standard_normal((M, K)).astype(np.float32)
    for i, at in enumerate((5, 200, 383, 639)):
        W[:, :, at] = 0.0
        x[:, at] = big * (-1.0) ** i
    xg = torch.from_numpy(x).to(gpu).to(BF16)
    Wg = torch.from_numpy(W).to(gpu)
    q, d = w4.quantize_rtn_experts(Wg, scale_dtype)
    for out_dtype in (F32, BF16):
        if E > 1:
            ys = [w4.grouped_linear(xg, torch.from_numpy(off).to(gpu), q, d, N, out_dtype=out_dtype)]
        else:
            paths = ("gemv", "mfma", "auto") if M <= 4 else ("mfma", "auto")
            ys = [w4.linear(xg, q[0], d[0], N, path=p, out_dtype=out_dtype) for p in paths]
        for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
            if a == b:
                continue
            xb = _bits(xg)[a:b]
            qc, dc = oracle.rtn_quantize_ref(W[e], "bf16" if scale_dtype == BF16 else "f32")
            ref, absdot = oracle.w4_linear_ref(xb, qc, dc)
            abs_ = oracle.ABS_TOL + oracle.OFFSET_TOL * oracle.offset_scale_ref(xb, dc)
            for y in ys:
                ok = oracle.admissible(_bits(y[a:b]), ref, absdot, "f32" if out_dtype == F32 else "bf16", abs_=abs_)
                assert ok.all(), f"expert {e} {out_dtype}: {int((~ok).sum())} of {ok.size} outputs out of tolerance"


# ----------------------------------------------------------------------------
# more rows than one launch takes
# ----------------------------------------------------------------------------

def test_quantize_w8_rows_past_one_launch(w4, gpu):
    """2^25 rows of 128 inputs fill a launch: the rows around its end, and the last ones, bit for bit."""
    N, K = (1 << 25) + 1037, 128
    _say(f"quantize_w8 {N} x {K}")
    W = torch.empty((N, K), device=gpu)
    g = torch.Generator(device=gpu)
    g.manual_seed(5)
    W.normal_(generator=g)
    q, d = w4.quantize_w8(W)
    assert bool(torch.isfinite(d).all()) and bool((d > 0).all())
    for a, b in ((0, 160), ((1 << 25) - 160, (1 << 25) + 160), ((1 << 25) + 1008, N)):  # (a: whole row blocks)
        q_ref, d_ref = oracle.rtn_rows_ref(W[a:b].cpu().numpy())
        assert np.array_equal(d[a:b].cpu().numpy().view(np.uint32), d_ref.view(np.uint32)), "scales differ"
        packed = oracle.pack_w8_ref(q_ref)
        assert np.array_equal(q[a * K:a * K + packed.size].cpu().numpy(), packed), "codes differ"
    want, most = torch.empty_like(d), torch.full((1,), 127.0, device=gpu)
    for a in range(0, N, 1 << 22):  # every scale
        want[a:a + (1 << 22)] = W[a:a + (1 << 22)].abs().amax(dim=1) / most
    assert torch.equal(d, want)


def test_pack_w8_rows_past_one_launch(w4, gpu):
    """2^30 chunks of 16 codes fill a launch: every code goes there and back, and the layout around the
    launch's end is the oracle's."""
    N, K = (1 << 27) + 1037, 128
    _say(f"pack_w8 {N} x {K}")
    c = torch.empty((N, K), dtype=torch.int8, device=gpu)
    g = torch.Generator(device=gpu)
    g.manual_seed(6)
    for a in range(0, N, 1 << 24):
        c[a:a + (1 << 24)].random_(-128, 128, generator=g)
    q = w4.pack_w8(c)
    for a, b in ((0, 160), ((1 << 27) - 160, (1 << 27) + 160), ((1 << 27) + 1008, N)):
        packed = oracle.pack_w8_ref(c[a:b].cpu().numpy())
        assert np.array_equal(q[a * K:a * K + packed.size].cpu().numpy(), packed), "layout differs"
    back = w4.unpack_w8(q, N, K)
    for a in range(0, N, 1 << 24):
        assert torch.equal(back[a:a + (1 << 24)], c[a:a + (1 << 24)])


def test_grouped_linear_refuses_another_number_of_experts(w4, gpu):
    """Four experts of 512 inputs take as many bytes as two of 1024, which x and the offsets ask for."""
    _say("grouped_linear, four experts for offsets of two")
    _, q, d = _w4_experts(w4, gpu, 61, 4, 32, 512, F32)
    x = workloads.random_activations(6, 1024, seed=61, device=gpu)
    with pytest.raises(ValueError, match="experts"):
        w4.grouped_linear(x, torch.tensor([0, 2, 6], dtype=torch.int32, device=gpu), q, d, 32)


# ----------------------------------------------------------------------------
# scale and output types; rows that do not disturb each other
# ----------------------------------------------------------------------------

def _check_experts(w4, gpu, W, q, d, sizes, first, extra, N, K, scale_dtype, out_dtype, seed):
    off = _offsets(sizes, first)
    M = first + sum(sizes) + extra
    x = workloads.random_activations(M, K, seed=seed, device=gpu)
    y = torch.full((M, N), 7.0, dtype=out_dtype, device=gpu)
    w4.grouped_linear(x, torch.from_numpy(off).to(gpu), q, d, N, out=y)
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if a < b:
            ref, absdot = _w4_ref(W[e].cpu().numpy(), _bits(x)[a:b], scale_dtype)
            check_w4(y[a:b], ref, absdot, f"expert {e}")
    assert bool((y[:first] == 7.0).all()) and bool((y[off[-1]:] == 7.0).all()), "a row of no expert was written"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("si", range(len(SIZES)))
def test_grouped_linear_scales_typed_as_outputs(w4, gpu, si, dtype):
    """bf16 scales with bf16 outputs and fp32 with fp32: streamed, 32-row and 64-row tiles."""
    N, K = [(33, 256), (130, 640), (513, 128)][si % 3]
    _say(f"grouped_linear sizes={SIZES[si][:6]} N={N} K={K} scales and outputs {dtype}")
    W, q, d = _w4_experts(w4, gpu, 70 + si, len(SIZES[si]), N, K, dtype)
    first, extra = (2, 3) if si % 2 else (0, 0)
    _check_experts(w4, gpu, W, q, d, SIZES[si], first, extra, N, K, dtype, dtype, si)


# Streamed with four row blocks per wavefront, 32-row and 64-row tiles of several panels.
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K,sizes", [(2050, 256, [3, 0] * 11 + [7, 8, 1] * 4), (1000, 4224, [40, 8, 0, 33]),
                                       (2304, 1152, [290, 0, 45])])
def test_grouped_linear_larger_scales_typed_as_outputs(w4, gpu, N, K, sizes, dtype):
    _say(f"grouped_linear N={N} K={K} sizes={sizes[:6]} scales and outputs {dtype}")
    W, q, d = _w4_experts(w4, gpu, 90, len(sizes), N, K, dtype)
    _check_experts(w4, gpu, W, q, d, sizes, 0, 0, N, K, dtype, dtype, 90)


@pytest.mark.parametrize("M", [20, 120, 600])
def test_grouped_linear_rows_are_independent(w4, gpu, M):
    """Within calls of one size (M, N and experts choose the kernel) a 4-bit row's bits depend on its own
    values and its own expert alone: not on the other rows' values, nor on how these are routed, nor
    on where in the call the row stands."""
    _say(f"grouped_linear rows beside others, M={M}")
    E, N, K = 4, 200, 1152
    _, q, d = _w4_experts(w4, gpu, 51, E, N, K, BF16)
    rng = np.random.default_rng(M)
    mine = workloads.random_activations(3, K, seed=51, device=gpu)  # rows of expert 2

    def run(before, own, at, seed):
        """before rows of experts 0 and 1, `own` of expert 2 with `mine` from its row `at` on, the rest expert 3's"""
        x = workloads.random_activations(M, K, seed=seed, device=gpu)
        x[before + at:before + at + 3] = mine
        if seed % 2:
            x[before + own - 1] = float("nan")  # the last row of the expert: another tile's or the same one's
        off = torch.tensor([0, int(rng.integers(0, before + 1)), before, before + own, M], dtype=torch.int32, device=gpu)
        return w4.grouped_linear(x, off, q, d, N, out_dtype=F32)[before + at:before + at + 3]

    want = run(0, 4, 0, 2)
    assert bool(torch.isfinite(want).all())
    for before, own, at, seed in ((0, 4, 0, 3), (5, 9, 2, 4), (M // 2, 5, 1, 5), (3, M - 3, M - 10, 7), (M - 6, 6, 2, 8)):
        assert same_bits(run(before, own, at, seed), want)
