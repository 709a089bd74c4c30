"""8-bit and expert-grouped operators on an MI355X, against the oracle.

Codes, scales and layouts are compared bit for bit.  The int8 product's sum is
exact, so its fp32 value v lies within W8A8_REL = 3 * 2^-24 (three fp32
roundings) of the exact y, relative, and a bf16 output is the nearest-even bf16
of such a v.  Grouped 4-bit outputs obey the dense linear's convention:
|v - y| <= 2e-3 * sum |w_hat x| + 1e-6.
"""

import numpy as np
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(f"\n[case] {msg}", flush=True)


def _bits(y):
    y = y.detach().cpu()
    return y.numpy().view(np.uint32) if y.dtype == F32 else y.view(torch.int16).numpy().view(np.uint16)


def _fmt(y):
    return "f32" if y.dtype == F32 else "bf16"


def check_w8a8(y, ref, what):
    ok = oracle.admissible(_bits(y), ref, np.abs(ref), _fmt(y), rel=oracle.W8A8_REL, abs_=0.0)
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} outputs differ"


def check_w4(y, ref, absdot, what):
    ok = oracle.admissible(_bits(y), ref, absdot, _fmt(y))
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} outputs out of tolerance"


def same_bits(a, b):
    return a.shape == b.shape and np.array_equal(_bits(a), _bits(b))


def _codes(rng, rows, K):
    return rng.integers(-127, 128, (rows, K)).astype(np.int8)


def _offsets(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


# ----------------------------------------------------------------------------
# quantizers and layout: bit-exact
# ----------------------------------------------------------------------------

def special_rows(rng, N, K, dtype=np.float32):
    """Normal rows with hard ones among them: zeros, NaN, infinity, subnormals, huge values, one
    large member, and quotients on and next to half-integers."""
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    for n in range(N):
        kind = n % 11
        if kind == 1:
            W[n] = 0.0
        elif kind == 2:
            W[n, K - 1] = np.nan
        elif kind == 3:
            W[n, 0] = -np.inf
        elif kind == 4:
            W[n] *= np.float32(2.0 ** -140)
        elif kind == 5:
            W[n] *= np.float32(2.0 ** 120)
        elif kind == 6:
            W[n, K // 2] = 30.0
        elif kind in (7, 8):
            # members a few ulps from (k + 1/2) d
            a = np.float32(rng.uniform(0.5, 300.0))
            d = np.float32(a / np.float32(127.0))
            t = (rng.integers(-126, 126, K) + 0.5) * np.float64(d)
            w = t.astype(np.float32)
            W[n] = (w.view(np.int32) + rng.integers(-2, 3, K).astype(np.int32)).view(np.float32)
            W[n, rng.integers(0, K)] = a
        elif kind == 9:
            W[n] = np.float32(190 * 2.0 ** -149) * rng.choice([-1.0, 1.0, 0.0], K).astype(np.float32)
    return W


@pytest.mark.parametrize("N,K", [(1, 128), (11, 128), (16, 256), (37, 384), (100, 1152), (33, 2560), (64, 9216),
                                 (45, 28672), (18, 65536), (13, 130944)])
def test_quantize_w8(w4, gpu, N, K):
    _say(f"quantize_w8 {N}x{K}")
    W = special_rows(np.random.default_rng(N * 7 + K), N, K)
    q_ref, d_ref = oracle.rtn_rows_ref(W)
    nb = w4.packed_bytes_w8(N, K)
    qbuf = torch.full((nb + 64,), 99, dtype=torch.int8, device=gpu)
    dbuf = torch.full((N + 8,), -5.0, device=gpu)
    q, d = w4.quantize_w8(torch.from_numpy(W).to(gpu), out=(qbuf[16:16 + nb], dbuf[4:4 + N]))
    assert np.array_equal(d.cpu().numpy().view(np.uint32), d_ref.view(np.uint32)), "scales differ"
    assert np.array_equal(q.cpu().numpy(), oracle.pack_w8_ref(q_ref)), "codes differ"
    assert bool((qbuf[:16] == 99).all()) and bool((qbuf[16 + nb:] == 99).all()), "bytes around the codes were written"
    assert bool((dbuf[:4] == -5.0).all()) and bool((dbuf[4 + N:] == -5.0).all())
    assert np.array_equal(w4.unpack_w8(q.clone(), N, K).cpu().numpy(), q_ref)


def test_quantize_w8_experts_is_each_matrix(w4, gpu):
    _say("quantize_w8 of a stack of experts")
    W = torch.from_numpy(special_rows(np.random.default_rng(8), 3 * 21, 256).reshape(3, 21, 256)).to(gpu)
    q, d = w4.quantize_w8(W)
    for e in range(3):
        qe, de = w4.quantize_w8(W[e])
        assert torch.equal(q[e], qe) and same_bits(d[e], de)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K", [(1, 128), (1, 5120), (2, 28672), (15, 256), (22, 1152), (33, 9216), (300, 2560),
                                 (12, 65536), (11, 130944)])
def test_quantize_tokens(w4, gpu, M, K, dtype):
    _say(f"quantize_tokens {M}x{K} {dtype}")
    x = torch.from_numpy(special_rows(np.random.default_rng(M + 3 * K), M, K)).to(dtype)
    q_ref, d_ref = oracle.rtn_rows_ref(x.float().numpy())
    buf = torch.full((M + 2, K), 99, dtype=torch.int8, device=gpu)
    sbuf = torch.full((M + 8,), -5.0, device=gpu)
    q, s = w4.quantize_tokens(x.to(gpu), out=(buf[1:1 + M], sbuf[4:4 + M]))
    assert np.array_equal(s.cpu().numpy().view(np.uint32), d_ref.view(np.uint32)), "scales differ"
    assert np.array_equal(q.cpu().numpy(), q_ref), "codes differ"
    assert bool((buf[0] == 99).all()) and bool((buf[1 + M:] == 99).all())
    assert bool((sbuf[:4] == -5.0).all()) and bool((sbuf[4 + M:] == -5.0).all())


def test_quantize_tokens_many_rows(w4, gpu):
    """More rows than any launch has blocks resident, every code checked on the GPU."""
    _say("quantize_tokens 70001 x 128")
    g = torch.Generator(device=gpu)
    g.manual_seed(3)
    x = torch.randn((70001, 128), generator=g, device=gpu).to(BF16)
    q, s = w4.quantize_tokens(x)
    q_ref, d_ref = oracle.rtn_rows_ref(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), q_ref)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), d_ref.view(np.uint32))


@pytest.mark.parametrize("N,K", [(1, 128), (16, 128), (37, 384), (257, 2560)])
def test_pack_w8_round_trip(w4, gpu, N, K):
    _say(f"pack_w8 {N}x{K}")
    c = np.random.default_rng(N).integers(-128, 128, (N, K)).astype(np.int8)
    q = w4.pack_w8(torch.from_numpy(c).to(gpu))
    assert np.array_equal(q.cpu().numpy(), oracle.pack_w8_ref(c))
    assert np.array_equal(w4.unpack_w8(q, N, K).cpu().numpy(), c)


# ----------------------------------------------------------------------------
# int8 product
# ----------------------------------------------------------------------------

def _w8a8_inputs(seed, M, N, K):
    rng = np.random.default_rng(seed)
    xq, q = _codes(rng, M, K), _codes(rng, N, K)
    sx = rng.uniform(1e-3, 0.1, M).astype(np.float32)
    d = rng.uniform(1e-4, 1e-2, N).astype(np.float32)
    return xq, sx, q, d


def _dev(gpu, *arrays):
    return [torch.from_numpy(a).to(gpu) for a in arrays]


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 128), (1, 16, 128), (1, 2560, 2560), (1, 9216, 2560), (2, 17, 256), (7, 1000, 1152), (13, 2561, 4096),
    (16, 64, 28672), (17, 37, 384), (31, 512, 640), (32, 257, 1408), (33, 300, 128), (63, 129, 256), (64, 640, 2560),
    (65, 1024, 896), (96, 255, 5120), (127, 130, 384), (129, 513, 128), (200, 1000, 1024), (256, 256, 256),
    (257, 769, 640), (333, 2561, 1152), (511, 31, 128), (1025, 300, 256), (2049, 513, 384)])
def test_linear_w8a8(w4, gpu, M, N, K, out_dtype):
    _say(f"linear_w8a8 M={M} N={N} K={K} {out_dtype}")
    xq, sx, q, d = _w8a8_inputs(M * 31 + N * 7 + K, M, N, K)
    txq, tsx, tc, td = _dev(gpu, xq, sx, q, d)
    tq = w4.pack_w8(tc)
    buf = torch.full((M + 2, N), 7.0, dtype=out_dtype, device=gpu)
    y = w4.linear_w8a8(txq, tsx, tq, td, N, out=buf[1:1 + M])
    check_w8a8(y, oracle.w8a8_linear_ref(xq, sx, q, d), "linear_w8a8")
    assert bool((buf[0] == 7.0).all()) and bool((buf[1 + M:] == 7.0).all()), "rows around y were written"
    assert same_bits(w4.linear_w8a8(txq, tsx, tq, td, N, out_dtype=out_dtype), y)


def _w8a8_exact(xq, sx, c, d):
    """The definition in 64 bits, on the GPU: sums of products below 2^53 are exact there."""
    return ((xq.double() @ c.double().T.contiguous()) * sx.double()[:, None] * d.double()[None, :]).cpu().numpy()


# At these sizes every kernel that the choice by estimated cost can take is taken, with its steps
# along K an odd number, an even one, fewer than the ring of buffers, and with ragged tiles.
@pytest.mark.parametrize("M,N,K", [
    (9, 5000, 1152), (16, 9216, 2560), (13, 6000, 11264), (5, 9216, 9216), (3, 4090, 128),
    (17, 9216, 640), (25, 17408, 128), (40, 9216, 640), (33, 9200, 128), (64, 9216, 1408), (200, 2561, 896),
    (65, 17400, 384), (130, 9216, 128), (300, 5000, 1152), (200, 9216, 1152), (1025, 2561, 128), (300, 9201, 640),
    (400, 17408, 256), (1025, 5000, 640), (2049, 2561, 384), (2048, 9216, 128),
    (1500, 9216, 384), (2900, 5003, 1152), (700, 17408, 128), (1111, 17405, 640)])
def test_linear_w8a8_wide(w4, gpu, M, N, K):
    _say(f"linear_w8a8 M={M} N={N} K={K}")
    xq, sx, q, d = _w8a8_inputs(M + N + K, M, N, K)
    txq, tsx, tc, td = _dev(gpu, xq, sx, q, d)
    tq, ref = w4.pack_w8(tc), _w8a8_exact(txq, tsx, tc, td)
    check_w8a8(w4.linear_w8a8(txq, tsx, tq, td, N), ref, "bf16")
    check_w8a8(w4.linear_w8a8(txq, tsx, tq, td, N, out_dtype=F32), ref, "fp32")


@pytest.mark.parametrize("M,N", [(3, 70), (40, 70), (40, 64), (300, 70), (300, 9216), (700, 17408)])
def test_linear_w8a8_tiny_and_huge_outputs(w4, gpu, M, N):
    """Scales are powers of two, so that the fp32 value is exact, subnormal outputs among them, and a
    bf16 output is its nearest, ties to even; what is too large is infinite."""
    _say(f"linear_w8a8 tiny and huge outputs M={M} N={N}")
    xq, _, q, _ = _w8a8_inputs(11, M, N, 128)
    xq[1:, 40:] = 0  # smaller sums, halves of a bf16 step among them
    txq, tc = _dev(gpu, xq, q)
    sums = txq.double() @ tc.double().T.contiguous()
    for es, ed in ((-70, -70), (-60, -66), (0, 0), (52, 60), (60, 52)):
        sx, d = torch.full((M,), 2.0 ** es, device=gpu), torch.full((N,), 2.0 ** ed, device=gpu)
        y32 = (sums * 2.0 ** (es + ed)).cpu().float()
        for out_dtype in (BF16, F32):
            y = w4.linear_w8a8(txq, sx, w4.pack_w8(tc), d, N, out_dtype=out_dtype).cpu()
            want = y32.to(out_dtype)
            assert torch.equal(y, want), f"2^{es} 2^{ed} {out_dtype}: {int((y != want).sum())} of {y.numel()} differ"


@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_w8a8_largest_sums(w4, gpu, M):
    """K = 130944 of products 2^14: the int32 sum ends 2^21 below its limit, at either sign."""
    _say(f"linear_w8a8 largest sums M={M}")
    K, N = 130944, 33
    xq, q = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
    q[1::2] = 127
    sx, d = np.full(M, 0.5, np.float32), np.full(N, 0.25, np.float32)
    txq, tsx, tc, td = _dev(gpu, xq, sx, q, d)
    y = w4.linear_w8a8(txq, tsx, w4.pack_w8(tc), td, N, out_dtype=F32)
    check_w8a8(y, oracle.w8a8_linear_ref(xq, sx, q, d), "largest sums")


@pytest.mark.parametrize("M", [1, 24, 300])
def test_linear_w8a8_scales(w4, gpu, M):
    """A NaN scale poisons its row or column and nothing else; a zero scale gives zeros."""
    _say(f"linear_w8a8 scales M={M}")
    xq, sx, q, d = _w8a8_inputs(5, M, 40, 256)
    sx[M // 2], d[3], d[5] = np.nan, np.nan, 0.0
    txq, tsx, tc, td = _dev(gpu, xq, sx, q, d)
    y = w4.linear_w8a8(txq, tsx, w4.pack_w8(tc), td, 40, out_dtype=F32)
    check_w8a8(y, oracle.w8a8_linear_ref(xq, sx, q, d), "scales")


def test_linear_w8a8_rows_are_independent(w4, gpu):
    """A row's bits do not depend on how many rows the call has."""
    _say("linear_w8a8 rows alone and together")
    xq, sx, q, d = _w8a8_inputs(6, 520, 333, 1152)
    txq, tsx, tc, td = _dev(gpu, xq, sx, q, d)
    tq = w4.pack_w8(tc)
    y = w4.linear_w8a8(txq, tsx, tq, td, 333, out_dtype=F32)
    for a, b in ((0, 1), (3, 19), (100, 165), (200, 520)):
        assert same_bits(w4.linear_w8a8(txq[a:b], tsx[a:b].clone(), tq, td, 333, out_dtype=F32), y[a:b])


def test_linear_w8a8_far_outputs(w4, gpu):
    """Outputs past element 2^31 of y."""
    _say("linear_w8a8 M=262140 N=8200 K=128")
    M, N, K = 262140, 8200, 128
    g = torch.Generator(device=gpu)
    g.manual_seed(1)
    xq = torch.randint(-127, 128, (M, K), generator=g, device=gpu, dtype=torch.int8)
    c = torch.randint(-127, 128, (N, K), generator=g, device=gpu, dtype=torch.int8)
    sx = torch.rand(M, generator=g, device=gpu) + 0.5
    d = torch.rand(N, generator=g, device=gpu) + 0.5
    y = w4.linear_w8a8(xq, sx, w4.pack_w8(c), d, N)
    rows = torch.tensor([0, 1, 131071, 261871, 262000, M - 2, M - 1], device=gpu)
    ref = oracle.w8a8_linear_ref(xq[rows].cpu().numpy(), sx[rows].cpu().numpy(), c.cpu().numpy(), d.cpu().numpy())
    check_w8a8(y[rows], ref, "far outputs")


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("es,ed", [(-60, -60), (48, 48), (-60, 48)])
def test_linear_w8a8_range_of_scales(w4, gpu, M, es, ed):
    """The ends of the range of scales in which every intermediate is a normal fp32."""
    _say(f"linear_w8a8 scales 2^{es}, 2^{ed} M={M}")
    xq, _, q, _ = _w8a8_inputs(7, M, 70, 256)
    xq[0] = 0
    xq[0, 0] = 1  # sums down to single products
    sx, d = np.full(M, 2.0 ** es, np.float32), np.full(70, 2.0 ** ed, np.float32)
    txq, tsx, tc, td = _dev(gpu, xq, sx, q, d)
    for out_dtype in (BF16, F32):
        y = w4.linear_w8a8(txq, tsx, w4.pack_w8(tc), td, 70, out_dtype=out_dtype)
        check_w8a8(y, oracle.w8a8_linear_ref(xq, sx, q, d), "scales")


# ----------------------------------------------------------------------------
# rows sorted by expert
# ----------------------------------------------------------------------------

SIZES = [
    [1], [0, 1], [3], [16], [17], [0, 0, 5, 0], [1, 1, 1, 1], [2, 0, 31, 16, 1], [15, 17, 0, 64, 65],
    [129, 0, 1, 127, 128], [300, 7], [0, 513, 0, 40], [1] * 130, [2, 0] * 70,
]


def _int8_experts(seed, E, N, K):
    rng = np.random.default_rng(seed)
    return rng.integers(-127, 128, (E, N, K)).astype(np.int8), rng.uniform(1e-4, 1e-2, (E, N)).astype(np.float32)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("si", range(len(SIZES)))
def test_grouped_linear_w8a8(w4, gpu, si, out_dtype):
    sizes = SIZES[si]
    E, rows = len(sizes), sum(sizes)
    N, K = [(33, 256), (130, 384), (513, 128)][si % 3]
    first, extra = (0, 0) if si % 2 else (3, 5)  # rows before the first expert and after the last
    M = first + rows + extra
    _say(f"grouped_linear_w8a8 sizes={sizes[:6]} N={N} K={K} {out_dtype}")
    rng = np.random.default_rng(si)
    xq, sx = _codes(rng, M, K), rng.uniform(1e-3, 0.1, M).astype(np.float32)
    q, d = _int8_experts(si, E, N, K)
    off = _offsets(sizes, first)
    txq, tsx, td, toff = _dev(gpu, xq, sx, d, off)
    tq = torch.stack([w4.pack_w8(torch.from_numpy(q[e]).to(gpu)) for e in range(E)])
    y = torch.full((M, N), 7.0, dtype=out_dtype, device=gpu)
    w4.grouped_linear_w8a8(txq, tsx, toff, tq, td, N, out=y)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        check_w8a8(y[a:b], oracle.w8a8_linear_ref(xq[a:b], sx[a:b], q[e], d[e]), f"expert {e}")
        # the dense product of the same rows, bit for bit
        assert same_bits(w4.linear_w8a8(txq[a:b], tsx[a:b].clone(), tq[e], td[e].clone(), N, out_dtype=out_dtype), y[a:b])
    assert bool((y[:first] == 7.0).all()) and bool((y[first + rows:] == 7.0).all()), "a row of no expert was written"


def _w4_experts(w4, gpu, seed, E, N, K, scale_dtype):
    W = torch.from_numpy(np.stack([workloads.random_weight(N, K, seed=seed * 1000 + e) for e in range(E)])).to(gpu)
    q, d = w4.quantize_rtn_experts(W, scale_dtype)
    return W, q, d


def _w4_ref(W, x, scale_dtype):
    qc, dc = oracle.rtn_quantize_ref(W, "bf16" if scale_dtype == BF16 else "f32")
    return oracle.w4_linear_ref(x, qc, dc)


@pytest.mark.parametrize("out_dtype,scale_dtype", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("si", range(len(SIZES)))
def test_grouped_linear(w4, gpu, si, out_dtype, scale_dtype):
    sizes = SIZES[si]
    E, rows = len(sizes), sum(sizes)
    N, K = [(33, 256), (130, 640), (513, 128)][si % 3]
    first, extra = (0, 0) if si % 2 else (3, 5)
    M = first + rows + extra
    _say(f"grouped_linear sizes={sizes[:6]} N={N} K={K} {out_dtype} scales {scale_dtype}")
    W, q, d = _w4_experts(w4, gpu, si, E, N, K, scale_dtype)
    x = workloads.random_activations(M, K, seed=si, device=gpu)
    off = _offsets(sizes, first)
    y = torch.full((M, N), 7.0, dtype=out_dtype, device=gpu)
    w4.grouped_linear(x, torch.from_numpy(off).to(gpu), q, d, N, out=y)
    xb = _bits(x)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        ref, absdot = _w4_ref(W[e].cpu().numpy(), xb[a:b], scale_dtype)
        check_w4(y[a:b], ref, absdot, f"expert {e}")
    assert bool((y[:first] == 7.0).all()) and bool((y[first + rows:] == 7.0).all()), "a row of no expert was written"
    assert same_bits(w4.grouped_linear(x, torch.from_numpy(off).to(gpu), q, d, N, out_dtype=out_dtype)[first:first + rows],
                     y[first:first + rows]), "not reproducible"


@pytest.mark.parametrize("N,K,sizes", [
    (5000, 640, [40, 0, 150, 33, 60]), (2561, 384, [100, 90, 80, 0, 20, 95, 110, 200]), (2561, 128, [400, 0, 700, 300]),
    (1000, 1152, [300] * 9 + [0, 2000]), (5003, 256, [3000, 0, 500, 1500]), (9216, 128, [2, 0, 1, 1]), (9216, 3840, [2, 3]),
    (70, 256, [500] * 10), (1037, 640, [40, 1, 0, 20, 3, 16, 17])])
def test_grouped_linear_w8a8_wide(w4, gpu, N, K, sizes):
    _say(f"grouped_linear_w8a8 sizes={sizes} N={N} K={K}")
    rng = np.random.default_rng(N + K)
    off = _offsets(sizes)
    xq, sx = _codes(rng, int(off[-1]), K), rng.uniform(1e-3, 0.1, int(off[-1])).astype(np.float32)
    q, d = _int8_experts(N, len(sizes), N, K)
    txq, tsx, tc, td, toff = _dev(gpu, xq, sx, q, d, off)
    tq = torch.stack([w4.pack_w8(tc[e]) for e in range(len(sizes))])
    for out_dtype in (BF16, F32):
        y = w4.grouped_linear_w8a8(txq, tsx, toff, tq, td, N, out_dtype=out_dtype)
        for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
            if a < b:
                check_w8a8(y[a:b], _w8a8_exact(txq[a:b], tsx[a:b], tc[e], td[e]), f"expert {e}")


@pytest.mark.parametrize("N,K,sizes", [(2048, 640, [1] * 19 + [0, 3]), (2050, 256, [3, 0] * 11 + [17, 8, 1] * 8),
                                       (2048, 2560, [1, 0, 2, 1, 4]), (1000, 4224, [40, 8, 0, 33]), (600, 9216, [5, 130, 0, 21]),
                                       (256, 28672, [3, 16]), (1, 128, [1, 2]), (2304, 2688, [290, 0, 45])])
def test_grouped_linear_larger(w4, gpu, N, K, sizes):
    _say(f"grouped_linear N={N} K={K} sizes={sizes}")
    for scale_dtype, out_dtype in ((F32, BF16), (BF16, F32)):
        W, q, d = _w4_experts(w4, gpu, N + K, len(sizes), N, K, scale_dtype)
        off = _offsets(sizes)
        x = workloads.random_activations(int(off[-1]), K, seed=K, device=gpu)
        y = w4.grouped_linear(x, torch.from_numpy(off).to(gpu), q, d, N, out_dtype=out_dtype)
        for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
            if a < b:
                ref, absdot = _w4_ref(W[e].cpu().numpy(), _bits(x)[a:b], scale_dtype)
                check_w4(y[a:b], ref, absdot, f"expert {e}")


@pytest.mark.parametrize("sizes", [[3, 1, 20], [150, 0, 400]])
def test_grouped_linear_poisoned_rows(w4, gpu, sizes):
    """A NaN or infinity in a row of x makes that row of y NaN and no other; a non-finite weight
    group poisons its output of its own expert only.  Groups past K (a partial last quad of
    scales) read no row's neighbour."""
    _say(f"grouped_linear non-finite {sizes}")
    N, K = 70, 640
    W, q, d = _w4_experts(w4, gpu, 9, len(sizes), N, K, F32)
    W[1, 5, 200] = float("inf")
    W[2, 6, 3] = float("nan")
    q, d = w4.quantize_rtn_experts(W)
    off = _offsets(sizes)
    M = int(off[-1])
    x = workloads.random_activations(M, K, seed=9, device=gpu)
    x[1, 0], x[off[1] - 1, K - 1], x[M - 2, 130] = float("nan"), float("inf"), float("-inf")
    for out_dtype in (BF16, F32):
        y = w4.grouped_linear(x, torch.from_numpy(off).to(gpu), q, d, N, out_dtype=out_dtype)
        for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
            if a < b:
                ref, absdot = _w4_ref(W[e].cpu().numpy(), _bits(x)[a:b], F32)
                check_w4(y[a:b], ref, absdot, f"expert {e}")


def test_grouped_rows_are_independent(w4, gpu):
    """A row's bits depend on its own expert alone: not on the rows beside it, nor on the call's other experts."""
    _say("grouped rows alone and together")
    N, K, sizes = 200, 1152, [5, 0, 70, 300, 1]
    W, q, d = _w4_experts(w4, gpu, 4, 5, N, K, F32)
    q8, d8 = w4.quantize_w8(W)
    off = _offsets(sizes)
    x = workloads.random_activations(int(off[-1]), K, seed=4, device=gpu)
    xq, sx = w4.quantize_tokens(x)
    toff = torch.from_numpy(off).to(gpu)
    y8 = w4.grouped_linear_w8a8(xq, sx, toff, q8, d8, N, out_dtype=F32)
    for e in (2, 3):
        alone = torch.tensor([0, sizes[e]], dtype=torch.int32, device=gpu)
        a, b = off[e], off[e + 1]
        got = w4.grouped_linear_w8a8(xq[a:b], sx[a:b].clone(), alone, q8[e:e + 1], d8[e:e + 1], N, out_dtype=F32)
        assert same_bits(got, y8[a:b])


def test_grouped_offsets_out_of_range(w4, gpu):
    """Offsets that decrease or leave [0, M] are clamped: nothing outside y is written, and a row
    that only the first expert's range holds is right (ranges that overlap both write their rows)."""
    _say("grouped offsets out of range")
    N, K, M = 40, 256, 50
    W, q, d = _w4_experts(w4, gpu, 6, 4, N, K, F32)
    q8, d8 = w4.quantize_w8(W)
    x = workloads.random_activations(M, K, seed=6, device=gpu)
    xq, sx = w4.quantize_tokens(x)
    for off in ([0, 7, 90, 2000000000, 1], [0, 7, 3, 20, -5], [-2000000000, 7, 7, 7, 60], [0, 7, 0, 50, 0]):
        toff = torch.tensor(off, dtype=torch.int32, device=gpu)
        buf = torch.full((M + 40, N), 7.0, device=gpu)
        w4.grouped_linear(x, toff, q, d, N, out=buf[20:20 + M])
        clamped = np.clip(off, 0, M)
        mine = [m for m in range(7) if not any(a <= m < b for a, b in zip(clamped[1:-1], clamped[2:]))]
        ref, absdot = _w4_ref(W[0].cpu().numpy(), _bits(x)[:7], F32)
        check_w4(buf[20:27][mine], ref[mine], absdot[mine], "expert 0")
        assert bool((buf[:20] == 7.0).all()) and bool((buf[20 + M:] == 7.0).all())
        buf8 = torch.full((M + 40, N), 7.0, device=gpu)
        w4.grouped_linear_w8a8(xq, sx, toff, q8, d8, N, out=buf8[20:20 + M])
        dense = w4.linear_w8a8(xq[:7], sx[:7].clone(), q8[0], d8[0].clone(), N, out_dtype=F32)
        assert same_bits(buf8[20:27][mine], dense[mine])
        assert bool((buf8[:20] == 7.0).all()) and bool((buf8[20 + M:] == 7.0).all())


def test_grouped_far_experts(w4, gpu):
    """Weights past 4 GiB from the first expert's."""
    _say("grouped, 5 GiB of 8-bit and 2.5 GiB of 4-bit weights")
    E, N, K = 40, 8192, 16384
    q8 = torch.zeros((E, w4.packed_bytes_w8(N, K)), dtype=torch.int8, device=gpu)
    d8 = torch.zeros((E, N), device=gpu)
    W = workloads.random_weight(N, K, seed=2, device=gpu)
    q, d = w4.quantize_w8(W)
    q8[E - 1], d8[E - 1] = q, d
    x = workloads.random_activations(5, K, seed=2, device=gpu)
    off = torch.tensor([0] * (E - 1) + [1, 5], dtype=torch.int32, device=gpu)
    xq, sx = w4.quantize_tokens(x)
    y = w4.grouped_linear_w8a8(xq, sx, off, q8, d8, N, out_dtype=F32)
    assert same_bits(y[1:], w4.linear_w8a8(xq[1:], sx[1:].clone(), q, d, N, out_dtype=F32))
    assert bool((y[0] == 0).all())
    del q8
    nb, ns = w4.packed_bytes(N, K), w4.scale_count(N, K)
    q4, d4 = torch.zeros((E, nb), dtype=torch.uint8, device=gpu), torch.zeros((E, ns), device=gpu)
    q4[E - 1], d4[E - 1] = w4.quantize_rtn(W)
    y = w4.grouped_linear(x, off, q4, d4, N, out_dtype=F32)
    rows = np.arange(0, N, 61)
    ref, absdot = _w4_ref(W[torch.from_numpy(rows).to(gpu)].cpu().numpy(), _bits(x)[1:], F32)
    check_w4(y[1:][:, torch.from_numpy(rows).to(gpu)].contiguous(), ref, absdot, "last expert")
    assert bool((y[0] == 0).all())  # zero scales


def test_grouped_far_outputs(w4, gpu):
    """Outputs past element 2^31 of y, rows of the last tiles of three experts."""
    _say("grouped, M=262140 N=8200 K=128")
    M, N, K, E = 262140, 8200, 128, 3
    W, q, d = _w4_experts(w4, gpu, 12, E, N, K, BF16)
    q8, d8 = w4.quantize_w8(W)
    g = torch.Generator(device=gpu)
    g.manual_seed(12)
    x = torch.randn((M, K), generator=g, device=gpu).to(BF16)
    off = torch.tensor([0, 131071, 261000, M], dtype=torch.int32, device=gpu)
    rows = np.array([0, 131070, 131071, 260999, 261000, 262101, M - 2, M - 1])
    expert = np.searchsorted([131071, 261000, M], rows, side="right")
    trows = torch.from_numpy(rows).to(gpu)
    y = w4.grouped_linear(x, off, q, d, N)
    for e in range(E):
        mine = expert == e
        ref, absdot = _w4_ref(W[e].cpu().numpy(), _bits(x[trows[torch.from_numpy(mine).to(gpu)]]), BF16)
        check_w4(y[trows[torch.from_numpy(mine).to(gpu)]], ref, absdot, f"expert {e}")
    del y
    xq, sx = w4.quantize_tokens(x)
    y = w4.grouped_linear_w8a8(xq, sx, off, q8, d8, N)
    for r, e in zip(rows.tolist(), expert.tolist()):
        assert same_bits(w4.linear_w8a8(xq[r:r + 1].clone(), sx[r:r + 1].clone(), q8[e], d8[e].clone(), N), y[r:r + 1])


def test_grouped_many_experts(w4, gpu):
    """As many experts as a call takes, most without rows."""
    _say("grouped, 4096 experts")
    E, N, K = 4096, 16, 128
    W = torch.from_numpy(np.random.default_rng(13).standard_normal((E, N, K)).astype(np.float32)).to(gpu)
    q8, d8 = w4.quantize_w8(W)
    q, d = w4.quantize_rtn_experts(W)
    sizes = np.zeros(E, np.int64)
    for e, s in ((0, 3), (63, 1), (64, 20), (1000, 40), (4031, 2), (4032, 1), (4095, 17)):
        sizes[e] = s
    off = _offsets(sizes)
    x = workloads.random_activations(int(off[-1]), K, seed=13, device=gpu)
    xq, sx = w4.quantize_tokens(x)
    toff = torch.from_numpy(off).to(gpu)
    y8, y4 = w4.grouped_linear_w8a8(xq, sx, toff, q8, d8, N), w4.grouped_linear(x, toff, q, d, N)
    for e in np.flatnonzero(sizes):
        a, b = off[e], off[e + 1]
        assert same_bits(y8[a:b], w4.linear_w8a8(xq[a:b].clone(), sx[a:b].clone(), q8[e], d8[e].clone(), N))
        ref, absdot = _w4_ref(W[e].cpu().numpy(), _bits(x)[a:b], F32)
        check_w4(y4[a:b], ref, absdot, f"expert {e}")


# ----------------------------------------------------------------------------
# together, as a model uses them
# ----------------------------------------------------------------------------

def test_w8linear(w4, gpu):
    _say("W8Linear on bf16 and fp32 activations")
    W = workloads.random_weight(300, 1152, seed=3)
    lin = w4.W8Linear.from_float(torch.from_numpy(W).to(gpu))
    q, d = oracle.rtn_rows_ref(W)
    for M in (1, 9, 270):
        x = workloads.random_activations(M, 1152, seed=M, device=gpu)
        xq, sx = oracle.rtn_rows_ref(x.float().cpu().numpy())
        ref = oracle.w8a8_linear_ref(xq, sx, q, d)
        check_w8a8(lin(x), ref, "W8Linear")
        check_w8a8(lin(x.float(), out_dtype=F32), ref, "W8Linear fp32")


def test_expert_layer(w4, gpu):
    """A layer of experts: 4-bit gate and up projections, their product re-quantized token by token,
    and the 8-bit down projection, over one set of offsets written on the GPU."""
    _say("expert layer: grouped_linear x2 -> quantize_tokens -> grouped_linear_w8a8")
    E, top, tokens, hidden, ffn = 6, 2, 37, 640, 384
    g = torch.Generator(device=gpu)
    g.manual_seed(11)
    picks = torch.rand((tokens, E), generator=g, device=gpu).topk(top, dim=1).indices.reshape(-1)
    order = torch.argsort(picks, stable=True)
    off = torch.searchsorted(picks[order].contiguous(), torch.arange(E + 1, device=gpu)).to(torch.int32)
    x = workloads.random_activations(tokens, hidden, seed=11, device=gpu)[order // top].contiguous()
    Wg, qg, dg = _w4_experts(w4, gpu, 21, E, ffn, hidden, BF16)
    Wu, qu, du = _w4_experts(w4, gpu, 22, E, ffn, hidden, F32)
    Wd = torch.from_numpy(np.stack([workloads.random_weight(hidden, ffn, seed=2300 + e) for e in range(E)])).to(gpu)
    qd, dd = w4.quantize_w8(Wd)
    gate = w4.grouped_linear(x, off, qg, dg, ffn, out_dtype=F32)
    up = w4.grouped_linear(x, off, qu, du, ffn, out_dtype=F32)
    h = torch.nn.functional.silu(gate) * up
    hq, hs = w4.quantize_tokens(h)
    y = w4.grouped_linear_w8a8(hq, hs, off, qd, dd, hidden)
    ends = off.tolist()
    assert ends[0] == 0 and ends[-1] == tokens * top
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        for got, W, sd in ((gate, Wg, BF16), (up, Wu, F32)):
            ref, absdot = _w4_ref(W[e].cpu().numpy(), _bits(x)[a:b], sd)
            check_w4(got[a:b], ref, absdot, "projection")
        rq, rs = oracle.rtn_rows_ref(h[a:b].cpu().numpy())
        assert np.array_equal(hq[a:b].cpu().numpy(), rq)
        wq, wd = oracle.rtn_rows_ref(Wd[e].cpu().numpy())
        check_w8a8(y[a:b], oracle.w8a8_linear_ref(rq, rs, wq, wd), "down projection")


@pytest.mark.parametrize("M", [24, 400])
def test_graph_replays_with_new_routing(w4, gpu, M):
    """A captured pass follows the offsets, tokens and activations of each replay."""
    _say(f"graph of the expert operators, M={M}")
    E, N, K = 5, 300, 640
    W, q, d = _w4_experts(w4, gpu, 31, E, N, K, F32)
    q8, d8 = w4.quantize_w8(W)
    x, off = torch.zeros((M, K), dtype=BF16, device=gpu), torch.zeros(E + 1, dtype=torch.int32, device=gpu)
    y4, y8 = torch.zeros((M, N), dtype=BF16, device=gpu), torch.zeros((M, N), device=gpu)
    xq, sx = torch.zeros((M, K), dtype=torch.int8, device=gpu), torch.zeros(M, device=gpu)
    yd = torch.zeros((M, N), dtype=BF16, device=gpu)

    def step():
        w4.grouped_linear(x, off, q, d, N, out=y4)
        w4.quantize_tokens(x, out=(xq, sx))
        w4.grouped_linear_w8a8(xq, sx, off, q8, d8, N, out=y8)
        w4.linear_w8a8(xq, sx, q8[0], d8[0], N, out=yd)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(31)
    for it in range(4):
        x.copy_(workloads.random_activations(M, K, seed=100 + it, device=gpu))
        cut = np.sort(rng.integers(0, M + 1, E - 1))
        off.copy_(torch.from_numpy(np.concatenate([[0], cut, [M]]).astype(np.int32)))
        for t in (y4, y8, yd):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y4, y8, yd)]
        for t in (y4, y8, yd):
            t.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (y4, y8, yd)):
            assert same_bits(a, b), f"replay {it}"


def test_two_streams_at_once(w4, gpu):
    """Calls that run at the same time on two streams do not disturb each other (no shared state)."""
    _say("two streams")
    E, N, K, sizes = 8, 512, 1152, [30, 0, 200, 1, 77, 16, 0, 60]
    W, q, d = _w4_experts(w4, gpu, 41, E, N, K, F32)
    q8, d8 = w4.quantize_w8(W)
    off = torch.from_numpy(_offsets(sizes)).to(gpu)
    M = sum(sizes)
    xs = [workloads.random_activations(M, K, seed=50 + i, device=gpu) for i in range(2)]

    def run(x):
        xq, sx = w4.quantize_tokens(x)
        return w4.grouped_linear(x, off, q, d, N), w4.grouped_linear_w8a8(xq, sx, off, q8, d8, N)

    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(same_bits(a, b) for a, b in zip(r, want[i]))


def test_binding_refuses_wrong_sizes(w4, gpu):
    _say("binding refusals")
    xq, sx, q, d = _dev(gpu, *_w8a8_inputs(1, 4, 16, 128))
    q = w4.pack_w8(q)
    off = torch.tensor([0, 4], dtype=torch.int32, device=gpu)
    with pytest.raises(ValueError, match="sx"):
        w4.linear_w8a8(xq, sx[:3].clone(), q, d, 16)
    with pytest.raises(ValueError, match="q must hold"):
        w4.linear_w8a8(xq, sx, q[:-16].clone(), d, 16)
    with pytest.raises(ValueError, match="d must"):
        w4.linear_w8a8(xq, sx, q, d[:8].clone(), 16)
    with pytest.raises(ValueError, match="out must"):
        w4.linear_w8a8(xq, sx, q, d, 16, out=torch.empty((4, 17), dtype=BF16, device=gpu))
    with pytest.raises(TypeError):
        w4.linear_w8a8(xq, sx, q, d, 16, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        w4.linear_w8a8(xq.t().contiguous().t(), sx, q, d, 16)
    with pytest.raises(TypeError, match="offsets"):
        w4.grouped_linear_w8a8(xq, sx, off.long(), q.view(1, -1), d.view(1, -1), 16)
    with pytest.raises(ValueError, match="d must"):
        w4.grouped_linear_w8a8(xq, sx, off, q.view(1, -1), d, 16)
    with pytest.raises(w4.W4Error):
        w4.quantize_tokens(torch.zeros((2, 100), device=gpu))
    with pytest.raises(ValueError, match="several devices"):
        w4.linear_w8a8(xq, sx.cpu(), q, d, 16)
    # nothing to do
    assert w4.linear_w8a8(xq[:0], sx[:0], q, d, 16).shape == (0, 16)
    assert w4.quantize_tokens(torch.zeros((0, 128), dtype=BF16, device=gpu))[0].shape == (0, 128)
    none = torch.zeros(1, dtype=torch.int32, device=gpu)
    y = torch.full((4, 16), 7.0, device=gpu)
    w4.grouped_linear_w8a8(xq, sx, none, torch.empty((0, q.numel()), dtype=torch.int8, device=gpu),
                           torch.empty((0, 16), device=gpu), 16, out=y)
    assert bool((y == 7.0).all())
