"""Microscaled 4-bit floating point on an MI355X, against the oracle.

Codes, scales, values and layouts are compared bit for bit.  The product's fp32
value lies within (K / 128 + 8) * 2^-22 of sum |x^ w^| (plus what underflows, K *
2^-120) of the exact one: the promise of include/w4.h, from the rounding of one
product of the matrix unit; a bf16 output is the nearest-even bf16 of such a value.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(f"\n[case] {msg}", flush=True)


def _bits(y):
    y = y.detach().cpu()
    return y.numpy().view(np.uint32) if y.dtype == F32 else y.view(torch.int16).numpy().view(np.uint16)


def check(y, ref, absdot, K, what):
    ok = oracle.admissible(_bits(y), ref, oracle.mx4_tolerance(absdot, K), "f32" if y.dtype == F32 else "bf16", rel=1.0,
                           abs_=0.0)
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} outputs out of tolerance"


def same_bits(a, b):
    return a.shape == b.shape and np.array_equal(_bits(a), _bits(b))


def special_rows(rng, N, K):
    """Normal rows with hard blocks among them: zeros of both signs, NaN, infinity, subnormals, huge values,
    one large member, every tie between two codes and its neighbours."""
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    for n in range(N):
        b = 32 * int(rng.integers(0, K // 32))
        block = slice(b, b + 32)
        kind = n % 11
        if kind == 1:
            W[n, block] = np.where(rng.random(32) < 0.5, 0.0, -0.0)
        elif kind == 2:
            W[n, b + int(rng.integers(0, 32))] = np.nan
        elif kind == 3:
            W[n, b + int(rng.integers(0, 32))] = -np.inf
        elif kind == 4:
            W[n] *= np.float32(2.0 ** -122)  # some blocks' scales at 2^-127, members subnormal
        elif kind == 5:
            W[n, block] = np.float32(1e-40) * rng.standard_normal(32).astype(np.float32)
        elif kind == 6:
            W[n] *= np.float32(2.0 ** 126)
        elif kind == 7:
            W[n, block] *= np.float32(1e6)
        elif kind in (8, 9):
            # ties between two codes, and the values next to them
            e = int(rng.integers(-100, 100))
            t = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], 32) * rng.choice([-1.0, 1.0], 32)
            v = np.ldexp(t, e).astype(np.float32)
            v = (v.view(np.int32) + (rng.integers(-1, 2, 32) if kind == 9 else 0)).astype(np.int32).view(np.float32)
            v[0] = np.ldexp(4.0, e)  # the block's scale is 2^e
            W[n, block] = v
    return W


# ----------------------------------------------------------------------------
# quantizers, values and layout: bit-exact
# ----------------------------------------------------------------------------

SHAPES = [(1, 128), (11, 128), (16, 256), (37, 384), (100, 1152), (33, 2560), (48, 640), (23, 28672), (13, 130944)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", SHAPES)
def test_quantize_and_back(w4, gpu, N, K, dtype):
    _say(f"quantize_mx4 {N}x{K} {dtype}")
    W = torch.from_numpy(special_rows(np.random.default_rng(N * 7 + K), N, K)).to(dtype)
    codes, scales = oracle.mx4_quantize_ref(W.float().numpy())
    q_ref, s_ref = oracle.pack_mx4_ref(codes, scales)
    nb, ns = w4.packed_bytes_mx4(N, K), w4.scale_bytes_mx4(N, K)
    assert (nb, ns) == (q_ref.size, s_ref.size)
    qbuf = torch.full((nb + 64,), 99, dtype=torch.uint8, device=gpu)
    sbuf = torch.full((ns + 64,), 99, dtype=torch.uint8, device=gpu)
    q, s = w4.quantize_mx4(W.to(gpu), out=(qbuf[16:16 + nb], sbuf[32:32 + ns]))
    assert np.array_equal(s.cpu().numpy(), s_ref), "scales differ"
    assert np.array_equal(q.cpu().numpy(), q_ref), "codes differ"
    for buf, a, n in ((qbuf, 16, nb), (sbuf, 32, ns)):
        assert bool((buf[:a] == 99).all()) and bool((buf[a + n:] == 99).all()), "bytes around were written"
    qc, sc = w4.unpack_mx4(q.clone(), s.clone(), N, K)
    assert np.array_equal(qc.cpu().numpy(), oracle.mx4_bytes_ref(codes)) and np.array_equal(sc.cpu().numpy(), scales)
    qbuf.fill_(7), sbuf.fill_(7)
    w4.pack_mx4(qc, sc, out=(qbuf[16:16 + nb], sbuf[32:32 + ns]))
    assert np.array_equal(q.cpu().numpy(), q_ref) and np.array_equal(s.cpu().numpy(), s_ref)
    values = oracle.mx4_values_ref(codes, scales).astype(np.float32)
    for out in (BF16, F32):
        got = w4.dequantize_mx4(q, s, N, K, out_dtype=out).float().cpu().numpy()
        assert np.array_equal(got, values, equal_nan=True) and np.array_equal(np.signbit(got) | np.isnan(got),
                                                                              np.signbit(values) | np.isnan(values))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K", SHAPES + [(3, 896), (300, 2560)])
def test_quantize_tokens_and_back(w4, gpu, M, K, dtype):
    _say(f"quantize_tokens_mx4 {M}x{K} {dtype}")
    x = torch.from_numpy(special_rows(np.random.default_rng(M + 3 * K), M, K)).to(dtype)
    codes, scales = oracle.mx4_quantize_ref(x.float().numpy())
    qbuf = torch.full((M + 2, K // 2), 99, dtype=torch.uint8, device=gpu)
    sbuf = torch.full((M + 2, K // 32), 99, dtype=torch.uint8, device=gpu)
    q, s = w4.quantize_tokens_mx4(x.to(gpu), out=(qbuf[1:1 + M], sbuf[1:1 + M]))
    assert np.array_equal(s.cpu().numpy(), scales), "scales differ"
    assert np.array_equal(q.cpu().numpy(), oracle.mx4_bytes_ref(codes)), "codes differ"
    for buf in (qbuf, sbuf):
        assert bool((buf[0] == 99).all()) and bool((buf[1 + M:] == 99).all())
    values = oracle.mx4_values_ref(codes, scales).astype(np.float32)
    for out in (BF16, F32):
        obuf = torch.full((M + 2, K), 5.0, dtype=out, device=gpu)
        w4.dequantize_tokens_mx4(q, s, out=obuf[1:1 + M])
        assert np.array_equal(obuf[1:1 + M].float().cpu().numpy(), values, equal_nan=True)
        assert bool((obuf[0] == 5).all()) and bool((obuf[1 + M] == 5).all())


def test_every_code_under_every_scale(w4, gpu):
    """Any byte is a scale and any four bits a code: values and the way back to the codes."""
    _say("mx4: every code under every scale")
    codes = np.tile(np.arange(32) % 16, (256, 4)).astype(np.uint8)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, axis=1)
    q, s = (torch.from_numpy(v).to(gpu) for v in (oracle.mx4_bytes_ref(codes), scales))
    with np.errstate(over="ignore"):
        want = oracle.mx4_values_ref(codes, scales).astype(np.float32)
    for out in (BF16, F32):
        got = w4.dequantize_tokens_mx4(q, s, out_dtype=out).float().cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)
        # blocks whose largest member is 6 have a scale of their own
        rows = slice(0, 253)
        q2, s2 = w4.quantize_tokens_mx4(torch.from_numpy(want[rows]).to(gpu).to(out))
        assert torch.equal(q2, q[rows]) and torch.equal(s2, s[rows])


@pytest.mark.parametrize("N", [32, 21])
def test_experts_are_each_matrix(w4, gpu, N):
    _say(f"quantize_mx4 of a stack of experts of {N} rows")
    W = torch.from_numpy(special_rows(np.random.default_rng(8), 3 * N, 384).reshape(3, N, 384)).to(gpu)
    q, s = w4.quantize_mx4(W)
    for e in range(3):
        qe, se = w4.quantize_mx4(W[e].contiguous())
        assert torch.equal(q[e], qe) and torch.equal(s[e], se)


def test_quantize_many_rows(w4, gpu):
    """More rows than any launch has blocks resident, every code checked on the GPU."""
    _say("quantize_tokens_mx4 and quantize_mx4 70001 x 128")
    g = torch.Generator(device=gpu)
    g.manual_seed(3)
    x = torch.randn((70001, 128), generator=g, device=gpu).to(BF16)
    q, s = w4.quantize_tokens_mx4(x)
    v = w4.dequantize_tokens_mx4(q, s, out_dtype=F32)
    top = x.float().reshape(-1, 4, 32).abs().amax(-1)
    step = torch.ldexp(torch.ones_like(top), torch.frexp(top)[1] - 3)  # the scale
    # a member is off by at most half the widest gap (2 of the scale), or was above 6 (at most 2 more)
    assert bool(((v - x.float()).reshape(-1, 4, 32).abs().amax(-1) <= 2 * step).all())
    qc, sc = w4.unpack_mx4(*w4.quantize_mx4(x), 70001, 128)
    assert torch.equal(qc, q) and torch.equal(sc, s)


# ----------------------------------------------------------------------------
# product
# ----------------------------------------------------------------------------

def _random(rng, rows, K, spread=6, nan=()):
    """Codes and scales of rows, all codes alike likely; rows `nan` hold one NaN scale each."""
    codes = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    scales = rng.integers(127 - spread, 128 + spread, (rows, K // 32)).astype(np.uint8)
    for r in nan:
        scales[r, int(rng.integers(0, K // 32))] = 255
    return codes, scales


def _gpu(gpu, codes, scales):
    return torch.from_numpy(oracle.mx4_bytes_ref(codes)).to(gpu), torch.from_numpy(scales).to(gpu)


def _native(gpu, codes, scales):
    return tuple(torch.from_numpy(v).to(gpu) for v in oracle.pack_mx4_ref(codes, scales))


def _framed(gpu, M, N, out):
    """An output with rows around it that a call may not touch."""
    buf = torch.full((M + 2, N), 77.0, dtype=out, device=gpu)
    return buf, buf[1:1 + M]


def _frame_kept(buf):
    return bool((buf[0] == 77).all()) and bool((buf[-1] == 77).all())


ROWS = [1, 2, 5, 16, 17, 33, 48, 64, 65, 130, 257, 300]
MATRICES = [(16, 128), (1, 256), (37, 384), (100, 640), (65, 1152), (129, 2560), (257, 512), (520, 1408), (96, 4736)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N,K", MATRICES)
def test_linear_mx4(w4, gpu, N, K, out):
    rng = np.random.default_rng(N + K)
    wc, ws = _random(rng, N, K, nan=(N // 2,) if N > 1 else ())
    q, s = _native(gpu, wc, ws)
    for M in ROWS:
        _say(f"linear_mx4 {M} rows of {N}x{K} {out}")
        xc, xs = _random(rng, M, K, nan=(M - 1,) if M > 2 else ())
        y_ref, a_ref = oracle.mx4_linear_ref(xc, xs, wc, ws)
        buf, y = _framed(gpu, M, N, out)
        w4.linear_mx4(*_gpu(gpu, xc, xs), q, s, N, out=y)
        check(y, y_ref, a_ref, K, f"{M} rows")
        assert _frame_kept(buf)


@pytest.mark.parametrize("M", [1, 16, 40, 200])
def test_linear_mx4_is_exact_on_small_integers(w4, gpu, M):
    """Values that are halves up to 6 with scales of 1: every sum is exact in fp32, in any order."""
    _say(f"linear_mx4 exact, {M} rows")
    rng = np.random.default_rng(M)
    N, K = 200, 9216
    xc, wc = rng.integers(0, 16, (M, K)).astype(np.uint8), rng.integers(0, 16, (N, K)).astype(np.uint8)
    one = lambda rows: np.full((rows, K // 32), 127, np.uint8)  # noqa: E731
    y_ref, _ = oracle.mx4_linear_ref(xc, one(M), wc, one(N))
    y = w4.linear_mx4(*_gpu(gpu, xc, one(M)), *_native(gpu, wc, one(N)), N, out_dtype=F32)
    assert np.array_equal(y.cpu().numpy(), y_ref.astype(np.float32))


def test_linear_mx4_places(w4, gpu):
    """One code in x and one in w: every input meets its own counterpart and scale, and no other."""
    _say("linear_mx4 places")
    K = 1152
    rng = np.random.default_rng(5)
    for M in (16, 64, 300):
        k = rng.integers(0, K, M)
        xc, xs = np.zeros((M, K), np.uint8), np.full((M, K // 32), 127, np.uint8)
        xc[np.arange(M), k] = 2  # 1.0
        xs[np.arange(M), k // 32] = 130
        wc, ws = _random(rng, 48, K)
        y = w4.linear_mx4(*_gpu(gpu, xc, xs), *_native(gpu, wc, ws), 48, out_dtype=F32).cpu().numpy()
        assert np.array_equal(y, 8.0 * oracle.mx4_values_ref(wc, ws)[:, k].T.astype(np.float32))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_linear_mx4_wide_scales(w4, gpu, M):
    """Scales far apart: 2^-60 to 2^60 in one row, blocks of zeros with the smallest scale, large cancellation."""
    _say(f"linear_mx4 wide scales, {M} rows")
    rng = np.random.default_rng(7)
    N, K = 70, 1408
    xc, xs = _random(rng, M, K, spread=30)
    wc, ws = _random(rng, N, K, spread=30)
    zero = rng.random((M, K // 32)) < 0.1
    xs[zero] = 0
    xc[np.repeat(zero, 32, axis=1)] = 0
    y_ref, a_ref = oracle.mx4_linear_ref(xc, xs, wc, ws)
    y = w4.linear_mx4(*_gpu(gpu, xc, xs), *_native(gpu, wc, ws), N, out_dtype=F32)
    check(y, y_ref, a_ref, K, "wide")


def test_linear_mx4_long_rows(w4, gpu):
    _say("linear_mx4 K = 130944")
    rng = np.random.default_rng(9)
    K = 130944
    wc, ws = _random(rng, 33, K)
    for M in (1, 20, 70):
        xc, xs = _random(rng, M, K)
        y_ref, a_ref = oracle.mx4_linear_ref(xc, xs, wc, ws)
        y = w4.linear_mx4(*_gpu(gpu, xc, xs), *_native(gpu, wc, ws), 33, out_dtype=F32)
        check(y, y_ref, a_ref, K, f"{M} rows")


def test_linear_mx4_from_floats(w4, gpu):
    """The way a program takes: weights and activations quantized on the GPU, MX4Linear."""
    _say("MX4Linear")
    g = torch.Generator(device=gpu)
    g.manual_seed(4)
    W = torch.randn((777, 2560), generator=g, device=gpu) * 0.02
    x = torch.randn((45, 2560), generator=g, device=gpu).to(BF16)
    layer = w4.MX4Linear.from_float(W)
    wc, ws = oracle.mx4_quantize_ref(W.cpu().numpy())
    xc, xs = oracle.mx4_quantize_ref(x.float().cpu().numpy())
    y_ref, a_ref = oracle.mx4_linear_ref(xc, xs, wc, ws)
    check(layer(x), y_ref, a_ref, 2560, "MX4Linear")
    check(layer(x, out_dtype=F32), y_ref, a_ref, 2560, "MX4Linear fp32")


def test_linear_mx4_repeats(w4, gpu):
    """The same bits from call to call, on another stream, and from a graph replayed with other inputs between."""
    _say("linear_mx4 repeats")
    rng = np.random.default_rng(11)
    N, K = 520, 2560
    wc, ws = _random(rng, N, K)
    q, s = _native(gpu, wc, ws)
    for M in (1, 30, 270):
        xq, xs = _gpu(gpu, *_random(rng, M, K))
        want = w4.linear_mx4(xq, xs, q, s, N)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            y = w4.linear_mx4(xq, xs, q, s, N)
        torch.cuda.current_stream().wait_stream(other)
        assert same_bits(y, want)
        held_q, held_s, out = xq.clone(), xs.clone(), torch.zeros((M, N), dtype=BF16, device=gpu)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w4.linear_mx4(held_q, held_s, q, s, N, out=out)
        for _ in range(3):
            held_q.copy_(xq), held_s.copy_(xs)
            out.zero_()
            graph.replay()
            assert same_bits(out, want)
            q2, s2 = _gpu(gpu, *_random(rng, M, K))
            held_q.copy_(q2), held_s.copy_(s2)
            graph.replay()
            assert same_bits(out, w4.linear_mx4(q2, s2, q, s, N))


# ----------------------------------------------------------------------------
# rows sorted by expert
# ----------------------------------------------------------------------------

ROUTINGS = {
    "even": [16] * 6,
    "uneven": [1, 40, 0, 7, 300, 17],
    "one": [0, 0, 90, 0],
    "few": [1, 0, 2, 1, 0, 0, 3],
    "long": [70, 513, 130],
}


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N,K", [(48, 384), (37, 1152), (300, 640)])
@pytest.mark.parametrize("routing", sorted(ROUTINGS))
def test_grouped_linear_mx4(w4, gpu, routing, N, K, out):
    _say(f"grouped_linear_mx4 {routing} {N}x{K} {out}")
    rng = np.random.default_rng(len(routing) + N)
    sizes, first, after = ROUTINGS[routing], 3, 5
    E, M = len(sizes), first + sum(sizes) + after
    offsets = np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)
    made = [_random(rng, N, K) for _ in range(E)]
    packed = [oracle.pack_mx4_ref(*m) for m in made]
    q, s = (torch.from_numpy(np.stack([p[i] for p in packed])).to(gpu) for i in (0, 1))
    # rows of no expert may hold anything
    xc, xs = _random(rng, M, K, nan=(0, M - 1))
    buf, y = _framed(gpu, M, N, out)
    w4.grouped_linear_mx4(*_gpu(gpu, xc, xs), torch.from_numpy(offsets).to(gpu), q, s, N, out=y)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            y_ref, a_ref = oracle.mx4_linear_ref(xc[a:b], xs[a:b], *made[e])
            check(y[a:b], y_ref, a_ref, K, f"expert {e}")
    assert bool((y[:first] == 77).all()) and bool((y[M - after:] == 77).all()) and _frame_kept(buf)


def test_grouped_linear_mx4_odd_offsets(w4, gpu):
    """Offsets that decrease, overlap or leave [0, M]: rows outside are never touched."""
    _say("grouped_linear_mx4 odd offsets")
    rng = np.random.default_rng(3)
    N, K, M = 40, 256, 50
    made = [_random(rng, N, K) for _ in range(4)]
    packed = [oracle.pack_mx4_ref(*m) for m in made]
    q, s = (torch.from_numpy(np.stack([p[i] for p in packed])).to(gpu) for i in (0, 1))
    xq, xs = _gpu(gpu, *_random(rng, M, K))
    for offsets in ([0, 60, 20, 30, 90], [-5, 10, 10, 200, 20], [50, 50, 50, 50, 50], [7, 3, 2, 1, 0],
                    [2 ** 31 - 1, -2 ** 31, 5, 60, 70]):
        buf, y = _framed(gpu, M, N, BF16)
        w4.grouped_linear_mx4(xq, xs, torch.tensor(offsets, dtype=torch.int32, device=gpu), q, s, N, out=y)
        torch.cuda.synchronize()
        assert _frame_kept(buf), offsets


def test_many_experts_mx4(w4, gpu):
    """More experts than lanes of a wavefront, most without rows."""
    _say("grouped_linear_mx4 300 experts")
    rng = np.random.default_rng(6)
    N, K, E = 32, 128, 300
    sizes = rng.integers(0, 3, E) * (rng.random(E) < 0.3)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    M = int(offsets[-1])
    made = [_random(rng, N, K) for _ in range(E)]
    packed = [oracle.pack_mx4_ref(*m) for m in made]
    q, s = (torch.from_numpy(np.stack([p[i] for p in packed])).to(gpu) for i in (0, 1))
    xc, xs = _random(rng, M, K)
    y = w4.grouped_linear_mx4(*_gpu(gpu, xc, xs), torch.from_numpy(offsets).to(gpu), q, s, N, out_dtype=F32)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            y_ref, a_ref = oracle.mx4_linear_ref(xc[a:b], xs[a:b], *made[e])
            check(y[a:b], y_ref, a_ref, K, f"expert {e}")


def test_refusals_on_the_gpu(w4, gpu):
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=gpu)  # noqa: E731
    q, s = u8(2048), u8(256)
    for call in (lambda: w4.linear_mx4(u8(2, 64), u8(2, 4), u8(2047), s, 16),
                 lambda: w4.linear_mx4(u8(2, 64), u8(2, 4), q, u8(255), 16),
                 lambda: w4.linear_mx4(u8(2, 64), u8(2, 5), q, s, 16),
                 lambda: w4.linear_mx4(u8(2, 128)[:, ::2], u8(2, 4), q, s, 16),
                 lambda: w4.linear_mx4(u8(2, 64), u8(2, 4), q, s, 16, out=torch.zeros((2, 17), device=gpu)),
                 lambda: w4.dequantize_mx4(q, s, 17, 128),
                 lambda: w4.quantize_tokens_mx4(torch.zeros((2, 256), device=gpu), out=(u8(2, 64), u8(2, 8))),
                 lambda: w4.grouped_linear_mx4(u8(2, 64), u8(2, 4), torch.zeros(3, dtype=torch.int32, device=gpu),
                                               u8(1, 2048), u8(1, 256), 16)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        w4.linear_mx4(u8(2, 64), u8(2, 4), q, s, 16, out_dtype=torch.float16)
    for call in (lambda: w4.linear_mx4(u8(2, 50), u8(2, 3), q, s, 16), lambda: w4.quantize_mx4(torch.zeros((4, 96), device=gpu)),
                 lambda: w4.quantize_tokens_mx4(torch.zeros((4, 96), device=gpu))):
        with pytest.raises(w4.W4Error, match="SHAPE"):
            call()
    # empty calls
    assert w4.linear_mx4(u8(0, 64), u8(0, 4), q, s, 16).shape == (0, 16)
    assert w4.linear_mx4(u8(2, 64), u8(2, 4), u8(0), u8(0), 0).shape == (2, 0)
    assert w4.quantize_tokens_mx4(torch.zeros((0, 128), device=gpu))[0].shape == (0, 64)


# ----------------------------------------------------------------------------
# larger sizes, which reach every kernel: against float64 on the GPU
# ----------------------------------------------------------------------------

def _draw(gpu, seed, rows, K, spread=6):
    g = torch.Generator(device=gpu)
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, device=gpu, dtype=torch.int32).to(torch.uint8)
    return codes, torch.randint(127 - spread, 128 + spread, (rows, K // 32), generator=g, device=gpu).to(torch.uint8)


def _values(codes, scales):
    """float64 values, by the table of E2M1."""
    grid = torch.tensor(list(oracle.E2M1) + [-v for v in oracle.E2M1], dtype=torch.float64, device=codes.device)
    v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).reshape(codes.shape[0], -1, 32)
    return (v * torch.exp2(scales.double() - 127)[..., None]).reshape(codes.shape[0], -1)


def _check_on_gpu(y32, x, w, K, what):
    ref, absdot = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    off = (y32.double() - ref).abs() - oracle.mx4_tolerance(absdot, K)
    assert bool((off <= 0).all()), f"{what}: {int((off > 0).sum())} of {off.numel()} out of tolerance"


@pytest.mark.parametrize("M,N,K", [
    (16, 2000, 4736), (9, 5000, 1152), (3, 9216, 2560), (13, 20000, 640),  # streamed: 1, 2 row blocks; 4, 2, 1 wavefronts
    (333, 1000, 640), (130, 520, 2560),                                    # streamed, many row tiles
    (33, 5000, 4736), (64, 5000, 1408),                                    # 32 x 64
    (333, 3000, 384), (300, 5000, 2560),                                   # 64 x 64
    (512, 2560, 9216),                                                     # 64 x 128
    (512, 9000, 1152), (2000, 3001, 1152),                                 # 128 x 128
    (1200, 2561, 1408),                                                    # 256 x 256, every tile cut
    (2100, 2561, 640), (3900, 5000, 1152), (2048, 9216, 128),              # whole and low ones; and cut ones
    (4096, 2048, 1408),                                                    # rows of whole lines
])
def test_linear_mx4_every_kernel(w4, gpu, M, N, K):
    _say(f"linear_mx4 {M} rows of {N}x{K}")
    wq, ws = _draw(gpu, M + N, N, K)
    xq, xs = _draw(gpu, K, M, K)
    q, s = w4.pack_mx4(wq, ws)
    buf = torch.full((M + 2, N), 77.0, device=gpu)
    y32 = w4.linear_mx4(xq, xs, q, s, N, out=buf[1:1 + M])
    assert _frame_kept(buf)
    _check_on_gpu(y32, _values(xq, xs), _values(wq, ws), K, "fp32")
    buf16, y16 = _framed(gpu, M, N, BF16)
    w4.linear_mx4(xq, xs, q, s, N, out=y16)
    assert _frame_kept(buf16) and torch.equal(y16, y32.to(BF16))


@pytest.mark.parametrize("sizes,N,K", [([700, 0, 1030, 257, 90], 2100, 640), ([3, 20, 41, 0, 64, 33, 17, 9], 1500, 1152),
                                       ([200, 100, 150, 130], 3000, 1408), ([1500, 1, 1300, 2], 1280, 896),
                                       ([20, 12, 0, 15, 9, 30, 17], 5000, 384),
                                       ([128, 100, 151, 140, 90, 133, 127, 161], 5120, 2560),
                                       ([31, 50, 0, 7, 40, 32], 5000, 2560)])
def test_grouped_linear_mx4_larger(w4, gpu, sizes, N, K):
    _say(f"grouped_linear_mx4 {sizes} {N}x{K}")
    E, first, after = len(sizes), 5, 3
    M = first + sum(sizes) + after
    offsets = torch.tensor([first] + [first + sum(sizes[:e + 1]) for e in range(E)], dtype=torch.int32, device=gpu)
    made = [_draw(gpu, 10 + e, N, K) for e in range(E)]
    packed = [w4.pack_mx4(*m) for m in made]
    q, s = torch.stack([p[0] for p in packed]), torch.stack([p[1] for p in packed])
    xq, xs = _draw(gpu, 9, M, K)
    buf = torch.full((M + 2, N), 77.0, device=gpu)
    y32 = w4.grouped_linear_mx4(xq, xs, offsets, q, s, N, out=buf[1:1 + M])
    assert _frame_kept(buf) and bool((y32[:first] == 77).all()) and bool((y32[M - after:] == 77).all())
    x = _values(xq, xs)
    at = first
    for e in range(E):
        if sizes[e]:
            _check_on_gpu(y32[at:at + sizes[e]], x[at:at + sizes[e]], _values(*made[e]), K, f"expert {e}")
        at += sizes[e]
    y16 = w4.grouped_linear_mx4(xq, xs, offsets, q, s, N)
    assert torch.equal(y16[first:M - after], y32[first:M - after].to(BF16))


def test_next_rows_do_not_matter(w4, gpu):
    """Where K ends inside 512 inputs, what follows a row of x (the next row: NaN scales, infinities' codes) and
    what follows the last one must not reach it."""
    _say("linear_mx4 rows beside rows of NaN")
    for K in (128, 384, 640, 1152, 1408):
        for M, N in ((16, 300), (40, 5000), (130, 5000), (600, 9000), (1500, 3000)):
            wq, ws = _draw(gpu, 1, N, K)
            xq, xs = _draw(gpu, 2, M, K)
            q, s = w4.pack_mx4(wq, ws)
            want = w4.linear_mx4(xq, xs, q, s, N)
            xs2 = xs.clone()
            xs2[1::2] = 255
            got = w4.linear_mx4(xq, xs2, q, s, N)
            assert torch.equal(got[0::2], want[0::2]) and bool(got[1::2].isnan().all()), (K, M, N)
