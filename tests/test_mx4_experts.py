"""Microscaled 4-bit floating point and the way to the experts and back, without a GPU: the
oracle's own pins, the refusals of the C entry points (each rejected on the host
before any HIP call) and those of the Python binding."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_ARG = range(6)
FAKE = 0x10000000  # a 256-byte aligned address that is never dereferenced
MiB = 1 << 20


# ----------------------------------------------------------------------------
# oracle
# ----------------------------------------------------------------------------

def _nearest(v):
    """E2M1 code of a Fraction by trying all eight, ties to the even code."""
    grid = [Fraction(g) for g in (0, Fraction(1, 2), 1, Fraction(3, 2), 2, 3, 4, 6)]
    return min(range(8), key=lambda c: (abs(abs(v) - grid[c]), c % 2))


def test_mx4_quantize_ref_against_fractions():
    rng = np.random.default_rng(1)
    v = (rng.standard_normal((40, 64)) * 10.0 ** rng.integers(-30, 30, (40, 1))).astype(np.float32)
    v[3, :32] = 0.0
    v[4, 5] = np.float32(1e-44)  # a block whose largest member is subnormal, the others zeros
    v[4, :5] = v[4, 6:32] = 0.0
    v[5] = rng.integers(-48, 49, 64) / 8.0  # every tie of a block with scale 1
    v[5, 0] = v[5, 32] = 6.0
    v[6, :32] = np.float32(3.4e38)
    codes, scales = oracle.mx4_quantize_ref(v)
    for r in range(40):
        for b in range(2):
            block = [Fraction(float(x)) for x in v[r, 32 * b:32 * b + 32]]
            top = max(abs(x) for x in block)
            e = -127
            if top:
                e = 0
                while Fraction(2) ** e <= top:
                    e += 1
                while Fraction(2) ** e > top:
                    e -= 1
                e = max(e - 2, -127)
            assert int(scales[r, b]) == e + 127
            for k, x in enumerate(block):
                want = _nearest(x / Fraction(2) ** e) + (8 if np.signbit(v[r, 32 * b + k]) else 0)
                assert int(codes[r, 32 * b + k]) == want, (r, b, k)


def test_mx4_quantize_ref_non_finite():
    v = np.ones((3, 64), np.float32)
    v[0, 3], v[1, 40], v[2, 63] = np.nan, np.inf, -np.inf
    codes, scales = oracle.mx4_quantize_ref(v)
    assert scales.tolist() == [[255, 125], [125, 255], [125, 255]]
    assert not codes[0, :32].any() and (codes[0, 32:] == 6).all() and not codes[1:, 32:].any()
    assert np.isnan(oracle.mx4_values_ref(codes, scales)[0, :32]).all()


def test_mx4_linear_ref_against_fractions():
    rng = np.random.default_rng(2)
    xc, wc = rng.integers(0, 16, (3, 64)), rng.integers(0, 16, (4, 64))
    xs, ws = rng.integers(100, 150, (3, 2)), rng.integers(100, 150, (4, 2))
    y, a = oracle.mx4_linear_ref(xc, xs, wc, ws)
    grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    val = lambda c, s: Fraction(grid[c & 7]) * (-1 if c & 8 else 1) * Fraction(2) ** (int(s) - 127)  # noqa: E731
    for m in range(3):
        for n in range(4):
            terms = [val(int(xc[m, k]), xs[m, k // 32]) * val(int(wc[n, k]), ws[n, k // 32]) for k in range(64)]
            assert abs(Fraction(y[m, n]) - sum(terms)) <= sum(map(abs, terms)) * Fraction(64, 2 ** 53)
            assert abs(Fraction(a[m, n]) - sum(map(abs, terms))) <= sum(map(abs, terms)) * Fraction(64, 2 ** 53)
    ws[1, 0] = 255
    y, _ = oracle.mx4_linear_ref(xc, xs, wc, ws)
    assert np.isnan(y[:, 1]).all() and not np.isnan(y[:, [0, 2, 3]]).any()


def test_pack_mx4_ref_places():
    rng = np.random.default_rng(3)
    codes, scales = rng.integers(0, 16, (37, 640)).astype(np.uint8), rng.integers(0, 255, (37, 20)).astype(np.uint8)
    q, s = oracle.pack_mx4_ref(codes, scales)
    assert q.size == 48 * 768 // 2 and s.size == 48 * 1024 // 32
    assert int(s.astype(np.int64).sum()) == int(scales.astype(np.int64).sum())
    at = lambda c, k: c[k] | c[k + 1] << 4  # noqa: E731
    # row 18, input 64 + 32 + 6: row block 1, pair 0, lane 2 + 16, second tile, byte 3
    assert q[((1 * 3 + 0) * 2 + 1) * 1024 + 16 * 18 + 3] == at(codes[18], 64 + 32 + 6)
    # row 5, input 512 + 64: row block 0, pair 2, lane 5 + 16, first tile
    assert q[((0 * 3 + 2) * 2 + 0) * 1024 + 16 * 21] == at(codes[5], 576)
    # scales of row 5, inputs 256 + 128 + 32 ..: lane 5 + 32, fourth byte
    assert s[4 * 37 + 3] == scales[5, 13] and s[256 + 4 * 21] == scales[5, 18]


def test_expert_refs_agree_with_each_other():
    rng = np.random.default_rng(4)
    ids = rng.integers(-1, 6, (9, 3))
    offsets, place, order = oracle.expert_sort_ref(ids, 5)
    assert offsets[-1] == ((ids >= 0) & (ids < 5)).sum() == (order >= 0).sum() == (place >= 0).sum()
    for r, slot in enumerate(order):
        if slot >= 0:
            e = ids.reshape(-1)[slot]
            assert offsets[e] <= r < offsets[e + 1] and place.reshape(-1)[slot] == r
    for e in range(5):
        mine = order[offsets[e]:offsets[e + 1]]
        assert (np.diff(mine) > 0).all()
    # <take(x), g> = <x, combine(g)>, and the gradients of combine by differences
    x, g, w = rng.standard_normal((9, 7)), rng.standard_normal((27, 7)), rng.standard_normal((9, 3))
    xs = oracle.expert_take_ref(x, place)
    g[offsets[-1]:] = 0
    back, _ = oracle.expert_combine_ref(g, None, place)
    assert np.isclose((xs * g).sum(), (x * back).sum())
    dout = rng.standard_normal((9, 7))
    dy, dw, _ = oracle.expert_combine_backward_ref(dout, g, w, place)
    f = lambda y, w: (oracle.expert_combine_ref(y, w, place)[0] * dout).sum()  # noqa: E731
    # (bilinear: a difference is exact but for rounding)
    for r, k in ((0, 0), (3, 6), (26, 2)):
        p = g.copy()
        p[r, k] += 1.0
        assert np.isclose(f(p, w) - f(g, w), dy[r, k])
    for t, j in ((0, 0), (4, 2), (8, 1)):
        p = w.copy()
        p[t, j] += 1.0
        assert np.isclose(f(g, p) - f(g, w), dw[t, j])


# ----------------------------------------------------------------------------
# C entry points
# ----------------------------------------------------------------------------

def test_mx4_sizes(w4):
    lib = w4.library()
    assert lib.w4_mx4_packed_bytes(2560, 9216) == 2560 * 9216 // 2
    assert lib.w4_mx4_scale_bytes(2560, 9216) == 2560 * 9216 // 32
    assert lib.w4_mx4_packed_bytes(37, 384) == 48 * 512 // 2 and lib.w4_mx4_scale_bytes(37, 384) == 48 * 512 // 32
    assert lib.w4_mx4_packed_bytes(1, 640) == 16 * 768 // 2 and lib.w4_mx4_scale_bytes(1, 640) == 16 * 1024 // 32
    assert lib.w4_mx4_packed_bytes(0, 128) == 0
    for N, K in ((16, 100), (16, 32), (16, 0), (16, -128), (-1, 128), (16, 131072)):
        assert lib.w4_mx4_packed_bytes(N, K) == 0 and lib.w4_mx4_scale_bytes(N, K) == 0


@pytest.mark.parametrize("es", [2, 4])
def test_mx4_quantizer_refusals(w4, es):
    lib, wide = w4.library(), "_f32" if es == 4 else ""
    W, q, s = FAKE, FAKE + MiB, FAKE + 2 * MiB
    for name in ("w4_quantize_mx4", "w4_dequantize_mx4"):
        fn = getattr(lib, name + wide)
        call = lambda W=W, N=16, K=128, q=q, s=s: (  # noqa: E731
            fn(W, N, K, q, s, None) if name == "w4_quantize_mx4" else fn(q, s, N, K, W, None))
        for bad in (dict(K=100), dict(K=32), dict(K=131072), dict(N=-1)):
            assert call(**bad) == ERR_SHAPE
        for bad in (dict(W=None), dict(q=None), dict(s=None)):
            assert call(**bad) == ERR_NULL
        for bad in (dict(W=W + 8), dict(q=q + 8), dict(s=s + 8)):
            assert call(**bad) == ERR_ALIGN
        for bad in (dict(s=q + 2032), dict(q=W + 16 * 128 * es - 16), dict(s=W + 16 * 128 * es - 16),
                    dict(q=s + 240)):  # codes of K = 128 are padded to 256, scales to 512
            assert call(**bad) == ERR_ARG, bad
        assert call(N=0, W=None, q=None, s=None) == OK
    for name in ("w4_quantize_tokens_mx4", "w4_dequantize_tokens_mx4"):
        fn = getattr(lib, name + wide)
        call = lambda x=W, M=3, K=128, q=q, s=s: (  # noqa: E731
            fn(x, M, K, q, s, None) if name == "w4_quantize_tokens_mx4" else fn(q, s, M, K, x, None))
        for bad in (dict(K=100), dict(M=-1), dict(M=262141)):
            assert call(**bad) == ERR_SHAPE
        for bad in (dict(x=None), dict(q=None), dict(s=None)):
            assert call(**bad) == ERR_NULL
        for bad in (dict(x=W + 8), dict(q=q + 8), dict(s=s + 2)):
            assert call(**bad) == ERR_ALIGN
        for bad in (dict(q=W + 3 * 128 * es - 16), dict(s=q + 3 * 64 - 4), dict(s=W + 4), dict(q=s)):
            assert call(**bad) == ERR_ARG, bad
        assert call(M=0, x=None, q=None, s=None) == OK


def test_mx4_pack_refusals(w4):
    lib = w4.library()
    c, cs, q, s = FAKE, FAKE + MiB, FAKE + 2 * MiB, FAKE + 3 * MiB
    for pack in (True, False):
        call = lambda c=c, cs=cs, N=16, K=128, q=q, s=s: (  # noqa: E731
            lib.w4_pack_mx4(c, cs, N, K, q, s, None) if pack else lib.w4_unpack_mx4(q, s, N, K, c, cs, None))
        assert call(K=96) == ERR_SHAPE and call(N=-1) == ERR_SHAPE
        for bad in (dict(c=None), dict(cs=None), dict(q=None), dict(s=None)):
            assert call(**bad) == ERR_NULL
        for bad in (dict(c=c + 8), dict(q=q + 4), dict(s=s + 8)):
            assert call(**bad) == ERR_ALIGN
        for bad in (dict(q=c + 1008), dict(s=c + 16), dict(cs=q + 2040), dict(cs=s + 255)):
            assert call(**bad) == ERR_ARG, bad
        # the two outputs
        assert call(**(dict(s=q + 16) if pack else dict(cs=c + 1023))) == ERR_ARG
        assert call(N=0, c=None, cs=None, q=None, s=None) == OK


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("grouped", [False, True])
def test_linear_mx4_refusals(w4, grouped, f32):
    fn = getattr(w4.library(), "w4_linear_" + ("grouped_" if grouped else "") + "mx4" + ("_f32" if f32 else ""))

    def call(**kw):
        a = dict(x=FAKE, xs=FAKE + MiB, M=8, K=256, off=FAKE + 2 * MiB, E=4, q=FAKE + 3 * MiB, s=FAKE + 4 * MiB, N=32,
                 y=FAKE + 5 * MiB)
        a.update(kw)
        return fn(a["x"], a["xs"], a["M"], a["K"], *((a["off"], a["E"]) if grouped else ()), a["q"], a["s"], a["N"],
                  a["y"], None)

    E, out = (4 if grouped else 1), (4 if f32 else 2)
    for bad in (dict(K=100), dict(K=0), dict(K=131072), dict(M=-1), dict(M=262141), dict(N=-1),
                dict(N=1 << 24, K=256, q=None)):  # the last: 2 GiB of codes
        assert call(**bad) == ERR_SHAPE, bad
    assert call(N=(1 << 24) - 16, K=256, q=None) == ERR_NULL
    for none in ("x", "xs", "q", "s", "y") + (("off",) if grouped else ()):
        assert call(**{none: None}) == ERR_NULL, none
    for bad in (dict(x=FAKE + 8), dict(q=FAKE + 3 * MiB + 8), dict(xs=FAKE + MiB + 2), dict(s=FAKE + 4 * MiB + 4),
                dict(y=FAKE + 5 * MiB + 1)) + ((dict(off=FAKE + 2 * MiB + 2),) if grouped else ()):
        assert call(**bad) == ERR_ALIGN, bad
    for bad in (dict(y=FAKE + 8 * 128 - out), dict(y=FAKE + MiB + 60), dict(y=FAKE + 3 * MiB + E * 32 * 128 - out),
                dict(y=FAKE + 4 * MiB + E * 32 * 16 - out)) + ((dict(y=FAKE + 2 * MiB + 16),) if grouped else ()):
        assert call(**bad) == ERR_ARG, bad
    assert call(M=0, x=None, y=None) == OK and call(N=0, q=None, s=None, y=None) == OK
    if grouped:
        assert call(E=0, off=None) == OK
        assert call(E=-1) == ERR_SHAPE and call(E=4097) == ERR_SHAPE


def test_linear_mx4_of_too_many_threads_is_refused(w4):
    """A grid of 2^32 threads or more cannot be launched; none is needed while
    (M / 16 + min(experts, M)) * (N + 63) < 2^30."""
    fn = w4.library().w4_linear_grouped_mx4
    call = lambda M, E, N: fn(None, None, M, 128, None, E, None, None, N, None, None)  # noqa: E731
    assert call(4096, 4096, 1 << 23) == ERR_SHAPE
    for M, E in ((262140, 4096), (262140, 1), (100, 64)):
        N = (1 << 30) // (M // 16 + min(E, M) + 1) - 64
        N = min(N, (1 << 24) - 16)
        assert call(M, E, N) == ERR_NULL, (M, E, N)


def test_expert_sort_refusals(w4):
    lib = w4.library()
    assert lib.w4_expert_sort_workspace_bytes(10, 2, 8) == 0  # few slots
    need = lib.w4_expert_sort_workspace_bytes(10000, 2, 8)
    assert need >= 9 * 4 and need % 4 == 0  # the counts of a block at least
    for T, top, E in ((-1, 2, 8), (10, 0, 8), (262140, 2, 8), (131071, 3, 8), (10, 2, 4097), (10, 2, -1)):
        assert lib.w4_expert_sort_workspace_bytes(T, top, E) == 0
    ids, off, place, order, ws = (FAKE + i * MiB for i in range(5))

    def call(**kw):
        a = dict(ids=ids, size=8, T=10000, top=2, E=8, off=off, place=place, order=order, ws=ws, n=need)
        a.update(kw)
        return lib.w4_expert_sort(a["ids"], a["size"], a["T"], a["top"], a["E"], a["off"], a["place"], a["order"],
                                  a["ws"], a["n"], None)

    for bad in (dict(T=-1), dict(top=0), dict(T=262141, top=1), dict(T=1 << 62, top=4), dict(E=-1), dict(E=4097)):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in (dict(size=2), dict(size=0), dict(n=need - 1)):
        assert call(**bad) == ERR_ARG, bad
    for bad in (dict(ids=None), dict(off=None), dict(place=None), dict(order=None), dict(ws=None)):
        assert call(**bad) == ERR_NULL, bad
    for bad in (dict(ids=ids + 4), dict(off=off + 2), dict(place=place + 1), dict(order=order + 2), dict(ws=ws + 2)):
        assert call(**bad) == ERR_ALIGN, bad
    assert call(T=10, ws=None, off=None) == ERR_NULL
    for bad in (dict(off=ids + 159992), dict(place=off + 32), dict(order=place + 79996), dict(ws=order + 79996),
                dict(ws=ids - need + 4)):
        assert call(**bad) == ERR_ARG, bad
    assert call(ids=ids + 4, size=4, off=None) == ERR_NULL  # 4-byte ids need 4


def test_expert_row_refusals(w4):
    lib = w4.library()
    x, off, place, xs, w, out, dy, dw = (FAKE + i * MiB for i in range(8))
    take = lambda x=x, T=10, n=64, top=2, off=off, E=8, place=place, xs=xs: (  # noqa: E731
        lib.w4_expert_take(x, T, n, top, off, E, place, xs, None))
    for bad in (dict(T=-1), dict(top=0), dict(T=200000), dict(E=-1), dict(E=4097), dict(n=-1), dict(n=(1 << 26) + 1)):
        assert take(**bad) == ERR_SHAPE, bad
    for bad in (dict(x=None), dict(off=None), dict(place=None), dict(xs=None)):
        assert take(**bad) == ERR_NULL, bad
    assert take(off=off + 2) == ERR_ALIGN and take(place=place + 2) == ERR_ALIGN
    for bad in (dict(xs=x + 639), dict(xs=off + 35), dict(xs=place - 1279)):
        assert take(**bad) == ERR_ARG, bad
    assert take(T=0, x=None, xs=None) == OK and take(n=0, x=None, xs=None) == OK

    ws, need = FAKE + 9 * MiB, lib.w4_expert_sort_workspace_bytes(10000, 2, 8)
    ids, order = FAKE + 10 * MiB, FAKE + 11 * MiB
    dispatch = lambda x=x, n=10, ids=ids, size=8, T=10000, xs=xs, ws=ws, nb=need: (  # noqa: E731
        lib.w4_expert_dispatch(x, n, ids, size, T, 2, 8, off, place, order, xs, ws, nb, None))
    assert dispatch(n=-1) == ERR_SHAPE and dispatch(T=-1) == ERR_SHAPE and dispatch(size=3) == ERR_ARG
    assert dispatch(x=None) == ERR_NULL and dispatch(xs=None) == ERR_NULL and dispatch(ids=None) == ERR_NULL
    assert dispatch(nb=need - 1) == ERR_ARG and dispatch(ids=ids + 4) == ERR_ALIGN
    for bad in (dict(xs=x + 99999), dict(xs=off + 32), dict(xs=place + 79996), dict(xs=order + 79996), dict(xs=ws + 4),
                dict(xs=ids + 159996), dict(ws=x + 99996)):
        assert dispatch(**bad) == ERR_ARG, bad

    for yt in (0, 1):
        es = 4 if yt else 2
        comb = lambda y=x, yt=yt, w=w, wt=1, T=10, top=2, K=32, place=place, out=out, ot=yt: (  # noqa: E731
            lib.w4_expert_combine(y, yt, w, wt, T, top, K, place, out, ot, None))
        for bad in (dict(T=-1), dict(top=0), dict(T=200000), dict(K=-1), dict(K=(1 << 24) + 1)):
            assert comb(**bad) == ERR_SHAPE, bad
        for bad in (dict(yt=2), dict(wt=-1), dict(ot=7)):
            assert comb(**bad) == ERR_ARG, bad
        for bad in (dict(y=None), dict(place=None), dict(out=None)):
            assert comb(**bad) == ERR_NULL, bad
        for bad in (dict(y=x + 1), dict(w=w + 2), dict(place=place + 2), dict(out=out + 1)):
            assert comb(**bad) == ERR_ALIGN, bad
        for bad in (dict(out=x + 20 * 32 * es - es), dict(out=w + 76), dict(out=place + 76)):
            assert comb(**bad) == ERR_ARG, bad
        assert comb(T=0, y=None, place=None, out=None) == OK and comb(K=0, y=None, out=None) == OK

        back = lambda g=out, ot=yt, y=x, yt=yt, w=w, wt=1, T=10, top=2, K=32, off=off, E=8, place=place, dy=dy, dw=dw: (  # noqa: E731
            lib.w4_expert_combine_backward(g, ot, y, yt, w, wt, T, top, K, off, E, place, dy, dw, None))
        for bad in (dict(T=-1), dict(top=0), dict(T=200000), dict(K=-1), dict(E=-1), dict(E=4097)):
            assert back(**bad) == ERR_SHAPE, bad
        for bad in (dict(yt=2), dict(wt=-1), dict(ot=7)):
            assert back(**bad) == ERR_ARG, bad
        for bad in (dict(g=None), dict(y=None), dict(place=None), dict(off=None)):
            assert back(**bad) == ERR_NULL, bad
        for bad in (dict(g=out + 1), dict(y=x + 1), dict(w=w + 2), dict(place=place + 2), dict(off=off + 2),
                    dict(dy=dy + 1), dict(dw=dw + 2)):
            assert back(**bad) == ERR_ALIGN, bad
        for bad in (dict(dy=x + 20 * 32 * es - es), dict(dy=dw - 4), dict(dw=w + 76), dict(dw=place + 76),
                    dict(dy=out + 10 * 32 * es - es), dict(dw=off + 32)):
            assert back(**bad) == ERR_ARG, bad
        assert back(dy=None, dw=None) == OK and back(T=0, g=None, y=None) == OK


# ----------------------------------------------------------------------------
# Python binding
# ----------------------------------------------------------------------------

def test_binding_refuses_cpu_tensors_and_types(w4):
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)  # noqa: E731
    off = torch.zeros(2, dtype=torch.int32)
    cpu = "GPU tensor"
    for call in (lambda: w4.quantize_mx4(torch.zeros(16, 128)), lambda: w4.quantize_tokens_mx4(torch.zeros(2, 128)),
                 lambda: w4.dequantize_mx4(u8(2048), u8(256), 16, 128),
                 lambda: w4.dequantize_tokens_mx4(u8(2, 64), u8(2, 4)),
                 lambda: w4.pack_mx4(u8(16, 64), u8(16, 4)), lambda: w4.unpack_mx4(u8(2048), u8(256), 16, 128),
                 lambda: w4.linear_mx4(u8(2, 64), u8(2, 4), u8(2048), u8(256), 16),
                 lambda: w4.grouped_linear_mx4(u8(2, 64), u8(2, 4), off, u8(1, 2048), u8(1, 256), 16),
                 lambda: w4.expert_sort(torch.zeros((4, 2), dtype=torch.int64), 4),
                 lambda: w4.expert_take(torch.zeros(4, 8), w4.ExpertRows(off, off, off)),
                 lambda: w4.expert_dispatch(torch.zeros(4, 8), torch.zeros((4, 2), dtype=torch.int64), 4),
                 lambda: w4.expert_combine(torch.zeros(8, 8), None, w4.ExpertRows(off, off, off))):
        with pytest.raises(ValueError, match=cpu):
            call()
    for call in (lambda: w4.quantize_mx4(torch.zeros(128)), lambda: w4.quantize_mx4(torch.zeros(16, 128).half()),
                 lambda: w4.quantize_tokens_mx4(torch.zeros(2, 128).half()), lambda: w4.quantize_mx4([1.0]),
                 lambda: w4.linear_mx4(torch.zeros(2, 64), u8(2, 4), u8(2048), u8(256), 16),
                 lambda: w4.expert_sort(torch.zeros((4, 2)), 4), lambda: w4.expert_take(torch.zeros(4, 8).half(), None),
                 lambda: w4.expert_combine(torch.zeros(8, 8).half(), None, None),
                 lambda: w4.grouped_linear_mx4(u8(2, 64), u8(2, 4), torch.zeros((1, 2), dtype=torch.int32), u8(1, 2048),
                                               u8(1, 256), 16),
                 lambda: w4.MX4Linear.from_float(torch.zeros(2, 16, 128))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="2-D"):
        w4.quantize_tokens_mx4(torch.zeros(128))
    with pytest.raises(ValueError, match="2-D"):
        w4.expert_sort(torch.zeros(4, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="1-D or 2-D"):
        w4.expert_take(torch.zeros(4, 2, 2), None)
    assert w4.packed_bytes_mx4(17, 384) == 32 * 256 and w4.scale_bytes_mx4(17, 384) == 32 * 16
    assert w4.packed_bytes_mx4(17, 100) == 0 and w4.scale_bytes_mx4(17, 100) == 0
