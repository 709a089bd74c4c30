"""8-bit and expert-grouped operators without a GPU: the oracle's own pins, the
refusals of the C entry points (each rejected on the host before any HIP call)
and those of the Python binding."""

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

def test_rows_ref_against_fractions():
    rng = np.random.default_rng(3)
    W = rng.standard_normal((6, 128)).astype(np.float32)
    W[1, 5] = np.float32(127.0)  # d = 1: codes are the rounded values themselves
    W[1, 6:10] = [2.5, -2.5, 0.5, -0.49999997]
    q, d = oracle.rtn_rows_ref(W)
    assert d[1] == 1.0 and q[1, 5:10].tolist() == [127, 3, -3, 1, 0]
    for n in range(6):
        a = max(abs(Fraction(float(v))) for v in W[n])
        assert abs(Fraction(float(d[n])) - a / 127) <= a / 127 / 2 ** 24  # half a step of fp32
        for k in range(128):
            t = Fraction(float(np.float32(W[n, k] / d[n])))
            want = int(abs(t) + Fraction(1, 2)) * (1 if t >= 0 else -1)
            assert int(q[n, k]) == want


def test_rows_ref_special_rows():
    W = np.zeros((5, 128), np.float32)
    W[1, 3] = np.nan
    W[2, 3] = -np.inf
    W[2, 4] = 5.0
    W[3, 0] = np.float32(1e-45)  # max / 127 underflows to zero
    W[4, 0] = np.float32(190 * 2.0 ** -149)  # d rounds to one subnormal step: the codes clamp
    W[4, 1] = np.float32(-190 * 2.0 ** -149)
    q, d = oracle.rtn_rows_ref(W)
    assert d[0] == 0 and not q[0].any()
    assert d[1:3].view(np.uint32).tolist() == [oracle.NAN_BITS] * 2 and not q[1:3].any()
    assert d[3] == 0 and not q[3].any()
    assert d[4] == np.float32(2.0 ** -149) and q[4, :3].tolist() == [127, -127, 0]


def test_w8a8_ref_against_integers():
    rng = np.random.default_rng(4)
    xq = rng.integers(-128, 128, (3, 256)).astype(np.int8)
    q = rng.integers(-128, 128, (5, 256)).astype(np.int8)
    sx, d = np.float32([0.5, 3.0, np.nan]), np.float32([1.0, 0.25, 0.0, 2.0, 1.5])
    y = oracle.w8a8_linear_ref(xq, sx, q, d)
    for m in range(2):
        for n in range(5):
            s = sum(int(a) * int(b) for a, b in zip(xq[m], q[n]))
            assert Fraction(float(y[m, n])) == s * Fraction(float(sx[m])) * Fraction(float(d[n]))
    assert np.isnan(y[2]).all()


def test_pack_ref_is_a_bijection():
    q = np.random.default_rng(5).integers(-128, 128, (37, 256)).astype(np.int8)
    p = oracle.pack_w8_ref(q)
    assert p.size == 48 * 256 and int(p.astype(np.int64).sum()) == int(q.astype(np.int64).sum())
    # the layout's words: byte 0 of lane 17 of tile (0, 0) is row 1, input 16
    assert p[17 * 16] == q[1, 16] and p[1024 + 3] == q[0, 67] and p[4 * 1024 + 2 * 16] == q[18, 0]


# ----------------------------------------------------------------------------
# C entry points
# ----------------------------------------------------------------------------

def test_w8_sizes(w4):
    lib = w4.library()
    assert lib.w4_w8_packed_bytes(2560, 9216) == 2560 * 9216
    assert lib.w4_w8_packed_bytes(37, 384) == 48 * 384
    assert lib.w4_w8_packed_bytes(0, 128) == 0
    assert lib.w4_w8_packed_bytes(1, 130944) == 16 * 130944
    for N, K in ((16, 100), (16, 0), (16, -128), (-1, 128), (16, 131072)):
        assert lib.w4_w8_packed_bytes(N, K) == 0


def test_w8_quantizer_refusals(w4):
    lib = w4.library()
    W, q, d = FAKE, FAKE + MiB, FAKE + 2 * MiB
    assert lib.w4_quantize_w8(W, 16, 100, q, d, None) == ERR_SHAPE
    assert lib.w4_quantize_w8(W, 16, 131072, q, d, None) == ERR_SHAPE
    assert lib.w4_quantize_w8(W, -1, 128, q, d, None) == ERR_SHAPE
    assert lib.w4_quantize_w8(None, 16, 128, q, d, None) == ERR_NULL
    assert lib.w4_quantize_w8(W, 16, 128, None, d, None) == ERR_NULL
    assert lib.w4_quantize_w8(W, 16, 128, q, None, None) == ERR_NULL
    assert lib.w4_quantize_w8(W + 4, 16, 128, q, d, None) == ERR_ALIGN
    assert lib.w4_quantize_w8(W, 16, 128, q + 8, d, None) == ERR_ALIGN
    assert lib.w4_quantize_w8(W, 16, 128, q, d + 2, None) == ERR_ALIGN
    assert lib.w4_quantize_w8(W, 16, 128, q, q + 1024, None) == ERR_ARG  # scales inside the codes
    assert lib.w4_quantize_w8(W, 1, 128, q, q + 512, None) == ERR_ARG    # the codes of one row fill 16
    assert lib.w4_quantize_w8(W, 16, 128, W + 64, d, None) == ERR_ARG
    assert lib.w4_quantize_w8(None, 0, 128, None, None, None) == OK
    for f, es in ((lib.w4_quantize_tokens, 2), (lib.w4_quantize_tokens_f32, 4)):
        assert f(W, 3, 100, q, d, None) == ERR_SHAPE
        assert f(W, -1, 128, q, d, None) == ERR_SHAPE
        assert f(W, 262141, 128, q, d, None) == ERR_SHAPE
        assert f(None, 3, 128, q, d, None) == ERR_NULL
        assert f(W, 3, 128, None, d, None) == ERR_NULL
        assert f(W, 3, 128, q, None, None) == ERR_NULL
        assert f(W + 8, 3, 128, q, d, None) == ERR_ALIGN
        assert f(W, 3, 128, q + 4, d, None) == ERR_ALIGN
        assert f(W, 3, 128, q, d + 1, None) == ERR_ALIGN
        assert f(W, 3, 128, W + 3 * 128 * es - 16, d, None) == ERR_ARG  # the last bytes of x
        assert f(W, 3, 128, q, q + 380, None) == ERR_ARG
        assert f(W, 3, 128, q, W + 4, None) == ERR_ARG
        assert f(None, 0, 128, None, None, None) == OK
    assert lib.w4_pack_w8(W, 16, 100, q, None) == ERR_SHAPE
    assert lib.w4_pack_w8(None, 16, 128, q, None) == ERR_NULL
    assert lib.w4_pack_w8(W + 8, 16, 128, q, None) == ERR_ALIGN
    assert lib.w4_pack_w8(W, 16, 128, W + 1024, None) == ERR_ARG
    assert lib.w4_unpack_w8(q, 16, 128, q + 2032, None) == ERR_ARG
    assert lib.w4_unpack_w8(q, -1, 128, W, None) == ERR_SHAPE
    assert lib.w4_unpack_w8(q, 1, 128, None, None) == ERR_NULL
    assert lib.w4_unpack_w8(None, 0, 128, None, None) == OK


def _w8a8(lib, grouped, f32, **kw):
    a = dict(x=FAKE, sx=FAKE + MiB, M=8, K=256, off=FAKE + 2 * MiB, E=4, q=FAKE + 3 * MiB, d=FAKE + 4 * MiB, N=32,
             y=FAKE + 5 * MiB)
    a.update(kw)
    name = "w4_linear_grouped_w8a8" if grouped else "w4_linear_w8a8"
    args = [a["x"], a["sx"], a["M"], a["K"]] + ([a["off"], a["E"]] if grouped else []) + [a["q"], a["d"], a["N"], a["y"]]
    return getattr(lib, name + ("_f32" if f32 else ""))(*args, None)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("grouped", [False, True])
def test_w8a8_refusals(w4, grouped, f32):
    lib = w4.library()
    call = lambda **kw: _w8a8(lib, grouped, f32, **kw)  # noqa: E731
    E, out = (4 if grouped else 1), (4 if f32 else 2)
    for bad in (dict(K=100), dict(K=0), dict(K=131072), dict(M=-1), dict(M=262141), dict(N=-1),
                dict(N=1 << 24, K=128, q=None)):  # the last: 2 GiB of codes
        assert call(**bad) == ERR_SHAPE, bad
    assert call(N=(1 << 24) - 16, K=128, q=None) == ERR_NULL
    for none in ("x", "sx", "q", "d", "y") + (("off",) if grouped else ()):
        assert call(**{none: None}) == ERR_NULL, none
    for bad in (dict(x=FAKE + 8), dict(q=FAKE + 3 * MiB + 8), dict(sx=FAKE + MiB + 2), dict(d=FAKE + 4 * MiB + 1),
                dict(y=FAKE + 5 * MiB + 1)) + ((dict(off=FAKE + 2 * MiB + 2),) if grouped else ()):
        assert call(**bad) == ERR_ALIGN, bad
    for bad in (dict(y=FAKE + 8 * 256 - out), dict(y=FAKE + MiB + 28), dict(y=FAKE + 3 * MiB + E * 32 * 256 - out),
                dict(y=FAKE + 4 * MiB + 4 * E * 32 - out)) + ((dict(y=FAKE + 2 * MiB + 16),) if grouped else ()):
        assert call(**bad) == ERR_ARG, bad
    # empty calls do nothing, whatever the pointers are
    assert call(M=0, x=None, y=None) == OK
    assert call(N=0, q=None, d=None, y=None) == OK
    if grouped:
        assert call(E=0, off=None) == OK
        assert call(E=-1) == ERR_SHAPE and call(E=4097) == ERR_SHAPE


@pytest.mark.parametrize("name,out,ds", [("w4_linear_grouped", 2, 4), ("w4_linear_grouped_s16", 2, 2),
                                         ("w4_linear_grouped_f32", 4, 4), ("w4_linear_grouped_f32_s16", 4, 2)])
def test_grouped_refusals(w4, name, out, ds):
    fn = getattr(w4.library(), name)

    def call(**kw):
        a = dict(x=FAKE, M=8, K=256, off=FAKE + 2 * MiB, E=4, q=FAKE + 3 * MiB, d=FAKE + 4 * MiB, N=32, y=FAKE + 5 * MiB)
        a.update(kw)
        return fn(a["x"], a["M"], a["K"], a["off"], a["E"], a["q"], a["d"], a["N"], a["y"], None)

    for bad in (dict(K=100), dict(K=(1 << 20) + 128), dict(M=-1), dict(M=262141), dict(N=-1), dict(E=-1), dict(E=4097),
                dict(N=1 << 23, K=512, q=None)):
        assert call(**bad) == ERR_SHAPE, bad
    assert call(N=(1 << 23) - 16, K=512, q=None) == ERR_NULL
    for none in ("x", "off", "q", "d", "y"):
        assert call(**{none: None}) == ERR_NULL, none
    for bad in (dict(x=FAKE + 8), dict(off=FAKE + 2 * MiB + 2), dict(q=FAKE + 3 * MiB + 8), dict(d=FAKE + 4 * MiB + 8),
                dict(y=FAKE + 5 * MiB + 1)):
        assert call(**bad) == ERR_ALIGN, bad
    codes, scales = 4 * 32 * 512 // 2, 4 * 32 * 4 * ds
    for bad in (dict(y=FAKE + 8 * 512 - out), dict(y=FAKE + 2 * MiB + 16), dict(y=FAKE + 3 * MiB + codes - out),
                dict(y=FAKE + 4 * MiB + scales - out)):
        assert call(**bad) == ERR_ARG, bad
    assert call(M=0, x=None) == OK and call(N=0, q=None) == OK and call(E=0, off=None) == OK


# ----------------------------------------------------------------------------
# Python binding
# ----------------------------------------------------------------------------

def test_binding_refuses_cpu_tensors_and_types(w4):
    x8, s = torch.zeros((2, 128), dtype=torch.int8), torch.zeros(2)
    q8, d8 = torch.zeros(16 * 128, dtype=torch.int8), torch.zeros(16)
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.quantize_w8(torch.zeros(16, 128))
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.quantize_tokens(torch.zeros(2, 128))
    with pytest.raises(TypeError):
        w4.quantize_tokens(torch.zeros(2, 128, dtype=torch.float16))
    with pytest.raises(TypeError):
        w4.quantize_w8(torch.zeros(128))
    with pytest.raises(ValueError, match="2-D"):
        w4.quantize_tokens(torch.zeros(128))
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.linear_w8a8(x8, s, q8, d8, 16)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.grouped_linear_w8a8(x8, s, off, q8, d8, 16)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.grouped_linear(torch.zeros((2, 128), dtype=torch.bfloat16), off, torch.zeros(4096, dtype=torch.uint8),
                          torch.zeros(64), 16)
    with pytest.raises(TypeError, match="offsets"):
        w4.grouped_linear_w8a8(x8, s, torch.zeros((1, 2), dtype=torch.int32), q8, d8, 16)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.pack_w8(x8)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.unpack_w8(q8, 16, 128)
    with pytest.raises(TypeError):
        w4.quantize_rtn_experts(torch.zeros(16, 128))
    assert w4.packed_bytes_w8(17, 256) == 32 * 256 and w4.packed_bytes_w8(17, 100) == 0
