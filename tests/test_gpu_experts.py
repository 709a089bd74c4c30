"""Rows to the experts and back on an MI355X, against the oracle.

Offsets, places, order and moved rows are compared bit for bit.  out = sum_j w y adds
`top` rounded products in fp32: within (top + 1) * 2^-24 of sum |w y|, then rounded once
to bf16 where that is its type.  dy is one rounded product (half a step of its type); dw
lies within (K / 64 + 16) * 2^-24 of sum |dout y| before it is rounded to its type.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TINY = 2.0 ** -126  # below this an fp32 step is no longer relative


def _say(msg):
    print(f"\n[case] {msg}", flush=True)


def _bits(y):
    y = y.detach().cpu()
    return y.numpy().view(np.uint32) if y.dtype == F32 else y.view(torch.int16).numpy().view(np.uint16)


def check(y, ref, tol, what):
    """y is the rounding to its type of a value within tol of ref."""
    ok = oracle.admissible(_bits(y), ref, tol, "f32" if y.dtype == F32 else "bf16", rel=1.0, abs_=TINY)
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} out of tolerance"


def same_bits(a, b):
    return a.shape == b.shape and np.array_equal(_bits(a), _bits(b))


def _ids(rng, T, top, E, kind):
    if kind == "random":
        ids = rng.integers(0, max(E, 1), (T, top))
    elif kind == "distinct":
        ids = np.stack([rng.permutation(E)[:top] for _ in range(T)]) if T else np.zeros((0, top), np.int64)
    elif kind == "dropped":
        ids = rng.integers(-2, E + 2, (T, top))
        ids[T // 2:T // 2 + 3] = -1
    elif kind == "one":
        ids = np.full((T, top), E - 1)
    elif kind == "none":
        ids = np.full((T, top), -1)
    else:  # far ids, which 32 bits would bring back into range
        ids = rng.integers(0, E, (T, top)) + (rng.integers(0, 2, (T, top)) << 32)
    return ids.astype(np.int64)


def _check_rows(rows, ids, E):
    offsets, place, order = oracle.expert_sort_ref(ids, E)
    assert np.array_equal(rows.offsets.cpu().numpy(), offsets), "offsets"
    assert np.array_equal(rows.place.cpu().numpy(), place), "place"
    assert np.array_equal(rows.order.cpu().numpy(), order), "order"
    return place


SORTS = [(0, 2, 8), (0, 100, 8), (1, 65, 300), (2, 64, 64), (2, 65, 64), (128, 8, 9), (129, 8, 9), (16384, 8, 128), (16385, 8, 128), (1, 1, 1), (1, 8, 128), (8, 2, 64), (5, 3, 0), (77, 3, 7), (64, 4, 300), (128, 8, 64), (300, 6, 4096),
         (333, 1, 5), (1111, 2, 33), (4095, 8, 128), (32768, 1, 2), (32767, 8, 256), (87380, 3, 4096)]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("T,top,E", SORTS)
def test_expert_sort(w4, gpu, T, top, E, wide):
    rng = np.random.default_rng(T + E)
    kinds = ["random", "dropped", "none"] + (["one"] if E else []) + (["far"] if wide and E else [])
    if T <= 4095 and top <= E:
        kinds.append("distinct")
    for kind in kinds:
        _say(f"expert_sort {T} x {top} of {E}, {kind}")
        ids = _ids(rng, T, top, E, kind)
        t = torch.from_numpy(ids).to(gpu)
        _check_rows(w4.expert_sort(t if wide else t.to(torch.int32), E), ids, E)


def test_expert_sort_extreme_ids(w4, gpu):
    _say("expert_sort extreme ids")
    for dtype in (torch.int64, torch.int32):
        i = torch.iinfo(dtype)
        ids = np.array([[i.min, 0, i.max], [3, 4, -1], [2, 3, 1]], np.int64)
        _check_rows(w4.expert_sort(torch.from_numpy(ids).to(dtype).to(gpu), 4), ids, 4)


DTYPES = {"bf16": BF16, "f32": F32, "u8": torch.uint8, "i8": torch.int8}


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("T,top,E,K", [(1, 1, 1, 1), (8, 2, 64, 2560), (9, 3, 5, 77), (40, 4, 16, 7), (33, 8, 64, 1409),
                                       (200, 2, 9, 130), (1200, 3, 16, 640), (2000, 3, 40, 16), (1500, 8, 128, 33), (3, 2, 4, 20000)])
def test_dispatch_and_take(w4, gpu, T, top, E, K, dtype):
    rng = np.random.default_rng(T + K)
    for kind in ("random", "dropped", "none"):
        _say(f"dispatch {T} x {top} of {E}, {K} {dtype}, {kind}")
        ids = _ids(rng, T, top, E, kind)
        x = torch.from_numpy(rng.integers(-100, 100, (T, K))).to(DTYPES[dtype])
        # rows that start anywhere their type may
        held = torch.zeros(T * K + 3, dtype=x.dtype, device=gpu)
        xg = held[3:].view(T, K)
        xg.copy_(x)
        xs, rows = w4.expert_dispatch(xg, torch.from_numpy(ids).to(gpu), E)
        place = _check_rows(rows, ids, E)
        want = oracle.expert_take_ref(x.float().numpy(), place)
        assert np.array_equal(xs.float().cpu().numpy(), want)
        obuf = torch.full((T * top * K + 2,), 9, dtype=x.dtype, device=gpu)
        out = obuf[1:-1].view(T * top, K)
        assert w4.expert_take(xg, rows, out=out) is out
        assert np.array_equal(out.float().cpu().numpy(), want)
        assert float(obuf[0]) == 9 and float(obuf[-1]) == 9


def test_take_of_scales(w4, gpu):
    """One value a token: the scales of 8-bit activations."""
    _say("take of a vector")
    rng = np.random.default_rng(2)
    ids = _ids(rng, 50, 4, 8, "dropped")
    rows = w4.expert_sort(torch.from_numpy(ids).to(gpu), 8)
    sx = rng.standard_normal(50).astype(np.float32)
    got = w4.expert_take(torch.from_numpy(sx).to(gpu), rows)
    assert np.array_equal(got.cpu().numpy(), oracle.expert_take_ref(sx, rows.place.cpu().numpy()))


COMBINES = [(1, 1, 1, 1), (1200, 3, 16, 640), (1100, 2, 16, 1027), (8, 2, 64, 2560), (9, 3, 5, 77), (40, 4, 16, 7), (33, 8, 64, 1409), (200, 2, 9, 130), (70, 10, 20, 264),
            (1500, 8, 128, 33), (3, 2, 4, 20000), (500, 1, 8, 512), (2, 70, 100, 100)]


def _combine_inputs(rng, gpu, T, top, E, K, yt, wt, kind):
    ids = _ids(rng, T, top, E, kind)
    rows = w4_rows(gpu, ids, E)
    y = torch.from_numpy(rng.standard_normal((T * top, K)).astype(np.float32)).to(yt)
    y[int(rows.offsets[E]):] = float("nan")  # rows of no slot may hold anything
    w = torch.from_numpy(rng.standard_normal((T, top)).astype(np.float32)).to(wt)
    w[rows.place.cpu() < 0] = float("nan")   # and so may weights of dropped slots
    return rows, y, w


def w4_rows(gpu, ids, E):
    import bit_group_quantized_w4_amd as w4

    return w4.ExpertRows(*(torch.from_numpy(v).to(gpu) for v in oracle.expert_sort_ref(ids, E)))


def _np(t):
    return np.nan_to_num(t.detach().float().cpu().numpy()).astype(np.float64)  # (NaN only where nothing reads it)


@pytest.mark.parametrize("yt,wt", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,top,E,K", COMBINES)
def test_combine(w4, gpu, T, top, E, K, yt, wt):
    rng = np.random.default_rng(T + K)
    for kind in ("random", "dropped"):
        _say(f"combine {T} x {top} of {E}, {K} {yt} {wt}, {kind}")
        rows, y, w = _combine_inputs(rng, gpu, T, top, E, K, yt, wt, kind)
        place = rows.place.cpu().numpy()
        held = torch.zeros(T * top * K + 3, dtype=yt, device=gpu)
        yg = held[3:].view(T * top, K)
        yg.copy_(y)
        for weights in (w, None):
            ref, a = oracle.expert_combine_ref(_np(y), None if weights is None else _np(w), place)
            for ot in (BF16, F32):
                obuf = torch.full((T * K + 2,), 9.0, dtype=ot, device=gpu)
                out = obuf[1:-1].view(T, K)
                w4.expert_combine(yg, None if weights is None else w.to(gpu), rows, out=out)
                check(out, ref, (top + 1) * 2.0 ** -24 * a, "out")
                assert float(obuf[0]) == 9 and float(obuf[-1]) == 9
        assert w4.expert_combine(yg, w.to(gpu), rows).dtype == yt
        assert w4.expert_combine(yg, w.to(gpu), rows, out_dtype=F32).dtype == F32


def _check_gradients(dy, dw, dout, y, w, place, K):
    yz = torch.nan_to_num(y.float()).cpu()
    wz = None if w is None else torch.nan_to_num(w.float()).cpu()
    ry, rw, a = oracle.expert_combine_backward_ref(_np(dout), _np(yz), None if w is None else _np(wz), place)
    if dy is not None:
        check(dy, ry, 2.0 ** -24 * np.abs(ry), "dy")
    if dw is not None:
        check(dw, rw, (K / 64 + 16) * 2.0 ** -24 * a, "dw")


@pytest.mark.parametrize("yt,wt,ot", [(BF16, F32, BF16), (BF16, BF16, F32), (F32, F32, F32), (F32, BF16, BF16)])
@pytest.mark.parametrize("T,top,E,K", COMBINES)
def test_combine_backward(w4, gpu, T, top, E, K, yt, wt, ot):
    rng = np.random.default_rng(T + K)
    for kind in ("random", "dropped"):
        _say(f"combine backward {T} x {top} of {E}, {K} {yt} {wt} {ot}, {kind}")
        rows, y, w = _combine_inputs(rng, gpu, T, top, E, K, yt, wt, kind)
        place = rows.place.cpu().numpy()
        dout = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(ot)
        yg, wg, dg = y.to(gpu), w.to(gpu), dout.to(gpu)
        dy, dw = w4.expert_combine_backward(dg, yg, wg, rows)
        assert dy.dtype == yt and dw.dtype == wt
        _check_gradients(dy, dw, dout, y, w, place, K)
        only, none = w4.expert_combine_backward(dg, yg, wg, rows, need_weights=False)
        assert none is None and same_bits(only, dy)
        none, only = w4.expert_combine_backward(dg, yg, wg, rows, need_y=False)
        assert none is None and same_bits(only, dw)
        dy, dw = w4.expert_combine_backward(dg, yg, None, rows)
        assert dw is None
        _check_gradients(dy, None, dout, y, None, place, K)


def test_gradients_by_autograd(w4, gpu):
    """backward() of dispatch, take and combine, with leaves that need it or not, and a gradient that is not
    contiguous."""
    _say("autograd")
    rng = np.random.default_rng(12)
    T, top, E, K = 60, 3, 7, 130
    ids = _ids(rng, T, top, E, "dropped")
    place = oracle.expert_sort_ref(ids, E)[1]
    idg = torch.from_numpy(ids).to(gpu)
    for dtype in (BF16, F32):
        x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(dtype).to(gpu).requires_grad_()
        g = torch.from_numpy(rng.standard_normal((T * top, K)).astype(np.float32)).to(dtype).to(gpu)
        ref, a = oracle.expert_combine_ref(_np(g), None, place)
        xs, rows = w4.expert_dispatch(x, idg, E)
        assert isinstance(rows, w4.ExpertRows) and not rows.place.requires_grad
        for out in (xs, w4.expert_take(x, rows)):
            x.grad = None
            out.backward(g)
            check(x.grad, ref, (top + 1) * 2.0 ** -24 * a, "dx")
        x.grad = None
        w4.expert_take(x, rows).backward(torch.ones((K, T * top), dtype=dtype, device=gpu).t())
        assert torch.equal(x.grad, (rows.place >= 0).sum(1, keepdim=True).to(dtype).expand(T, K))
        with torch.no_grad():
            assert not w4.expert_take(x, rows).requires_grad
        for need in ((True, True), (True, False), (False, True)):
            y = g.clone().requires_grad_(need[0])
            w = torch.rand((T, top), device=gpu).requires_grad_(need[1])
            dout = torch.randn((T, K), device=gpu).to(dtype)
            w4.expert_combine(y, w, rows).backward(dout)
            assert (y.grad is not None, w.grad is not None) == need
            _check_gradients(y.grad, w.grad, dout, y, w, place, K)
        y = g.clone().requires_grad_()
        w4.expert_combine(y, None, rows, out_dtype=F32).sum().backward()
        assert torch.equal(y.grad[:int(rows.offsets[E])], torch.ones_like(y.grad[:int(rows.offsets[E])]))
        assert not bool(y.grad[int(rows.offsets[E]):].any())


def test_gradients_by_differences(w4, gpu):
    """The loss is linear in y and in w: a difference over a step of 1 is the gradient, but for rounding."""
    _say("differences")
    rng = np.random.default_rng(13)
    T, top, E, K = 12, 2, 5, 40
    rows, y, w = _combine_inputs(rng, gpu, T, top, E, K, F32, F32, "random")
    y, w = y.to(gpu).requires_grad_(), w.to(gpu).requires_grad_()
    c = torch.randn((T, K), device=gpu)
    loss = lambda y, w: float((w4.expert_combine(y, w, rows).double() * c.double()).sum())  # noqa: E731
    (w4.expert_combine(y, w, rows) * c).sum().backward()
    # fp32 outputs of about 80 terms up to 4 each, 480 of them added in fp64: errors below 480 * 2^-24 * 16
    tol = 480 * 2.0 ** -24 * 16 * 2
    with torch.no_grad():
        for r, k in ((0, 0), (7, 39), (23, 11)):
            p = y.clone()
            p[r, k] += 1.0
            assert abs(loss(p, w) - loss(y, w) - float(y.grad[r, k])) < tol
        for t, j in ((0, 0), (5, 1), (11, 1)):
            p = w.clone()
            p[t, j] += 1.0
            assert abs(loss(y, p) - loss(y, w) - float(w.grad[t, j])) < tol


def test_wrong_places_stay_inside(w4, gpu):
    """Places and offsets that no sort wrote: rows outside the buffers are neither read nor written."""
    _say("wrong places")
    T, top, E, K = 20, 2, 4, 100
    place = torch.tensor([[-2 ** 31, 40], [39, 2 ** 31 - 1]] * 10, dtype=torch.int32, device=gpu)
    for end in (-5, 1000, 2 ** 31 - 1):
        rows = w4.ExpertRows(torch.full((E + 1,), end, dtype=torch.int32, device=gpu), place, place.reshape(-1))
        buf = torch.full((T * top + 2, K), 9.0, device=gpu)
        w4.expert_take(torch.ones((T, K), device=gpu), rows, out=buf[1:-1])
        torch.cuda.synchronize()
        assert bool((buf[0] == 9).all()) and bool((buf[-1] == 9).all())
        y = torch.full((T * top, K), 2.0, device=gpu)
        out = w4.expert_combine(y, None, rows)
        assert bool((out[1::2] == 2).all()) and not bool(out[0::2].any())
        dy, dw = w4.expert_combine_backward(torch.ones((T, K), device=gpu), y, torch.ones((T, top), device=gpu), rows)
        assert torch.equal(dw, torch.tensor([[0.0, 0.0], [2.0 * K, 0.0]] * 10, device=gpu))


def test_capture_and_streams(w4, gpu):
    """Captured and replayed with other choices and values between, every replay against the eager call; two
    graphs in flight on two streams."""
    _say("capture")
    rng = np.random.default_rng(14)
    for T, top, E, K in ((8, 2, 64, 320), (700, 4, 16, 130)):
        choices = [torch.from_numpy(_ids(rng, T, top, E, "dropped")).to(gpu) for _ in range(3)]
        inputs = [torch.randn((T, K), device=gpu).to(BF16) for _ in range(3)]
        w = torch.rand((T, top), device=gpu)

        def layer(x, ids):
            xs, rows = w4.expert_dispatch(x, ids, E)
            y = w4.expert_combine(xs, w, rows)
            dy, dw = w4.expert_combine_backward(x, xs, w, rows)
            return [rows.offsets, rows.place, rows.order, xs, y, dy, dw]

        want = [layer(x, i) for x, i in zip(inputs, choices)]
        held = [(inputs[0].clone(), choices[0].clone()) for _ in range(2)]
        graphs, outs = [], []
        for x, ids in held:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(layer(x, ids))
            graphs.append(graph)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for turn in range(6):
            for k in range(2):
                streams[k].wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(streams[k]):
                    held[k][0].copy_(inputs[(turn + k) % 3])
                    held[k][1].copy_(choices[(turn + k) % 3])
                    graphs[k].replay()
            torch.cuda.synchronize()
            for k in range(2):
                for a, b in zip(outs[k], want[(turn + k) % 3]):
                    assert torch.equal(a, b)


def test_an_expert_layer(w4, gpu):
    """The operators as they are used: tokens sorted by expert, quantized, multiplied with two 4-bit
    floating-point weights with an activation between, and brought back."""
    _say("expert layer")
    g = torch.Generator(device=gpu)
    g.manual_seed(5)
    T, top, E, H, F = 45, 2, 6, 256, 384
    x = torch.randn((T, H), generator=g, device=gpu).to(BF16)
    up = torch.randn((E, 2 * F, H), generator=g, device=gpu) * 0.05
    down = torch.randn((E, H, F), generator=g, device=gpu).to(BF16) * 0.05
    weights, ids = torch.softmax(torch.randn((T, E), generator=g, device=gpu), 1).topk(top, dim=1)
    ids = ids.clone()
    ids[40:] = -1  # padding
    upq, downq = w4.quantize_mx4(up), w4.quantize_mx4(down)
    xs, rows = w4.expert_dispatch(x, ids, E)
    h = w4.grouped_linear_mx4(*w4.quantize_tokens_mx4(xs), rows.offsets, *upq, 2 * F, out_dtype=F32)
    a = (torch.nn.functional.silu(h[:, :F]) * h[:, F:]).to(BF16)
    y = w4.grouped_linear_mx4(*w4.quantize_tokens_mx4(a), rows.offsets, *downq, H)
    out = w4.expert_combine(y, weights, rows)
    assert not bool(out[40:].any())

    # the same, token by token, each step from the step before's own outputs
    upc = [oracle.mx4_quantize_ref(up[e].cpu().numpy()) for e in range(E)]
    downc = [oracle.mx4_quantize_ref(down[e].float().cpu().numpy()) for e in range(E)]
    place = rows.place.cpu().numpy()
    for t in range(40):
        xc = oracle.mx4_quantize_ref(x[t:t + 1].float().cpu().numpy())
        for j in range(top):
            e, r = int(ids[t, j]), int(place[t, j])
            ref, ab = oracle.mx4_linear_ref(*xc, *upc[e])
            check(h[r:r + 1], ref, oracle.mx4_tolerance(ab, H), "up")
            ref, ab = oracle.mx4_linear_ref(*oracle.mx4_quantize_ref(a[r:r + 1].float().cpu().numpy()), *downc[e])
            check(y[r:r + 1], ref, oracle.mx4_tolerance(ab, F), "down")
    ref, ab = oracle.expert_combine_ref(_np(y), _np(weights), place)
    check(out, ref, (top + 1) * 2.0 ** -24 * ab, "out")

    # codes and scales taken by row are the codes and scales of the rows
    xq, xsc = w4.quantize_tokens_mx4(x)
    q2, s2 = w4.quantize_tokens_mx4(xs)
    n = int(rows.offsets[E])
    assert torch.equal(w4.expert_take(xq, rows)[:n], q2[:n]) and torch.equal(w4.expert_take(xsc, rows)[:n], s2[:n])
    # and the other formats take the same rows
    q8, d8 = w4.quantize_w8(up)
    y8 = w4.grouped_linear_w8a8(*w4.quantize_tokens(xs), rows.offsets, q8, d8, 2 * F)
    x8, sx = w4.quantize_tokens(x)
    z8 = w4.grouped_linear_w8a8(w4.expert_take(x8, rows), w4.expert_take(sx, rows), rows.offsets, q8, d8, 2 * F)
    assert torch.equal(y8[:n], z8[:n])


def test_refusals_on_the_gpu(w4, gpu):
    ids = torch.zeros((4, 2), dtype=torch.int64, device=gpu)
    rows = w4.expert_sort(ids, 3)
    x, y, w = torch.zeros((4, 8), device=gpu), torch.zeros((8, 8), device=gpu), torch.zeros((4, 2), device=gpu)
    for call in (lambda: w4.expert_take(torch.zeros((5, 8), device=gpu), rows),
                 lambda: w4.expert_take(x, rows, out=torch.zeros((8, 9), device=gpu)),
                 lambda: w4.expert_take(torch.zeros((4, 16), device=gpu)[:, ::2], rows),
                 lambda: w4.expert_dispatch(torch.zeros((5, 8), device=gpu), ids, 3),
                 lambda: w4.expert_combine(torch.zeros((7, 8), device=gpu), w, rows),
                 lambda: w4.expert_combine(y, torch.zeros((8, 2), device=gpu), rows),
                 lambda: w4.expert_combine(y, w, rows, out=torch.zeros((8, 8), device=gpu)),
                 lambda: w4.expert_combine_backward(torch.zeros((5, 8), device=gpu), y, w, rows),
                 lambda: w4.expert_combine_backward(x, torch.zeros((8, 9), device=gpu), w, rows),
                 lambda: w4.expert_sort(torch.zeros((4, 4), dtype=torch.int64, device=gpu)[:, ::2], 3),
                 lambda: w4.expert_take(torch.zeros(4, device=gpu).requires_grad_(), rows)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: w4.expert_take(x, tuple(rows)), lambda: w4.expert_combine(y, w.half(), rows),
                 lambda: w4.expert_combine(y, w, rows, out_dtype=torch.float16),
                 lambda: w4.expert_take(x, rows._replace(place=rows.place.long()))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: w4.expert_sort(ids, -1), lambda: w4.expert_sort(ids, 4097),
                 lambda: w4.expert_sort(torch.zeros((4, 0), dtype=torch.int64, device=gpu), 4),
                 lambda: w4.expert_sort(torch.zeros((131071, 3), dtype=torch.int32, device=gpu), 4)):
        with pytest.raises(w4.W4Error, match="SHAPE"):
            call()
    # no tokens, and rows of no values
    none = w4.expert_dispatch(torch.zeros((0, 8), device=gpu), torch.zeros((0, 2), dtype=torch.int64, device=gpu), 3)
    assert none[0].shape == (0, 8) and none[1].offsets.tolist() == [0, 0, 0, 0]
    assert w4.expert_combine(none[0], None, none[1]).shape == (0, 8)
    assert w4.expert_take(torch.zeros((4, 0), device=gpu), rows).shape == (8, 0)
    dy, dw = w4.expert_combine_backward(torch.zeros((4, 0), device=gpu), torch.zeros((8, 0), device=gpu),
                                        torch.ones((4, 2), device=gpu), rows)
    assert dy.shape == (8, 0) and not bool(dw.any())


def test_capture_of_a_backward_pass(w4, gpu):
    """Forward and backward of dispatch and combine in one graph, replayed with other values between."""
    _say("captured backward pass")
    rng = np.random.default_rng(15)
    T, top, E, K = 50, 2, 6, 136
    ids = torch.from_numpy(_ids(rng, T, top, E, "dropped")).to(gpu)

    def step(x, w, dout):
        xs, rows = w4.expert_dispatch(x, ids, E)
        return torch.autograd.grad(w4.expert_combine(xs * 2.0, w, rows), (x, w), dout)

    values = [(torch.randn((T, K), device=gpu), torch.rand((T, top), device=gpu), torch.randn((T, K), device=gpu))
              for _ in range(3)]
    want = [[g.clone() for g in step(x.clone().requires_grad_(), w.clone().requires_grad_(), d)] for x, w, d in values]
    x, w, d = (v.clone() for v in values[0])
    xg, wg = x.requires_grad_(), w.requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(xg, wg, d)
    for turn in range(6):
        k = turn % 3
        with torch.no_grad():
            xg.copy_(values[k][0]), wg.copy_(values[k][1]), d.copy_(values[k][2])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[k]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,top,E,K", [(9, 3, 5, 7), (9, 3, 5, 77), (40, 4, 16, 264), (300, 10, 16, 1027), (1100, 2, 16, 1024)])
@pytest.mark.parametrize("yt", [BF16, F32])
def test_gradients_of_infinite_outputs(w4, gpu, T, top, E, K, yt):
    """Dropped slots have zeros as gradients of their weights, whatever the gradient of the output holds."""
    rng = np.random.default_rng(T + K)
    _say(f"gradients of infinite outputs {T} x {top} of {E}, {K}")
    ids = _ids(rng, T, top, E, "dropped")
    rows, y, w = _combine_inputs(rng, gpu, T, top, E, K, yt, F32, "dropped")
    g = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32))
    g[::3, K // 2] = float("inf")
    g[1::3, K - 1] = float("nan")
    dy, dw = w4.expert_combine_backward(g.to(gpu), y.to(gpu), w.to(gpu), rows)
    place, n = rows.place.cpu().numpy(), int(rows.offsets[E])
    assert (place < 0).any() and (dw.cpu().numpy()[place < 0] == 0).all()
    assert not np.isfinite(dw.cpu().numpy()[:2][place[:2] >= 0]).any()
    assert (dy[n:] == 0).all()
