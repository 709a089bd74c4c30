"""Every kernel of the microscaled product on an MI355X, at sizes that end inside its tiles, against float64 (which
size reaches which kernel: test_mx4_choice.py).  The tolerance is that of test_gpu_mx4.py."""

import pytest
import torch

from tests import mx4_choice
from tests.test_gpu_mx4 import BF16, _check_on_gpu, _draw, _frame_kept, _framed, _say, _values

pytestmark = pytest.mark.gpu


def _cases(table):
    return [pytest.param(*case, id=f"{kind}-{i}") for kind in sorted(table) for i, case in enumerate(table[kind])]


@pytest.mark.parametrize("M,N,K", _cases(mx4_choice.DENSE))
def test_linear_mx4_at_ends_of_tiles(w4, gpu, M, N, K):
    _say(f"linear_mx4 {M} rows of {N}x{K}, {mx4_choice.kernel(M, N, K)}")
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
    # a row of NaN scales (and of the weights, one) is NaN, and what lies beside it is what it was
    xs2, ws2 = xs.clone(), ws.clone()
    xs2[1::2] = 255
    ws2[N - 1, 0] = 255
    got = w4.linear_mx4(xq, xs2, *w4.pack_mx4(wq, ws2), N, out_dtype=torch.float32)
    assert torch.equal(got[0::2, :-1], y32[0::2, :-1]) and bool(got[1::2].isnan().all()) and bool(got[:, -1].isnan().all())


@pytest.mark.parametrize("sizes,N,K", _cases(mx4_choice.GROUPED))
def test_grouped_linear_mx4_at_ends_of_tiles(w4, gpu, sizes, N, K):
    E, first, after = len(sizes), mx4_choice.NONE_BEFORE, mx4_choice.NONE_BEHIND
    M = first + sum(sizes) + after
    _say(f"grouped_linear_mx4 {sizes} {N}x{K}, {mx4_choice.kernel(M, N, K, E)}")
    ends = [first + sum(sizes[:e + 1]) for e in range(E)]
    offsets = torch.tensor([first] + ends, dtype=torch.int32, device=gpu)
    made = [_draw(gpu, 10 + e, N, K) for e in range(E)]
    packed = [w4.pack_mx4(*m) for m in made]
    q, s = torch.stack([p[0] for p in packed]), torch.stack([p[1] for p in packed])
    xq, xs = _draw(gpu, 9, M, K)
    xs[:first], xs[M - after:] = 255, 255  # rows of no expert are not read
    buf = torch.full((M + 2, N), 77.0, device=gpu)
    y32 = w4.grouped_linear_mx4(xq, xs, offsets, q, s, N, out=buf[1:1 + M])
    assert _frame_kept(buf) and bool((y32[:first] == 77).all()) and bool((y32[M - after:] == 77).all())
    for e in range(E):
        a, b = ends[e] - sizes[e], ends[e]
        if a < b:
            _check_on_gpu(y32[a:b], _values(xq[a:b], xs[a:b]), _values(*made[e]), K, f"expert {e}")
    buf16, y16 = _framed(gpu, M, N, BF16)
    w4.grouped_linear_mx4(xq, xs, offsets, q, s, N, out=y16)
    assert _frame_kept(buf16) and torch.equal(y16[first:M - after], y32[first:M - after].to(BF16))
    # the rows of one expert, NaN, do not reach the next one's
    e = max(range(E), key=lambda i: sizes[i])
    xs[ends[e] - sizes[e]:ends[e]] = 255
    got = w4.grouped_linear_mx4(xq, xs, offsets, q, s, N, out_dtype=torch.float32)
    assert bool(got[ends[e] - sizes[e]:ends[e]].isnan().all())
    assert torch.equal(got[first:ends[e] - sizes[e]], y32[first:ends[e] - sizes[e]])
    assert torch.equal(got[ends[e]:M - after], y32[ends[e]:M - after])


@pytest.mark.parametrize("M,N,K,kind", [(700, 2100, 640, "Deep64"), (330, 1130, 5248, "Deep32x64"), (900, 1746, 6784, "Deep128"),
                                        (1600, 1281, 896, "Tile256")])
def test_odd_offsets_at_tiles(w4, gpu, M, N, K, kind):
    """Offsets that decrease, overlap or leave [0, M] in the kernels of tiles: rows outside are never touched, rows of
    one range alone are right, and rows of none are left."""
    assert mx4_choice.kernel(M, N, K, 4) == kind
    made = [_draw(gpu, 20 + e, N, K) for e in range(4)]
    packed = [w4.pack_mx4(*m) for m in made]
    q, s = torch.stack([p[0] for p in packed]), torch.stack([p[1] for p in packed])
    xq, xs = _draw(gpu, 9, M, K)
    a, b = M // 3 + 1, M // 2 + 3
    for offsets in ([0, M + 9, 20, b, M], [-5, a, a, 2 * M, 20], [M] * 5, [7, 3, 2, 1, 0], [2 ** 31 - 1, -2 ** 31, 5, M, M + 1],
                    [0, M, 0, M, M]):
        _say(f"grouped_linear_mx4 {offsets} of {M} rows {N}x{K}, {kind}")
        buf, y = _framed(gpu, M, N, torch.float32)
        w4.grouped_linear_mx4(xq, xs, torch.tensor(offsets, dtype=torch.int32, device=gpu), q, s, N, out=y)
        torch.cuda.synchronize()
        assert _frame_kept(buf), offsets
        at = [min(max(o, 0), M) for o in offsets]
        owners = [[e for e in range(4) if at[e] <= m < at[e + 1]] for m in range(M)]
        none = [m for m in range(M) if not owners[m]]
        assert bool((y[none] == 77).all()), offsets
        if all(len(o) <= 1 for o in owners):
            for e in range(4):
                rows = [m for m in range(M) if owners[m] == [e]]
                if rows:
                    _check_on_gpu(y[rows], _values(xq[rows], xs[rows]), _values(*made[e]), K, f"{offsets}, expert {e}")


@pytest.mark.parametrize("N,K,rows", [((1 << 24) - 19, 256, (3, 40)), (32750, 130944, (3, 70, 300))])
def test_largest_matrices(w4, gpu, N, K, rows):
    """Codes of nearly 2 GiB, the most that a product takes, many outputs and many inputs: outputs at both ends and
    where offsets pass 30 bits."""
    g = torch.Generator(device=gpu)
    g.manual_seed(4)
    nb, ns = w4.packed_bytes_mx4(N, K), w4.scale_bytes_mx4(N, K)
    assert 0 < (1 << 31) - nb <= 16 * 512 * 128  # (a row block of the longest rows)
    q = torch.empty(nb, dtype=torch.uint8, device=gpu)
    for at in range(0, nb, 1 << 28):
        q[at:at + (1 << 28)].random_(0, 256, generator=g)
    s = torch.empty(ns, dtype=torch.uint8, device=gpu).random_(121, 134, generator=g)
    wq, ws = w4.unpack_mx4(q, s, N, K)
    for M in rows:
        _say(f"linear_mx4 {M} rows of {N}x{K}, {mx4_choice.kernel(M, N, K)}")
        xq, xs = _draw(gpu, M, M, K)
        y = w4.linear_mx4(xq, xs, q, s, N, out_dtype=torch.float32)
        for n in (0, N // 2 - 40, N - 80):
            _check_on_gpu(y[:, n:n + 80], _values(xq, xs), _values(wq[n:n + 80], ws[n:n + 80]), K, f"from output {n}")
        assert torch.equal(w4.linear_mx4(xq, xs, q, s, N), y.to(BF16))
