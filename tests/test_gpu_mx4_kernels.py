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
