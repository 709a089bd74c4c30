"""Rows to the experts and back on an MI355X: what lies at the edges of their use."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(f"\n[case] {msg}", flush=True)


@pytest.mark.parametrize("T,top,E", [(2049, 1, 2), (5000, 3, 3), (20001, 6, 5), (65535, 4, 63)])
def test_sort_of_runs(w4, gpu, T, top, E):
    """Slots of one expert keep their order where lanes of one wavefront, and wavefronts of one block, share a key:
    runs of one expert that end inside and at the ends of wavefronts, two experts in turn, all the same."""
    slots = T * top
    i = np.arange(slots)
    for kind, ids in (("runs of 64", i // 64 % E), ("runs of 63", i // 63 % E), ("runs of 257", i // 257 % E),
                      ("in turn", i % E), ("in turn with dropped ones", i % (E + 1) - 1), ("one", i * 0)):
        _say(f"sort of {slots} slots of {E} experts, {kind}")
        ids = ids.reshape(T, top).astype(np.int64)
        want = oracle.expert_sort_ref(ids, E)
        for _ in range(2):
            got = w4.expert_sort(torch.from_numpy(ids).to(gpu), E)
            for a, b, what in zip(got, want, got._fields):
                assert np.array_equal(a.cpu().numpy(), b), what


def _layer(gpu, T=20, top=2, E=5, K=64, dtype=BF16):
    """x, ids, y and weights of a small layer, 1/6 of the slots dropped."""
    rng = np.random.default_rng(31)
    ids = torch.from_numpy(rng.integers(-1, E, (T, top))).to(gpu)
    make = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(gpu)  # noqa: E731
    return make(T, K).to(dtype), ids, make(T * top, K).to(dtype), make(T, top)


def _index_writes(rows):
    """The tensors of an ExpertRows by name, and what is written into them: other rows, inside their ranges."""
    return {"place": lambda: rows.place.copy_(rows.place.flip(0)), "offsets": lambda: rows.offsets.fill_(0),
            "order": lambda: rows.order.fill_(-1)}


@pytest.mark.parametrize("call,read", [("dispatch", ["place"]), ("take", ["place"]), ("combine y", ["place", "offsets"]),
                                       ("combine weights", ["place"]), ("combine sum", ["place", "offsets"])])
def test_indices_written_before_backward(w4, gpu, call, read):
    """A gradient whose places or offsets were written since the forward pass is refused; one that does not read
    what was written is what it was."""
    x, ids, y, w = _layer(gpu)
    for name in ("place", "offsets", "order"):
        _say(f"{call}, {name} written before backward")
        grads = []
        for write in (False, True):
            leaf = {"dispatch": x, "take": x, "combine y": y, "combine weights": w, "combine sum": y}[call]
            leaf = leaf.clone().requires_grad_()
            rows = w4.expert_sort(ids, 5)
            if call == "dispatch":
                out, rows = w4.expert_dispatch(leaf, ids, 5)
            elif call == "take":
                out = w4.expert_take(leaf, rows)
            elif call == "combine y":
                out = w4.expert_combine(leaf, w, rows)
            elif call == "combine weights":
                out = w4.expert_combine(y, leaf, rows)
            else:
                out = w4.expert_combine(leaf, None, rows)
            if write:
                _index_writes(rows)[name]()
            if write and name in read:
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    out.sum().backward()
            else:
                out.sum().backward()
                grads.append(leaf.grad)
        assert len(grads) == 1 or torch.equal(*grads)


def test_forward_mode_is_refused(w4, gpu):
    """There is no forward-mode derivative of these calls: a dual tensor is refused, and its tangent never dropped;
    within a dual level plain tensors are taken as ever."""
    _say("forward mode")
    x, ids, y, w = _layer(gpu, dtype=F32)
    rows = w4.expert_sort(ids, 5)
    plain = [w4.expert_dispatch(x, ids, 5)[0], w4.expert_take(x, rows), w4.expert_take(x[:, 0].contiguous(), rows),
             w4.expert_combine(y, w, rows), w4.expert_combine(y, None, rows)]
    with torch.autograd.forward_ad.dual_level():
        dual = lambda t: torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: w4.expert_dispatch(dual(x), ids, 5), lambda: w4.expert_take(dual(x), rows),
                     lambda: w4.expert_combine(dual(y), w, rows), lambda: w4.expert_combine(y, dual(w), rows),
                     lambda: w4.expert_combine(dual(y), None, rows),
                     lambda: w4.expert_combine(dual(y.clone().requires_grad_()), w, rows)):
            for grad in (True, False):
                with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError, match="jvp|forward"):
                    call()
        again = [w4.expert_dispatch(x, ids, 5)[0], w4.expert_take(x, rows), w4.expert_take(x[:, 0].contiguous(), rows),
                 w4.expert_combine(y, w, rows), w4.expert_combine(y, None, rows)]
    for a, b in zip(plain, again):
        assert torch.equal(a, b) and not b.requires_grad


def test_combine_keeps_what_its_gradients_read(w4, gpu):
    """y is kept for the gradient of the weights only, and the weights for that of y: the other may be freed or
    written before the backward pass."""
    x, ids, y, w = _layer(gpu)
    rows = w4.expert_sort(ids, 5)
    g = torch.ones_like(x)
    for weights in (w, None):
        _say(f"gradient of y alone, weights {weights is not None}")
        leaf = y.clone().requires_grad_()
        held = leaf * 2.0
        out = w4.expert_combine(held, weights, rows)
        want = w4.expert_combine_backward(g, held.detach(), weights, rows, need_weights=False)[0]
        with torch.no_grad():
            held.fill_(float("nan"))
        out.backward(g)
        assert torch.equal(leaf.grad, want * 2.0)
    _say("gradient of the weights alone")
    leaf = w.clone().requires_grad_()
    held = leaf * 2.0
    out = w4.expert_combine(y, held, rows)
    want = w4.expert_combine_backward(g, y, held.detach(), rows, need_y=False)[1]
    with torch.no_grad():
        held.fill_(float("nan"))
    out.backward(g)
    assert torch.equal(leaf.grad, want * 2.0)
    _say("what is read may not be written")
    for which in ("y", "w"):
        a, b = y.clone().requires_grad_(), w.clone().requires_grad_()
        ya, wb = a * 1.0, b * 1.0
        out = w4.expert_combine(ya, wb, rows)
        with torch.no_grad():
            (ya if which == "y" else wb).fill_(1.0)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.backward(g)
    _say("memory held between the passes")
    T, top, K = 512, 4, 4096
    big = w4.expert_sort(torch.zeros((T, top), dtype=torch.int64, device=gpu), 1)
    weights = torch.ones((T, top), device=gpu)
    leaf = torch.ones((1, K), dtype=BF16, device=gpu).requires_grad_()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated(gpu)
    out = w4.expert_combine(leaf * torch.ones((T * top, 1), dtype=BF16, device=gpu), weights, big)
    # (the factor, 2 bytes a row, and out, 2 bytes a value, stay; y, another T * top * K * 2 bytes, does not)
    assert torch.cuda.memory_allocated(gpu) - before < T * top * K
    _say("saved tensors that hooks carry away and bring back")
    x, ids, y, w = _layer(gpu)
    rows = w4.expert_sort(ids, 5)
    grads = []
    for away in (False, True):
        leaves = [v.clone().requires_grad_() for v in (x, y, w)]
        with torch.autograd.graph.save_on_cpu() if away else torch.enable_grad():
            out = (w4.expert_take(leaves[0], rows) + w4.expert_dispatch(leaves[0], ids, 5)[0]).sum() + w4.expert_combine(
                leaves[1], leaves[2], rows).sum()
        grads.append(torch.autograd.grad(out, leaves))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    with torch.autograd.graph.saved_tensors_hooks(lambda v: v.cpu(), lambda v: v):
        out = w4.expert_combine(y.clone().requires_grad_(), w, rows).sum()
        taken = w4.expert_take(x.clone().requires_grad_(), rows).sum()
    for loss in (out, taken):
        with pytest.raises(ValueError, match="several devices"):
            loss.backward()
