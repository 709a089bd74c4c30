"""Rows to the experts and back (oracle): plain loops and float64."""

import numpy as np


def expert_sort_ref(ids, E):
    """ids [T, top] -> (offsets [E + 1], place [T, top], order [T * top]), int32."""
    ids = np.asarray(ids)
    T, top = ids.shape
    flat = ids.reshape(-1).tolist()
    rows = [[] for _ in range(E)]
    for slot, e in enumerate(flat):
        if 0 <= e < E:
            rows[e].append(slot)
    offsets = np.zeros(E + 1, np.int32)
    place = np.full(T * top, -1, np.int32)
    order = np.full(T * top, -1, np.int32)
    r = 0
    for e in range(E):
        offsets[e] = r
        for slot in rows[e]:
            place[slot], order[r] = r, slot
            r += 1
    offsets[E] = r
    return offsets, place.reshape(T, top), order


def expert_take_ref(x, place):
    """xs [T * top, ...]: row place[t, j] is x[t], the others zeros."""
    T, top = place.shape
    xs = np.zeros((T * top,) + x.shape[1:], x.dtype)
    for t in range(T):
        for r in place[t]:
            if r >= 0:
                xs[r] = x[t]
    return xs


def expert_combine_ref(y, w, place):
    """(out, sum_j |w y|) in float64 (w None: ones)."""
    T, top = place.shape
    out, a = np.zeros((2, T, y.shape[1]))
    for t in range(T):
        for j, r in enumerate(place[t]):
            if r >= 0:
                v = (1.0 if w is None else float(w[t, j])) * y[r].astype(np.float64)
                out[t] += v
                a[t] += np.abs(v)
    return out, a


def expert_combine_backward_ref(dout, y, w, place):
    """(dy, dw, sum_k |dout y|) in float64 (w None: ones)."""
    T, top = place.shape
    dy = np.zeros(y.shape)
    dw, a = np.zeros((2, T, top))
    for t in range(T):
        g = dout[t].astype(np.float64)
        for j, r in enumerate(place[t]):
            if r >= 0:
                v = y[r].astype(np.float64)
                dy[r] = (1.0 if w is None else float(w[t, j])) * g
                dw[t, j], a[t, j] = (g * v).sum(), np.abs(g * v).sum()
    return dy, dw, a
