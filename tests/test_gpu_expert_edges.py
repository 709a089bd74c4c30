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
