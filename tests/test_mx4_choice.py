"""The sizes that the GPU tests multiply reach the kernels they are meant for (host only)."""

import pytest

from tests import mx4_choice


def test_the_source_is_what_the_choice_repeats():
    text = " ".join(mx4_choice.source().split())
    for line in mx4_choice.REPEATED:
        assert line in text, line
    kinds = [s[0] for s in mx4_choice.shapes()]
    assert len(kinds) == len(set(kinds)) == 9 and set(kinds) | {"Stream2x1Past"} == set(mx4_choice.DENSE)


@pytest.mark.parametrize("kind", sorted(mx4_choice.DENSE))
def test_sizes_reach_their_kernel(kind):
    _, BM, BN = next(s for s in mx4_choice.shapes() if s[0] == kind.replace("Past", ""))[:3]
    ends = [(M, N, K) for M, N, K in mx4_choice.DENSE[kind]]
    for M, N, K in ends:
        assert mx4_choice.kernel(M, N, K) == kind, (M, N, K, mx4_choice.kernel(M, N, K))
    assert any(M % BM and N % BN and K % 512 for M, N, K in ends)
    for sizes, N, K in mx4_choice.GROUPED[kind]:
        M = mx4_choice.NONE_BEFORE + sum(sizes) + mx4_choice.NONE_BEHIND
        assert mx4_choice.kernel(M, N, K, len(sizes)) == kind, (sizes, N, K, mx4_choice.kernel(M, N, K, len(sizes)))
        assert N % BN and K % 512 and 0 in sizes and any(s % BM for s in sizes)
    if kind == "Stream2x1Past":  # experts with one tile of rows, and with several, whose weights come through the caches
        assert all(any(0 < s <= 16 for s in sizes) and any(s > 16 for s in sizes) for sizes, _, _ in mx4_choice.GROUPED[kind])
        assert {M > 16 for M, _, _ in ends} == {True, False}


def test_the_kernels_of_some_sizes():
    """Sizes of tests that say otherwise beside them: few outputs and few steps are streamed."""
    assert mx4_choice.kernel(64, 5000, 1408) == mx4_choice.kernel(333, 3000, 384) == "Stream2x1"
    assert mx4_choice.kernel(512, 2560, 9216) == "Deep64x128"


def test_few_blocks_take_their_steps():
    """No kernel's estimate leaves out the steps of a launch of few blocks, and few outputs of many inputs are not given
    to the larger tiles (us as 64 x 128 and streamed by two and two: 37.8 and 18.8, 60.4 and 22.5, 35.0 and 18.3)."""
    for kind, _, _, _, slots, start, one, every, bare, step in mx4_choice.shapes():
        # (256 x 256: half a round of tiles is the least there is)
        assert not slots or max(one, step, 0.45 * every if kind == "Tile256" else 0) > 0, kind
    for M, N, K in ((512, 256, 28672), (64, 2048, 28672), (100, 1024, 28672)):
        assert mx4_choice.kernel(M, N, K) == "Stream2x2", (M, N, K)
