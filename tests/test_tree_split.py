"""The model of tree attention's split over the CTAs, and the layouts that the GPU tests rely on."""
import pytest

from tests import tree_split

# 320 units of 24 blocks, cut into 304 shares: every share ends the unit before and begins the next one
RUN_SUMS = ([1536] * 40, [8] * 40)


def has_run_sums_beside_a_one_block_segment(shares):
    """CTAs with a unit of several runs of 16 blocks (from its first block to its last), followed by exactly one block of
    the next unit: both segments keep what they sum up in the same part of the workspace."""
    return [i for i, segments in enumerate(shares)
            if any(x[3] == 0 and x[4] == x[5] > 16 and y[3:5] == (0, 1) and y[5] > 1
                   for x, y in zip(segments, segments[1:]))]


@pytest.mark.parametrize("contexts,nodes", [RUN_SUMS, ([9000], [3]), ([30000, 700], [40, 64]), ([20000, 64], [8, 64]),
                                            ([300, 0, 77, 64], [33, 0, 5, 64])])
def test_shares_hold_every_block_once(contexts, nodes):
    whole, shares = tree_split.split(contexts, nodes)
    if whole:
        return
    seen = {}
    for segments in shares:
        for s, g, t, j0, j1, nb in segments:
            assert 0 <= j0 < j1 <= nb
            seen.setdefault((s, g, t), []).extend(range(j0, j1))
    want = {(s, g, t): list(range(-(-c // 64))) for s, (c, n) in enumerate(zip(contexts, nodes)) if n
            for g in range(8) for t in range(-(-n // 32))}
    assert {u: sorted(b) for u, b in seen.items()} == want


def test_the_layout_of_run_sums_is_hit():
    whole, shares = tree_split.split(*RUN_SUMS)
    assert not whole and len(has_run_sums_beside_a_one_block_segment(shares)) == 16
