"""The limits of tree_limits reject what a kernel that loses keys or bits of the weights would give (mistakes are planted in
the oracle's inputs and results, on the CPU)."""
import numpy as np
import pytest

from tests import spec_util as S
from tests import tree_limits
from workloads import rng


def _rejected(got, ref, starts, bf16):
    try:
        tree_limits.assert_precise(got, ref, starts, bf16)
    except AssertionError:
        return True
    return False


def _attention(c, s, term):
    """Sequence s with weights of `term` bf16 terms (0: not rounded), in 64 bits otherwise."""
    def bf16(x):
        b = np.ascontiguousarray(x, np.float32).view(np.uint32)
        return ((b + 0x7FFF + (b >> 16 & 1)) & 0xFFFF0000).view(np.float32).astype(np.float64)
    ctx, n, a = int(c.lens[s]), c.nodes[s], c.starts[s]
    pages = c.bt[s, :-(-ctx // 16)]
    K, V = (rng.bf16_bits_to_f64(c.pool.data[pages, i].transpose(1, 0, 2, 3).reshape(8, -1, 64)[:, :ctx]) for i in (0, 1))
    q = rng.bf16_bits_to_f64(c.q[a:a + n]).reshape(n, 8, 4, 64)
    see = np.ones((n, ctx), bool)
    words = c.mask[a:a + n].view(np.uint32)
    for j in range(n):
        see[:, ctx - n + j] = words[:, j // 32] >> np.uint32(j % 32) & 1
    x = np.einsum("ngid,gtd->ngit", q, K) * c.wl.scale
    x = np.where(see[:, None, None], x, -np.inf)
    w = np.exp(x - x.max(-1, keepdims=True))
    used = w if term == 0 else bf16(w) if term == 1 else bf16(w) + bf16(w - bf16(w))
    return (np.einsum("ngit,gtd->ngid", used, V) / w.sum(-1)[..., None]).reshape(n, 32, 64)


@pytest.mark.parametrize("contexts,nodes,lost", [([9000], [3], 256), ([30000, 700], [4, 8], 1536)])
def test_keys_of_one_part_left_out(contexts, nodes, lost):
    c = S.TreeCase(contexts, nodes, seed=131)
    ref = c.reference()[0]
    bt = c.bt.copy()
    bt[0, 200:200 + lost // 16] = -1                       # pages that are not there are left out
    missing = c.reference(block_tables=bt)[0]
    for bf16 in (False, True):
        assert _rejected(missing, ref, c.starts, bf16)
    tree_limits.assert_precise(ref, ref, c.starts, False)
    one = np.flatnonzero(c.bt[0] >= 0)[-2]                 # a single page near the end: fp32 output shows that too
    bt = c.bt.copy()
    bt[0, one] = -1
    assert _rejected(c.reference(block_tables=bt)[0], ref, c.starts, False)


def test_a_weight_term_left_out():
    c = S.TreeCase([5000, 800], [3, 5], seed=132)
    ref = c.reference()[0]
    exact, one, two = (np.concatenate([_attention(c, s, t) for s in (0, 1)]) for t in (0, 1, 2))
    assert max(tree_limits.norm_errors(exact, ref, c.starts)) < 1e-12
    assert _rejected(one, ref, c.starts, False) and not _rejected(one, ref, c.starts, True)
    assert not _rejected(two, ref, c.starts, False)
    assert 1.5e-6 < max(tree_limits.norm_errors(two, ref, c.starts)) < 3e-6
