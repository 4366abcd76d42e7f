"""Answers of the allocator's calls on shared pages where the pool or the host's memory is full."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_180_gb300 import build
    build.build()
    import paged_kv_cache_180_gb300 as p
    return p


@pytest.mark.parametrize("layers", [1, 2])
@pytest.mark.parametrize("tokens", [40, 33, 32, 16, 1])
def test_a_fork_without_room_is_answered_as_an_admission(pkv, layers, tokens):
    # every page is assigned: whether or not a partly filled last page would have to be copied, the answer is the credits'
    a = pkv.Allocator(3 * layers, layers, 16, 256, 3)
    assert a.admit(0, 40, 8)[0] == a.OK                    # 47 tokens: three pages a layer, all of the pool
    for layer in range(layers):
        for block in range(3):
            a.page(0, layer, block)
    assert a.state() == (0, 3 * layers)
    before = a.block_tables()
    for new, want in ((1, a.NO_CREDIT), (8, a.NO_CREDIT), (100, a.EXCEEDS_POOL)):
        assert a.admit(1, tokens, new)[0] == want
        rc, src, dst = a.fork(0, 1, tokens, new)
        assert rc == want and len(src) == len(dst) == 0, (tokens, new)
    assert np.array_equal(a.block_tables(), before) and a.state() == (0, 3 * layers)
    a.free_seq(0)
    assert a.admit(1, tokens, 1)[0] == a.OK                # the refused forks hold nothing
