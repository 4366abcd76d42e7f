"""Limits of window prefill: what pools hold where nobody looks."""
import numpy as np
import pytest
import torch

from oracle import bounded
from tests import bounded_util as B
from tests import gpu_util as U
from tests import spec_util as S
from tests import tree_limits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_180_gb300 as p
    return p


def _prefill(pkv, c, pool, window, sinks, bf16, scale):
    dev = pkv.KVPool(pool.shape[0], device=U.dev())
    dev.buffer.copy_(U.to_dev(pool).view(-1))
    out = torch.full((c.rows, 32, 64), float("nan"), device=U.dev(), dtype=torch.bfloat16 if bf16 else torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    bt = U.to_dev(c.hide(window, sinks))
    pkv.paged_window_prefill_attention(dev, out, U.to_dev(c.q), U.to_dev(c.starts), bt, bt.shape[1], U.to_dev(c.lens),
                                       c.max_query, c.max_context, scale, window, sinks, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out


def _unseen(c, window, sinks):
    """Slots of the pool [page, row] that no query of c sees: behind the contexts, in free pages, outside every window."""
    hidden = np.ones((c.pool.num_pages, 16), bool)
    for s, ctx in enumerate(c.lens):
        for p in range(int(ctx) - c.nodes[s], int(ctx)):
            t = bounded.seen_by(p, window, sinks)
            hidden[c.bt[s, t // 16], t % 16] = False
    return hidden


SHAPES = {"one tile": ([40, 100, 300], [40, 30, 7]),
          "two tiles": ([70, 33, 50, 64, 300, 1, 129], [70, 33, 50, 64, 90, 1, 100]),
          "two heads": ([40, 17, 100, 1, 64, 300] * 5, [32, 1, 20, 1, 30, 9] * 5)}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("bf16", [False, True])
def test_what_nobody_sees_reaches_nothing(pkv, shape, bf16):
    """Recycled pages hold any finite value: the same bits come out whatever it is."""
    c = B.Cache(*SHAPES[shape], seed=71)
    for window, sinks, scale in ((128, 4, 0.125), (20, 0, 0.125), (1000, 0, -0.125), (16, 1, 0.125), (5, 40, 0.125)):
        hidden = _unseen(c, window, sinks)
        want = None
        for k, v in ((0, 0), (0x447A, 0xC47A), (0xC47A, 0x447A), (0x7F7F, 0xFF7F), (0xFF7F, 0x7F7F)):
            pool = c.pool.data.copy()
            pool[:, 0].transpose(0, 2, 1, 3)[hidden] = k
            pool[:, 1].transpose(0, 2, 1, 3)[hidden] = v
            got = _prefill(pkv, c, pool, window, sinks, bf16, scale)
            want = got if want is None else want
            assert torch.equal(got, want), (window, sinks, hex(k), float((got - want).abs().max()))


@pytest.mark.parametrize("contexts,nodes", [([1024, 1025, 2048, 2049, 3000], [8, 9, 32, 33, 1]), ([2048, 1100], [2048, 70]),
                                            ([1024, 1040, 2050] * 8, [8, 5, 32] * 8)])
def test_runs_of_a_row_are_added_up_in_fp32(pkv, contexts, nodes):
    """Rows of one to three runs of 1024 keys, runs that end with the item, rows stored by boxes and by their threads."""
    c = B.Cache(contexts, nodes, seed=72)
    want, _, size, spread = c.prefill(1 << 30, 0)
    got = _prefill(pkv, c, c.pool.data, 1 << 30, 0, False, c.scale)
    S.assert_within(got.double().cpu().numpy(), want, S.bound(want, size, spread, c.scale, 3000, False), "window prefill")
    tree_limits.assert_precise(got.cpu().numpy(), want, c.starts, False)
    for _ in range(5):
        assert torch.equal(_prefill(pkv, c, c.pool.data, 1 << 30, 0, False, c.scale), got)
