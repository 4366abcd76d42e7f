"""Limits of window prefill: what pools hold where nobody looks, and sums over long windows."""
import numpy as np
import pytest
import torch

from oracle import bounded
from tests import bounded_util as B
from tests import gpu_util as U
from tests import spec_util as S
from tests import tree_limits
from workloads import rng

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


def repeated_pages(pkv, pages, bf16, seed, positive=False, order=(0,), keys=None, seconds=None):
    """(output, expected output, weighted sum of |V|) of one query over a context of `pages` pages: those of `order`, then
    page 1, whose keys are equal, again and again.  keys(K): sets the K of the pages [page][head][row][dim] as bits.
    `seconds`: a list that receives the time the call took."""
    ctx, ids = 16 * pages, max(2, max(order) + 1)
    draw = lambda tag, n: rng.normal_bf16(rng.stream_key(seed, tag), 0, n)  # noqa: E731
    kv = draw("kv", ids * 2 * 8 * 16 * 64).reshape(ids, 2, 8, 16, 64)
    kv[1, 0] = kv[1, 0, :, :1]                                  # one K row, sixteen times
    if keys is None:
        kv[0, 0, :, 0, 7] = 0x4180                              # token 0: K_7 = 16
    else:
        keys(kv[:, 0])
    if positive:
        kv[:, 1] = kv[:, 1] & 0x7FFF                            # V > 0
    q = draw("q", 32 * 64).reshape(1, 32, 64)
    q[..., 7] = (q[..., 7] & 0x7F) | 0x3F80                     # q_7 in [1, 2)
    pool = pkv.KVPool(ids, device=U.dev())
    pool.buffer.copy_(U.to_dev(kv).view(-1))
    bt = torch.ones(1, pages, dtype=torch.int32, device=U.dev())
    bt[:, :len(order)] = torch.tensor(order, dtype=torch.int32, device=U.dev())
    out = torch.full((1, 32, 64), float("nan"), device=U.dev(), dtype=torch.bfloat16 if bf16 else torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    args = (pool, out, U.to_dev(q), torch.tensor([0, 1], dtype=torch.int32, device=U.dev()), bt, pages,
            torch.tensor([ctx], dtype=torch.int32, device=U.dev()), 1, ctx, 0.125, ctx, 0, status)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ends[0].record()
    pkv.paged_window_prefill_attention(*args)
    ends[1].record()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    if seconds is not None:
        seconds.append(ends[0].elapsed_time(ends[1]) * 1e-3)
    K, V = (rng.bf16_bits_to_f64(kv[:, i]).transpose(1, 0, 2, 3).reshape(8, ids * 16, 64) for i in (0, 1))
    times = np.array([order.count(i) for i in range(ids)], float)
    times[1] += pages - len(order)
    times = np.repeat(times, 16)
    x = np.einsum("sghd,gtd->sght", rng.bf16_bits_to_f64(q).reshape(1, 8, 4, 64), K) * 0.125
    w = np.exp(x - x[..., times > 0].max(-1, keepdims=True)) * times
    w /= w.sum(-1, keepdims=True)
    ref, size = (np.einsum("sght,gtd->sghd", w, v).reshape(1, 32, 64) for v in (V, np.abs(V)))
    return out.double().cpu().numpy(), ref, size


def _within(got, ref, size, lim):
    worst = float((np.abs(got - ref) / size).max())
    assert (np.abs(got - ref) <= size * lim).all(), (worst, lim)


def test_fp32_output_of_28000_equal_weights(pkv):
    got, ref, size = repeated_pages(pkv, 1750, False, 121)
    # relative to the weighted |V|: the one weight's split into two bf16 terms 2^-18; 8 blocks of 16 truncating MMAs a run,
    # 64 * 2^-24 of it in the mean of the growing sum; score and exponential 2^-19 + 2^-22; the row sum 8 + 16 + 14 half steps of
    # 2^-24 (32 keys, run, 28 runs), the same 14 for O
    lim = 2.0 ** -18 + 64 * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -22 + (38 + 14) * 2.0 ** -24
    _within(got, ref, size, lim)


def test_bf16_output_of_a_window_of_millions_of_equal_weights(pkv):
    got, ref, size = repeated_pages(pkv, 1 << 20, True, 122, positive=True)
    # the one weight as a single bf16 term 2^-8 and the output 2^-8; 128 blocks of 8 truncating MMAs a run (1024 2^-24), 1024
    # runs of O and 16384 of the row sum added up (512 and 8192 times 2^-24), a run's row sum (8 + 16) 2^-24, score, exponential
    lim = 2 * 2.0 ** -8 + (1024 + 512 + 8192 + 24) * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -22
    _within(got, ref, size, lim)


@pytest.mark.parametrize("contexts,nodes", [([16384, 16385, 16500], [3, 40, 1]), ([33000], [70])])
def test_bf16_output_of_windows_of_several_runs(pkv, contexts, nodes):
    c = B.Cache(contexts, nodes, seed=73)
    want, _, size, spread = c.prefill(1 << 30, 0)
    got = _prefill(pkv, c, c.pool.data, 1 << 30, 0, True, c.scale).double().cpu().numpy()
    S.assert_within(got, want, S.bound(want, size, spread, c.scale, max(contexts), True), "window prefill")
    tree_limits.assert_precise(got, want, c.starts, True)


def _grown(K):
    # the first 64 keys score about 0, a later one about 200 and the repeated ones a little less: out of the fast path's range
    K[1, :, :, 7] = 0x447A                                      # 1000
    K[2, :, 5, 7] = 0x447C                                      # 1008


@pytest.mark.parametrize("bf16", [False, True])
def test_sums_of_rows_that_are_computed_again(pkv, bf16):
    got, ref, size = repeated_pages(pkv, 1750, bf16, 123, order=(0, 0, 0, 0, 2), keys=_grown)
    # 110 stretches of 256 equal weights: (256 + 110) / 2 * 2^-24 in O and in the row sum; the exponential and the division 2^-22;
    # the scores (exponents of up to 2^9.5: 6 roundings of 2^-24) move weight between the one key, 0.2 % at the most, and the others
    lim = (256 + 110) * 2.0 ** -24 + 2.0 ** -22 + 0.002 * 6 * 2.0 ** (9.5 - 24) + (2.0 ** -8 if bf16 else 0)
    _within(got, ref, size, lim)


@pytest.fixture(scope="module")
def slow(pkv):
    """A call that takes longer than a wait inside a kernel may (2 s): one query over keys that make its rows be computed
    again, every key some 0.5 us at the least.  Gives a function that launches it and one that says how long it took."""
    kv = rng.normal_bf16(rng.stream_key(124, "kv"), 0, 3 * 2 * 8 * 16 * 64).reshape(3, 2, 8, 16, 64)
    kv[1, 0] = kv[1, 0, :, :1]
    _grown(kv[:, 0])
    q = rng.normal_bf16(rng.stream_key(124, "q"), 0, 32 * 64).reshape(1, 32, 64)
    q[..., 7] = (q[..., 7] & 0x7F) | 0x3F80
    pool, q = pkv.KVPool(3, device=U.dev()), U.to_dev(q)
    pool.buffer.copy_(U.to_dev(kv).view(-1))
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    status, out = torch.zeros(1, dtype=torch.int32, device=U.dev()), torch.empty(1, 32, 64, device=U.dev())
    starts = torch.tensor([0, 1], dtype=torch.int32, device=U.dev())

    def prepare(pages):
        bt = torch.ones(1, pages, dtype=torch.int32, device=U.dev())
        bt[0, :5] = torch.tensor([0, 0, 0, 0, 2])
        lens = torch.tensor([16 * pages], dtype=torch.int32, device=U.dev())

        def launch():
            ends[0].record()
            pkv.paged_window_prefill_attention(pool, out, q, starts, bt, pages, lens, 1, 16 * pages, 0.125, 16 * pages, 0, status)
        return launch

    def took():
        ends[1].record()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return ends[0].elapsed_time(ends[1]) * 1e-3

    for _ in range(2):
        prepare(4000)()
        seconds = took()
    pages = int(4000 * 2.8 / seconds)
    assert pages < 400_000, seconds
    return prepare(pages), took


def _follower(pkv, name):
    """(call(overlap), its output)"""
    c = B.Cache([300, 130, 77], [100, 130, 5] if "prefill" in name else None, seed=74)
    pool = pkv.KVPool(c.pool.num_pages, device=U.dev())
    pool.buffer.copy_(U.to_dev(c.pool.data).view(-1))
    q, bt, lens, starts = U.to_dev(c.q), U.to_dev(c.bt), U.to_dev(c.lens), U.to_dev(c.starts)
    out = torch.full((c.rows, 32, 64), float("nan"), device=U.dev())
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    sums = torch.zeros(3, 8, c.max_context, device=U.dev())

    def call(overlap):
        if name == "window prefill":
            pkv.paged_window_prefill_attention(pool, out, q, starts, bt, bt.shape[1], lens, c.max_query, c.max_context, c.scale, 90,
                                               4, status, overlap_previous=overlap)
        elif name == "prefill":
            pkv.paged_prefill_attention(pool, out, q, starts, bt, bt.shape[1], lens, c.max_query, c.max_context, c.scale, status,
                                        overlap_previous=overlap)
        elif name == "window decode":
            pkv.paged_window_decode_attention(pool, out, q, bt, bt.shape[1], lens, c.max_context, c.scale, 90, 4, status,
                                              overlap_previous=overlap)
        else:
            pkv.paged_decode_attention_weights(pool, out, q, bt, bt.shape[1], lens, c.max_context, c.scale, sums, 0.0, None,
                                               status, overlap_previous=overlap)
    return call, out, status


@pytest.mark.parametrize("name", ["window prefill", "window decode", "weights", "prefill"])
def test_waits_do_not_run_out_on_the_kernel_before(pkv, slow, name):
    """A call launched before a kernel of more than 2 s has ended."""
    launch, took = slow
    call, out, status = _follower(pkv, name)
    call(False)
    torch.cuda.synchronize()
    want = out.clone()
    out.fill_(float("nan"))
    torch.cuda.synchronize()
    launch()
    call(True)
    assert took() > 2.4
    assert int(status.item()) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("seqs", [1, 30])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("first,behind,zeros", [(0, (1 << 31) - 1, (0, 40)), (7, (1 << 31) - 1, (7, 40)),
                                                (-(1 << 31) + 9, 5, (0, 5)), (-20, 3, (0, 3)), (40, (1 << 31) - 1, (40, 40))])
def test_query_starts_far_outside_the_rows(pkv, seqs, bf16, first, behind, zeros):
    """A sequence of two thousand million query tokens gets zero rows where there are rows, and takes no longer than that."""
    pool = pkv.KVPool(4, device=U.dev())
    pool.buffer.zero_()
    starts = np.full(seqs + 1, behind, np.int32)
    starts[0] = first
    out = torch.ones(40, 32, 64, device=U.dev(), dtype=torch.bfloat16 if bf16 else torch.float32)
    q = torch.zeros(40, 32, 64, dtype=torch.bfloat16, device=U.dev())
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    bt, lens = torch.zeros(seqs, 4, dtype=torch.int32, device=U.dev()), torch.full((seqs,), 64, dtype=torch.int32, device=U.dev())
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in ends:
        pkv.paged_window_prefill_attention(pool, out, q, U.to_dev(starts), bt, 4, lens, 20, 64, 0.125, 8, 0, status)
        e.record()
    torch.cuda.synchronize()
    want = torch.ones(40, dtype=torch.bool, device=U.dev())
    want[zeros[0]:zeros[1]] = False
    assert int(status.item()) == 2 and torch.equal((out == 1).all(-1).all(-1), want) and (out[~want] == 0).all()
    assert ends[0].elapsed_time(ends[1]) < 50


def test_the_longest_context(pkv):
    """2^31 - 64 tokens of which the window and the sinks are there: the same bits as from a short context that ends alike."""
    ctx, n, window, sinks = (1 << 31) - 64, 70, 300, 4
    c = B.Cache([640], [n], seed=75)
    pool = pkv.KVPool(c.pool.num_pages, device=U.dev())
    pool.buffer.copy_(U.to_dev(c.pool.data).view(-1))
    short = U.to_dev(c.hide(window, sinks))
    blocks = ctx // 16
    far = torch.full((1, blocks), -1, dtype=torch.int32, device=U.dev())
    far[0, 0], far[0, blocks - 30:] = short[0, 0], short[0, 10:40]
    q, starts = U.to_dev(c.q), U.to_dev(c.starts)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    for dtype in (torch.float32, torch.bfloat16):
        got = []
        for bt, length in ((short, 640), (far, ctx)):
            lens = torch.tensor([length], dtype=torch.int32, device=U.dev())
            prefill, decode = (torch.full((k, 32, 64), float("nan"), dtype=dtype, device=U.dev()) for k in (n, 1))
            pkv.paged_window_prefill_attention(pool, prefill, q, starts, bt, bt.shape[1], lens, n, length, c.scale, window, sinks,
                                               status)
            pkv.paged_window_decode_attention(pool, decode, q[n - 1:], bt, bt.shape[1], lens, length, c.scale, window, sinks, status)
            got += [prefill, decode]
        assert torch.isfinite(got[0]).all() and torch.equal(got[0], got[2]) and torch.isfinite(got[1]).all()
        assert torch.allclose(got[1], got[3], rtol=2.0 ** -7 if dtype == torch.bfloat16 else 1e-5, atol=1e-6)
    assert int(status.item()) == 0


@pytest.mark.parametrize("window,sinks", [((1 << 31) - 1, 0), ((1 << 31) - 1, (1 << 31) - 1), (1, (1 << 31) - 1), ((1 << 31) - 2, 3)])
@pytest.mark.parametrize("bf16", [False, True])
def test_the_largest_windows_and_sinks(pkv, window, sinks, bf16):
    c = B.Cache([0, 1, 2, 15, 16, 17, 33, 64, 65, 100, 600, 1500], seed=76)
    want, _, size, spread, weights = c.decode(window, sinks)
    out = torch.full((12, 32, 64), float("nan"), device=U.dev(), dtype=torch.bfloat16 if bf16 else torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    pool = pkv.KVPool(c.pool.num_pages, device=U.dev())
    pool.buffer.copy_(U.to_dev(c.pool.data).view(-1))
    pkv.paged_window_decode_attention(pool, out, U.to_dev(c.q), U.to_dev(c.bt), c.bt.shape[1], U.to_dev(c.lens), c.max_context,
                                      c.scale, window, sinks, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    lim = B.decode_bound(want, size, spread, c.scale, max(t.size for t, _ in weights.values()), bf16)
    S.assert_within(out.double().cpu().numpy(), want, lim, "window decode")
    for shape in SHAPES.values():
        c = B.Cache(*shape, seed=77)
        want, _, size, spread = c.prefill(window, sinks)
        got = _prefill(pkv, c, c.pool.data, window, sinks, bf16, c.scale).double().cpu().numpy()
        S.assert_within(got, want, S.bound(want, size, spread, c.scale, 300, bf16), "window prefill")


@pytest.mark.parametrize("contexts,nodes,window,sinks", [([1100, 3000], [64, 40], 1000, 4), ([3000], [33], 2900, 0),
                                                         ([600, 200, 333], [200, 200, 1], 256, 4), ([9000], [2], 8000, 1),
                                                         ([2500, 1300, 40] * 8, [9, 32, 3] * 8, 1200, 4)])
def test_fp32_output_has_the_precision_of_fp32_arithmetic(pkv, contexts, nodes, window, sinks):
    """Norm of the error over the output's, by sequence.  Three bf16 terms of a weight: 2^-25.  48 MMAs to a run of 256 keys,
    each of which truncates O by half a unit in the mean, 2^-24 of a number of its size, 0.72 of that over a binade: with V of
    both signs O grows as the root of their number, 48 * 2 / 3 * 0.72 * 2^-24 = 1.4e-6 at the most (where all go the same way);
    score and exponential 2^-19 / sqrt(3) = 1.1e-6 at exponents of up to 2^4.  The root of the squares' sum: 1.8e-6."""
    c = B.Cache(contexts, nodes, seed=78)
    want = c.prefill(window, sinks)[0]
    got = _prefill(pkv, c, c.pool.data, window, sinks, False, c.scale).double().cpu().numpy()
    errors = tree_limits.norm_errors(got, want, c.starts)
    assert max(errors) < 1.8e-6, errors
