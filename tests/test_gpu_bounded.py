"""GPU parity of window attention, weight sums and eviction (through the C ABI) against the FP64 oracle.

Attention is held to bounds derived from its arithmetic; what eviction moves is bit-exact over the whole pool.  Untouched
pool slots hold NaN patterns, and table entries of pages that no query sees are -1, throughout.
"""
import numpy as np
import pytest
import torch

import oracle
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


def _pool(pkv, host):
    pool = pkv.KVPool(host.num_pages, device=U.dev())
    pool.buffer.copy_(U.to_dev(host.data).view(-1))
    return pool


def _out(rows, bf16, guard=3):
    return torch.full((rows + guard, 32, 64), float("nan"), device=U.dev(), dtype=torch.bfloat16 if bf16 else torch.float32)


def _guarded(out, rows):
    torch.cuda.synchronize()
    assert torch.isnan(out[rows:]).all(), "rows behind the last one were written"
    return out[:rows].double().cpu().numpy()


def _status():
    return torch.zeros(1, dtype=torch.int32, device=U.dev())


# ---- window decode -----------------------------------------------------------------------------
def _window_decode(pkv, c, window, sinks, bf16=False, scale=None, bt=None, max_context=None, **kw):
    out, status = _out(len(c.lens), bf16), _status()
    bt = U.to_dev(c.hide(window, sinks) if bt is None else bt)
    pkv.paged_window_decode_attention(_pool(pkv, c.pool), out, U.to_dev(c.q), bt, bt.shape[1], U.to_dev(c.lens),
                                      c.max_context if max_context is None else max_context,
                                      c.scale if scale is None else scale, window, sinks, status, **kw)
    return _guarded(out, len(c.lens)), int(status.item())


def _check_decode(pkv, c, window, sinks, bf16=False, scale=None, bt=None, max_context=None):
    got, status = _window_decode(pkv, c, window, sinks, bf16, scale, bt, max_context)
    ref, err, size, spread, weights = c.decode(window, sinks, scale, bt, max_context)
    assert status == err
    keys = max([t.size for t, _ in weights.values()], default=1)
    S.assert_within(got, ref, B.decode_bound(ref, size, spread, c.scale if scale is None else scale, keys, bf16),
                    "window decode")
    return got


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 16), (15, 17), (16, 0), (17, 4), (64, 33), (1000, 5),
                                          (1 << 31 - 1, 0), (3, (1 << 31) - 1)])
@pytest.mark.parametrize("bf16", [False, True])
def test_window_decode_lengths(pkv, window, sinks, bf16):
    window = min(window, 2 ** 31 - 1)
    _check_decode(pkv, B.Cache([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 600, 1500], seed=11), window, sinks, bf16)


@pytest.mark.parametrize("contexts", [[2048], [5000], [700, 3000], [300] * 5, [129] * 20, [20] * 60])
@pytest.mark.parametrize("window,sinks", [(512, 4), (2000, 20), (100000, 0)])
def test_window_decode_shares_of_a_unit(pkv, contexts, window, sinks):
    # one to eight CTAs to a unit, shares of no page among them
    _check_decode(pkv, B.Cache(contexts, seed=12), window, sinks)


@pytest.mark.parametrize("scale", [1.0, -0.125, 0.0, 1e-30, -2.0])
def test_window_decode_scales(pkv, scale):
    _check_decode(pkv, B.Cache([700, 40, 90], seed=13), 300, 4, scale=scale)


def test_window_decode_does_not_lose_precision(pkv):
    # fp32 output: weights of 24 bits, and sums that do not drift with the number of pages
    c = B.Cache([9000, 4000, 2500], seed=14)
    got, _ = _window_decode(pkv, c, 1 << 30, 0)
    ref = c.decode(1 << 30, 0)[0]
    for s in range(3):
        assert np.linalg.norm(got[s] - ref[s]) < 2e-6 * np.linalg.norm(ref[s])


def test_window_decode_what_is_outside_reaches_nothing(pkv):
    c = B.Cache([600, 50], seed=15)
    want = _check_decode(pkv, c, 100, 5)
    for kind in (0x7f80, 0xff80, 0x7fc0, 0xffff):
        for s, ctx in ((0, 600),):
            for t in list(range(5, 40)) + list(range(ctx - 130, ctx - 100)):
                c.token(s, t, 0)[:] = kind
                c.token(s, t, 1)[:] = kind
        assert np.array_equal(_window_decode(pkv, c, 100, 5)[0], want)


def test_window_decode_bad_lengths_and_pages(pkv):
    c = B.Cache([100, 200, 64, 33], seed=16)
    c.lens = np.array([-1, 200, 65, 33], np.int32)
    bt = c.bt.copy()
    bt[1, 3], bt[1, 12], bt[3, 0] = -7, c.pool.num_pages, c.pool.num_pages + 5
    got = _check_decode(pkv, c, 1000, 0, bt=bt, max_context=200)
    assert (got[0] == 0).all()
    _check_decode(pkv, c, 16, 4, bt=bt, max_context=200)
    _check_decode(pkv, c, 17, 0, bt=bt, max_context=64)      # sequences 1 and 2 are longer than the bound
    bt[:] = -1
    got, status = _window_decode(pkv, c, 17, 0, bt=bt, max_context=200)
    assert (got == 0).all() and status == 2 | 4


def test_window_decode_scores_without_a_weight(pkv):
    # K of -infinity: no weight; a row of nothing else gets zeros; +infinity and NaN leave NaN in that row's heads alone
    c = B.Cache([300, 40], seed=17)
    c.q[:] = np.where(c.q & 0x8000, c.q & 0x7fff, c.q)                     # positive queries
    want = _window_decode(pkv, c, 64, 0)[0]
    for t in range(236, 300):
        if t % 3:
            c.token(0, t, 0)[2] = 0xff80
    ref = c.pool.data.copy()
    got, _ = _window_decode(pkv, c, 64, 0)
    left = [t for t in range(236, 300) if t % 3 == 0]
    K, V = (np.stack([rng.bf16_bits_to_f64(c.token(0, t, i)[2]) for t in left]) for i in (0, 1))
    x = rng.bf16_bits_to_f64(c.q[0, 8:12]) @ K.T * c.scale
    w = np.exp(x - x.max(1, keepdims=True))
    assert np.abs(got[0, 8:12] - (w / w.sum(1, keepdims=True)) @ V).max() < 1e-5
    assert np.array_equal(np.delete(got[0], range(8, 12), 0), np.delete(want[0], range(8, 12), 0))
    for t in left:
        c.token(0, t, 0)[2] = 0xff80
    assert (_window_decode(pkv, c, 64, 0)[0][0, 8:12] == 0).all()
    c.pool.data[:] = ref
    for bits in (0x7f80, 0x7fc0):
        c.token(0, 299, 0)[2] = bits
        got = _window_decode(pkv, c, 64, 0)[0]
        assert np.isnan(got[0, 8:12]).all() and np.isfinite(np.delete(got[0], range(8, 12), 0)).all()
        assert np.isfinite(got[1]).all()


def test_window_decode_streams_graphs_and_overlap(pkv):
    c = B.Cache([900, 130, 77], seed=18)
    want, _ = _window_decode(pkv, c, 200, 4)
    pool, status = _pool(pkv, c.pool), _status()
    q, bt, lens = U.to_dev(c.q), U.to_dev(c.bt), U.to_dev(c.lens)
    outs = [_out(3, False) for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda o, **kw: pkv.paged_window_decode_attention(pool, o, q, bt, bt.shape[1], lens, c.max_context, c.scale,  # noqa: E731
                                                             200, 4, status, **kw)
    call(outs[0])
    call(outs[1], stream=side)                        # no workspace: calls may overlap
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[2])
    for _ in range(3):
        outs[2].fill_(float("nan"))
        graph.replay()
        for o in outs:
            assert np.array_equal(_guarded(o, 3), want)
    # behind the append of the last tokens, launched before that has ended
    empty = _pool(pkv, oracle.Pool(c.wl.num_pages))
    parts = [c.wl.kv_tokens(s, 0) for s in range(3)]
    k, v = (U.to_dev(np.concatenate([p[i] for p in parts])) for i in (0, 1))
    slots = U.to_dev(np.concatenate([c.wl.slot_mapping(s, 0, 0, int(c.lens[s])) for s in range(3)]))
    out = _out(3, False)
    pkv.kv_append(empty, k, v, slots, status)
    pkv.paged_window_decode_attention(empty, out, q, bt, bt.shape[1], lens, c.max_context, c.scale, 200, 4, status,
                                      overlap_previous=True)
    assert np.array_equal(_guarded(out, 3), want) and int(status.item()) == 0


def test_window_decode_split_pool_and_strided_tables(pkv):
    c = B.Cache([500, 90], seed=19)
    want, _ = _window_decode(pkv, c, 100, 4)
    half = 8 * 16 * 64
    k, v = (torch.full((c.pool.num_pages, half + 64), float("nan"), dtype=torch.bfloat16, device=U.dev()) for _ in range(2))
    k[:, :half], v[:, :half] = (U.to_dev(np.ascontiguousarray(c.pool.data[:, i])).view(-1, half) for i in (0, 1))
    pool = pkv.kv_pool_create(k, v, (half + 64) * 2, c.pool.num_pages)
    tables = torch.full((2, 3, c.bt.shape[1]), -9, dtype=torch.int32, device=U.dev())
    tables[:, 1] = U.to_dev(c.hide(100, 4))
    out, status = _out(2, False), _status()
    pkv.paged_window_decode_attention(pool, out, U.to_dev(c.q), tables[:, 1], tables.stride(0), U.to_dev(c.lens),
                                      c.max_context, c.scale, 100, 4, status)
    assert np.array_equal(_guarded(out, 2), want) and int(status.item()) == 0


# ---- window prefill ----------------------------------------------------------------------------
def _window_prefill(pkv, c, window, sinks, bf16=False, scale=None, bt=None, max_query=None, starts=None, lens=None,
                    rows=None, guarded=True, **kw):
    rows = c.rows if rows is None else rows
    out, status = _out(rows, bf16), _status()
    bt = U.to_dev(c.hide(window, sinks) if bt is None else bt)
    q = torch.cat([U.to_dev(c.q)[:rows], torch.full((3, 32, 64), float("nan"), dtype=torch.bfloat16, device=U.dev())])
    pkv.paged_window_prefill_attention(_pool(pkv, c.pool), out, q, U.to_dev(c.starts if starts is None else starts), bt,
                                       bt.shape[1], U.to_dev(c.lens if lens is None else lens),
                                       c.max_query if max_query is None else max_query, c.max_context,
                                       c.scale if scale is None else scale, window, sinks, status, **kw)
    return _guarded(out, rows) if guarded else out.double().cpu().numpy(), int(status.item())


def _check_prefill(pkv, c, window, sinks, bf16=False, scale=None, bt=None):
    got, status = _window_prefill(pkv, c, window, sinks, bf16, scale, bt)
    ref, err, size, spread = c.prefill(window, sinks, scale, bt)
    assert status == err
    keys = min(int(c.lens.max()), window + sinks)
    S.assert_within(got, ref, S.bound(ref, size, spread, c.scale if scale is None else scale, keys, bf16), "window prefill")
    return got, ref


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (5, 16), (16, 1), (33, 17), (128, 4), (1000, 0), (2, 300)])
@pytest.mark.parametrize("bf16", [False, True])
def test_window_prefill_lengths(pkv, window, sinks, bf16):
    contexts = [0, 1, 16, 17, 40, 64, 65, 100, 130, 257, 300]
    nodes = [0, 1, 16, 1, 33, 64, 20, 32, 97, 65, 3]
    _check_prefill(pkv, B.Cache(contexts, nodes, seed=21), window, sinks, bf16)


@pytest.mark.parametrize("contexts,nodes,window,sinks", [
    ([600], [200], 256, 4), ([2100], [40], 1500, 16), ([3000, 2500], [33, 64], 2900, 0), ([400] * 6, [400] * 6, 128, 1),
    ([2300], [2], 2200, 70)])
@pytest.mark.parametrize("bf16", [False, True])
def test_window_prefill_longer(pkv, contexts, nodes, window, sinks, bf16):
    c = B.Cache(contexts, nodes, seed=22)
    got, ref = _check_prefill(pkv, c, window, sinks, bf16)
    tree_limits.assert_precise(got, ref, c.starts, bf16)


# more than 19 sequences of at most 32 queries: two K/V heads to an item
def _many_spans(seed, n=26, top=700):
    r = np.random.RandomState(seed)
    ctx = r.randint(0, top, n)
    ctx[:4] = (top, 33, 16, 1)
    nodes = np.minimum(ctx, r.randint(0, 33, n))
    nodes[:3] = (32, 32, 8)
    return B.Cache(ctx.tolist(), nodes.tolist(), seed=seed)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 1), (33, 17), (128, 4), (1000, 0), (2, 300), (200, 40)])
@pytest.mark.parametrize("bf16", [False, True])
def test_window_prefill_short_spans(pkv, window, sinks, bf16):
    _check_prefill(pkv, _many_spans(57), window, sinks, bf16)


def test_window_prefill_short_spans_of_long_contexts(pkv):
    ctx, nodes = [2500, 40, 1700] + [600] * 20, [5, 32, 17] + [1, 2, 7, 31] * 5
    c = B.Cache(ctx, nodes, seed=58)
    for window, sinks, bf16 in ((2100, 20, False), (100000, 0, False), (1300, 4, True)):   # sums taken out after 1024 keys
        _check_prefill(pkv, c, window, sinks, bf16)


def test_window_prefill_short_spans_bad_lengths_pages_and_values(pkv):
    c = _many_spans(59)
    big = [s for s in range(26) if c.lens[s] > 250 and c.nodes[s] > 3]
    bt = c.bt.copy()
    bt[big[0], 3], bt[big[1], int(c.lens[big[1]]) // 16 - 1] = -7, c.pool.num_pages + 5
    _check_prefill(pkv, c, 1000, 2, bt=bt)
    lens = c.lens.copy()
    lens[big[0]], lens[big[1]], lens[big[2]] = 3, -5, c.max_context + 1            # fewer tokens than queries, bad lengths
    got, status = _window_prefill(pkv, c, 64, 2, lens=lens, bt=c.bt)
    ref, err, _, _ = c.prefill(64, 2, lens=lens)
    assert status == err == 2 and np.abs(got - ref).max() < 1e-4
    for s in big[:3]:
        assert (got[c.starts[s]:c.starts[s + 1]] == 0).all()
    # NaN in V of one head's token: rows that see it are NaN, all others as if it were not there
    s, head, window = big[3], 5, 40
    t = int(c.lens[s]) - int(c.nodes[s]) - 20
    want = c.prefill(window, 0)[0]
    c.token(s, t, 1)[head] = 0x7fc0
    got, status = _window_prefill(pkv, c, window, 0)
    hit = np.zeros((c.rows, 32), bool)
    for j in range(c.nodes[s]):
        if t in bounded.seen_by(int(c.lens[s]) - c.nodes[s] + j, window, 0):
            hit[c.starts[s] + j, 4 * head:4 * head + 4] = True
    assert status == 0 and hit.any() and not np.isfinite(got[hit]).any()
    assert np.abs(got[~hit] - want[~hit]).max() < 2e-5


def test_window_prefill_short_spans_in_graphs(pkv):
    c = _many_spans(60, 40, 300)
    want, _ = _window_prefill(pkv, c, 100, 4)
    pool, status, out = _pool(pkv, c.pool), _status(), _out(c.rows, False)
    q, bt, lens, starts = U.to_dev(c.q), U.to_dev(c.bt), U.to_dev(c.lens), U.to_dev(c.starts)
    args = (bt, bt.shape[1], lens, c.max_query, c.max_context, c.scale, 100, 4, status)
    pkv.paged_window_prefill_attention(pool, out, q, starts, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for overlap in (False, True):
            pkv.paged_window_prefill_attention(pool, out, q, starts, *args, overlap_previous=overlap)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        assert np.array_equal(_guarded(out, c.rows), want) and int(status.item()) == 0


def test_window_prefill_more_items_than_the_tables_of_all_sms_hold(pkv):
    r = np.random.RandomState(53)
    ctx = r.randint(0, 40, 1400)
    _check_prefill(pkv, B.Cache(ctx.tolist(), np.minimum(ctx, r.randint(0, 4, 1400)).tolist(), seed=54), 9, 2)


@pytest.mark.parametrize("scale", [1.0, -0.125, 0.0, 1e-30, -1.0])
def test_window_prefill_scales(pkv, scale):
    _check_prefill(pkv, B.Cache([300, 70], [60, 33], seed=23), 90, 4, scale=scale)


def test_window_prefill_is_window_decode_row_by_row(pkv):
    c = B.Cache([450], [70], seed=24)
    got, _ = _window_prefill(pkv, c, 100, 3)
    one = B.Cache([450], seed=24)
    for j in (0, 1, 31, 32, 69):
        one.lens = np.array([450 - 70 + j + 1], np.int32)
        one.q[:1] = c.q[j:j + 1]
        row, _ = _window_decode(pkv, one, 100, 3, bt=one.bt)
        assert np.linalg.norm(row[0] - got[j]) < 1e-5 * np.linalg.norm(row[0])


@pytest.mark.parametrize("bf16", [False, True])
def test_window_prefill_values_that_some_rows_do_not_see(pkv, bf16):
    # NaN and infinities in V (and K) of single tokens: rows that see them are NaN or infinite as the oracle says, all
    # others as if they were not there
    c = B.Cache([200, 60], [150, 40], seed=25)
    window, sinks = 40, 3
    want, _ = _window_prefill(pkv, c, window, sinks, bf16)
    for bits, kv, t in ((0x7fc0, 1, 90), (0x7f80, 1, 120), (0xff80, 1, 130), (0x7fc0, 0, 150), (0x7f80, 1, 199)):
        keep = c.token(0, t, kv).copy()
        c.token(0, t, kv)[3] = bits
        got, status = _window_prefill(pkv, c, window, sinks, bf16)
        assert status == 0
        hit = np.zeros((c.rows, 32), bool)
        for j in range(150):
            if t in bounded.seen_by(50 + j, window, sinks):
                hit[j, 12:16] = True
        assert hit.any() and not np.isfinite(got[hit]).any()
        if kv == 1 and bits != 0x7fc0:
            assert (got[hit] == (np.inf if bits == 0x7f80 else -np.inf)).all()
        assert np.isfinite(got[~hit]).all()
        ref = c.prefill(window, sinks)[0]
        assert np.abs(got[~hit] - ref[~hit]).max() < (2e-2 if bf16 else 2e-5)
        assert np.array_equal(got[150:], want[150:])
        c.token(0, t, kv)[:] = keep


def test_window_prefill_scores_that_grow(pkv):
    for gain, where in ((64, slice(100, 280)), (256, slice(133, 134)), (1 / 64, slice(70, 300))):
        c = B.Cache([300, 70], [200, 30], seed=26)
        for s in range(2):
            for t in range(*where.indices(int(c.lens[s]))):
                k = c.token(s, t, 0)
                k[:] = ((rng.bf16_bits_to_f64(k) * gain).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        _check_prefill(pkv, c, 110, 4)


def test_window_prefill_bad_lengths_and_pages(pkv):
    c = B.Cache([100, 200, 64, 33, 50], [40, 70, 20, 33, 10], seed=27)
    bt = c.bt.copy()
    bt[1, 9], bt[1, 12], bt[3, 0] = -7, c.pool.num_pages, c.pool.num_pages + 5
    _check_prefill(pkv, c, 64, 2, bt=bt)
    lens = np.array([30, 200, 64, -5, c.max_context + 1], np.int32)    # fewer tokens than queries, and two bad lengths
    got, status = _window_prefill(pkv, c, 64, 2, lens=lens, bt=c.bt)
    ref, err, _, _ = c.prefill(64, 2, lens=lens)
    assert status == err == 2 and np.abs(got - ref).max() < 1e-4 and (got[:40] == 0).all()
    got, status = _window_prefill(pkv, c, 64, 2, max_query=40, bt=c.bt)
    ref, err, _, _ = c.prefill(64, 2, max_query=40)
    assert status == err == 2 and (got[40:110] == 0).all() and np.abs(got - ref).max() < 1e-4
    starts = np.array([0, 40, 30, 60, 80, 90], np.int32)               # the second sequence has -10 queries
    got, status = _window_prefill(pkv, c, 64, 2, starts=starts, bt=c.bt, rows=85, guarded=False)
    assert status == 2 and got.shape[0] == 88 and np.isfinite(got[:40]).all() and (got[80:] == 0).all()  # 88 rows are there


def test_window_prefill_streams_graphs_and_overlap(pkv):
    c = B.Cache([300, 130, 77], [100, 130, 5], seed=28)
    want, _ = _window_prefill(pkv, c, 90, 4)
    pool, status = _pool(pkv, c.pool), _status()
    q, bt, lens, starts = U.to_dev(c.q), U.to_dev(c.bt), U.to_dev(c.lens), U.to_dev(c.starts)
    outs = [_out(c.rows, False) for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda p, o, **kw: pkv.paged_window_prefill_attention(p, o, q, starts, bt, bt.shape[1], lens, c.max_query,  # noqa: E731
                                                                 c.max_context, c.scale, 90, 4, status, **kw)
    call(pool, outs[0])
    call(pool, outs[1], stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(pool, outs[2])
    for _ in range(3):
        outs[2].fill_(float("nan"))
        graph.replay()
        for o in outs:
            assert np.array_equal(_guarded(o, c.rows), want)
    empty = _pool(pkv, oracle.Pool(c.wl.num_pages))
    parts = [c.wl.kv_tokens(s, 0) for s in range(3)]
    k, v = (U.to_dev(np.concatenate([p[i] for p in parts])) for i in (0, 1))
    slots = U.to_dev(np.concatenate([c.wl.slot_mapping(s, 0, 0, int(c.lens[s])) for s in range(3)]))
    out = _out(c.rows, False)
    pkv.kv_append(empty, k, v, slots, status)
    call(empty, out, overlap_previous=True)
    assert np.array_equal(_guarded(out, c.rows), want) and int(status.item()) == 0


# ---- decode with weight sums ---------------------------------------------------------------------
def _sums(c, seed, layers=None, extra=5):
    r = np.random.RandomState(seed)
    shape = (len(c.lens), 8, c.max_context + extra) if layers is None else (len(c.lens), layers, 8, c.max_context + extra)
    return (r.standard_exponential(shape) ** 3 * 0.02).astype(np.float32)


def _weights(pkv, c, sums, decay, bf16=False, scale=None, bt=None, max_context=None, workspace=None, **kw):
    out, status = _out(len(c.lens), bf16), _status()
    bt = U.to_dev(c.bt if bt is None else bt)
    mc = c.max_context if max_context is None else max_context
    ws = pkv.weights_workspace(len(c.lens), mc) if workspace is None else workspace
    pkv.paged_decode_attention_weights(_pool(pkv, c.pool), out, U.to_dev(c.q), bt, bt.shape[1], U.to_dev(c.lens), mc,
                                       c.scale if scale is None else scale, sums, decay, ws, status, **kw)
    return _guarded(out, len(c.lens)), int(status.item())


def _check_weights(pkv, c, decay, bf16=False, scale=None, bt=None, max_context=None):
    host = _sums(c, 31)
    old = host.copy()
    if decay == 0:
        old[:, :, ::3] = np.nan                    # not read
    dev = U.to_dev(old)
    got, status = _weights(pkv, c, dev, decay, bf16, scale, bt, max_context)
    ref, err, size, spread, weights = c.decode(1 << 31, 0, scale, bt, max_context)
    assert status == err
    keys = max([t.size for t, _ in weights.values()], default=1)
    scale = c.scale if scale is None else scale
    S.assert_within(got, ref, B.decode_bound(ref, size, spread, scale, keys, bf16), "decode with weights")
    after = dev.double().cpu().numpy()
    want, lim = old.astype(np.float64), np.zeros(old.shape)
    _, rows = bounded.decode_queries(c.lens, c.max_context if max_context is None else max_context)
    for s in rows:
        ctx = int(c.lens[s])
        want[s, :, :ctx] = old[s, :, :ctx] * np.float64(np.float32(decay)) if decay else 0
    for (i, _, g), (t, w) in weights.items():
        want[i, g, t] += w.sum(0)
        # four weights of that error, three additions of them, one rounding of the sum
        lim[i, g, t] = w.sum(0) * (B.weight_error(spread, scale, keys) + 4 * 2.0 ** -23)
    lim += np.abs(np.where(np.isnan(want), 0, want)) * 2.0 ** -23
    assert np.array_equal(np.isnan(want), np.isnan(after))
    S.assert_within(np.nan_to_num(after), np.nan_to_num(want), lim, "weight sums")
    return after


@pytest.mark.parametrize("decay", [1.0, 0.9, 0.0])
@pytest.mark.parametrize("bf16", [False, True])
def test_weights_lengths(pkv, decay, bf16):
    _check_weights(pkv, B.Cache([0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 600, 1500], seed=32), decay, bf16)


@pytest.mark.parametrize("contexts", [[2048], [6000], [700, 3000], [300] * 5, [129] * 20, [20] * 60])
def test_weights_shares_of_a_unit(pkv, contexts):
    _check_weights(pkv, B.Cache(contexts, seed=33), 1.0)


@pytest.mark.parametrize("contexts,blocks", [([300] * 9 + [700], 512), ([40] * 30 + [900], 2300), ([2000, 1], 2300),
                                             ([20] * 60, 512), ([6000], 2500), ([130, 0, 5000], 4200)])
def test_bounds_far_above_the_lengths(pkv, contexts, blocks):
    """Shares of a unit go by the bound on the lengths: short ones leave most of a cluster without pages."""
    c = B.Cache(contexts, seed=39, max_blocks=blocks)
    _check_weights(pkv, c, 0.9)
    _check_decode(pkv, c, 1 << 30, 0, bf16=True)
    _check_decode(pkv, c, 256, 3)


@pytest.mark.parametrize("scale", [1.0, -0.125, 0.0])
def test_weights_scales(pkv, scale):
    _check_weights(pkv, B.Cache([700, 40, 90], seed=34), 0.5, scale=scale)


def test_weights_add_up_to_the_heads(pkv):
    c = B.Cache([5000, 77], seed=35)
    after = _check_weights(pkv, c, 0.0)
    for s in range(2):
        assert np.abs(after[s, :, :c.lens[s]].sum(1) - 4).max() < 1e-4


def test_weights_bad_lengths_and_pages(pkv):
    c = B.Cache([100, 200, 64, 33], seed=36)
    c.lens = np.array([-1, 200, 65, 33], np.int32)
    bt = c.bt.copy()
    bt[1, 3], bt[1, 12], bt[3, 0] = -7, c.pool.num_pages, c.pool.num_pages + 5
    _check_weights(pkv, c, 0.9, bt=bt, max_context=200)
    _check_weights(pkv, c, 0.9, bt=bt, max_context=64)
    bt[:] = -1
    _check_weights(pkv, c, 0.9, bt=bt, max_context=200)


def test_weights_scores_in_the_workspace(pkv):
    # contexts whose scores do not fit on chip: the same sequences by a bound above 57344 tokens as by a small one
    c = B.Cache([3000, 100], seed=37, max_blocks=3700)
    host = _sums(c, 38)
    a, b = U.to_dev(host), U.to_dev(host)
    small, _ = _weights(pkv, c, a, 1.0, max_context=3008)
    large, status = _weights(pkv, c, b, 1.0, max_context=59200,
                             workspace=torch.full((pkv.weights_workspace_bytes(2, 59200),), 255, dtype=torch.uint8, device=U.dev()))
    assert status == 0 and np.abs(small - large).max() < 1e-5
    assert (a - b).abs().max().item() < 1e-5
    with pytest.raises(pkv.PkvError) as e:
        _weights(pkv, c, b, 1.0, max_context=59200, workspace=torch.empty(1024, dtype=torch.uint8, device=U.dev()))
    assert e.value.code == -6


def test_weights_of_a_long_context(pkv):
    # scores in the workspace over its whole length, against sums of the same formula in torch
    ctx = 60011
    pages = (ctx + 15) // 16
    g = torch.Generator(device=U.dev()).manual_seed(7)
    pool = pkv.KVPool(pages, device=U.dev())
    pool.buffer.copy_(torch.randn(pool.buffer.shape, device=U.dev(), generator=g))
    q = torch.randn(1, 32, 64, device=U.dev(), generator=g).bfloat16()
    bt = torch.randperm(pages, device=U.dev(), generator=g).int()[None]
    lens, status = torch.tensor([ctx], dtype=torch.int32, device=U.dev()), _status()
    kv = pool.view()[bt[0].long()].permute(1, 2, 0, 3, 4).reshape(2, 8, -1, 64)[:, :, :ctx].double()
    w = torch.softmax(q[0].double().view(8, 4, 64) @ kv[0].transpose(1, 2) * 0.125, -1)
    for bf16 in (False, True):
        sums, out = torch.zeros(1, 8, pages * 16, device=U.dev()), _out(1, bf16)
        pkv.paged_decode_attention_weights(pool, out, q, bt, pages, lens, pages * 16, 0.125, sums, 1.0,
                                           pkv.weights_workspace(1, pages * 16), status)
        ref = (w @ kv[1]).view(32, 64).cpu().numpy()
        assert np.linalg.norm(_guarded(out, 1)[0] - ref) < (5e-3 if bf16 else 2e-6) * np.linalg.norm(ref)
        assert int(status.item()) == 0
        want = w.sum(1)
        assert ((sums[0, :, :ctx].double() - want).norm() < 2e-6 * want.norm()).item() and (sums[0, :, ctx:] == 0).all()


def test_weights_behind_the_append_that_it_overlaps(pkv):
    c = B.Cache([900, 130, 77], seed=42)
    host = _sums(c, 43)
    want_sums = U.to_dev(host)
    want, _ = _weights(pkv, c, want_sums, 0.9)
    empty, status = _pool(pkv, oracle.Pool(c.wl.num_pages)), _status()
    parts = [c.wl.kv_tokens(s, 0) for s in range(3)]
    k, v = (U.to_dev(np.concatenate([p[i] for p in parts])) for i in (0, 1))
    slots = U.to_dev(np.concatenate([c.wl.slot_mapping(s, 0, 0, int(c.lens[s])) for s in range(3)]))
    q, bt, lens, out, sums = U.to_dev(c.q), U.to_dev(c.bt), U.to_dev(c.lens), _out(3, False), U.to_dev(host)
    pkv.kv_append(empty, k, v, slots, status)
    pkv.paged_decode_attention_weights(empty, out, q, bt, bt.shape[1], lens, c.max_context, c.scale, sums, 0.9, None, status,
                                       overlap_previous=True)
    assert np.array_equal(_guarded(out, 3), want) and torch.equal(sums, want_sums) and int(status.item()) == 0


@pytest.mark.parametrize("contexts", [[5000], [2500, 1], [300] * 40])  # clusters of 16 and 8, single CTAs
def test_shares_of_any_kind_behind_the_append_and_side_by_side(pkv, contexts):
    n = len(contexts)
    c = B.Cache(contexts, seed=55)
    host = _sums(c, 56)
    want_sums = U.to_dev(host)
    want, _ = _weights(pkv, c, want_sums, 1.0)
    want_window, _ = _window_decode(pkv, c, 1 << 30, 0)
    empty, status = _pool(pkv, oracle.Pool(c.wl.num_pages)), _status()
    parts = [c.wl.kv_tokens(s, 0) for s in range(n)]
    k, v = (U.to_dev(np.concatenate([p[i] for p in parts])) for i in (0, 1))
    slots = U.to_dev(np.concatenate([c.wl.slot_mapping(s, 0, 0, int(c.lens[s])) for s in range(n)]))
    q, bt, lens, sums = U.to_dev(c.q), U.to_dev(c.bt), U.to_dev(c.lens), U.to_dev(host)
    outs = [_out(n, False) for _ in range(4)]
    args = (bt, bt.shape[1], lens, c.max_context, c.scale)
    pkv.kv_append(empty, k, v, slots, status)
    pkv.paged_decode_attention_weights(empty, outs[0], q, *args, sums, 1.0, None, status, overlap_previous=True)
    pkv.paged_window_decode_attention(empty, outs[1], q, *args, 1 << 30, 0, status, overlap_previous=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for o, stream in zip(outs[2:], streams):
            pkv.paged_window_decode_attention(empty, o, q, *args, 1 << 30, 0, status, stream=stream)
    assert np.array_equal(_guarded(outs[0], n), want) and torch.equal(sums, want_sums) and int(status.item()) == 0
    for o in outs[1:]:
        assert np.array_equal(_guarded(o, n), want_window)


def test_weights_longest_first(pkv):
    # more units than are resident at once: sequences are taken by length, ties and empty ones among them
    r = np.random.RandomState(9)
    contexts = r.randint(0, 200, 60).tolist() + [0, 0, 150, 150, 150, 1]
    _check_weights(pkv, B.Cache(contexts, seed=44), 0.9)
    c = B.Cache(contexts, seed=45)
    c.lens[3], c.lens[10] = -4, c.max_context + 1
    c.bt[3] = c.bt[10] = -1
    _check_weights(pkv, c, 1.0)


def test_weights_strides_streams_and_graphs(pkv):
    c = B.Cache([300, 130, 77], seed=39)
    host = _sums(c, 40)
    one = U.to_dev(host)
    want, _ = _weights(pkv, c, one, 0.9)
    layered = torch.full((3, 4, 8, host.shape[2]), float("nan"), device=U.dev())
    layered[:, 2] = U.to_dev(host)
    got, _ = _weights(pkv, c, layered[:, 2], 0.9)
    assert np.array_equal(got, want) and torch.equal(layered[:, 2], one) and torch.isnan(layered[:, 3]).all()
    heads_first = U.to_dev(np.ascontiguousarray(host.transpose(1, 0, 2))).transpose(0, 1)
    assert np.array_equal(_weights(pkv, c, heads_first, 0.9)[0], want) and torch.equal(heads_first, one)
    # steps by a graph replay are steps by calls
    pool, status = _pool(pkv, c.pool), _status()
    q, bt, lens = U.to_dev(c.q), U.to_dev(c.bt), U.to_dev(c.lens)
    called, replayed, out = U.to_dev(host), U.to_dev(host), _out(3, False)
    step = lambda sums: pkv.paged_decode_attention_weights(pool, out, q, bt, bt.shape[1], lens, c.max_context, c.scale,  # noqa: E731
                                                           sums, 0.9, None, status)
    for _ in range(3):
        step(called)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(replayed)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(called, replayed)
    for bad in (host.shape[2] - 6, ):
        with pytest.raises(ValueError):
            _weights(pkv, c, U.to_dev(np.ascontiguousarray(host[:, :, :bad])), 0.9)


# ---- eviction --------------------------------------------------------------------------------------
class Evict:
    def __init__(self, contexts, layers=1, seed=1, ties=0, max_blocks=None, extra=0):
        blocks = max(2, max((c + 15) // 16 for c in contexts)) if max_blocks is None else max_blocks
        r = np.random.RandomState(seed)
        self.lens = np.array(contexts, np.int32)
        self.max_context = blocks * 16
        need = [max(0, min(c, self.max_context) + 15) // 16 for c in contexts]
        pages = sum(need) * layers + 3
        ids = r.permutation(pages)
        self.bt = np.full((len(contexts), layers, blocks), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            for layer in range(layers):
                self.bt[s, layer, :n] = ids[at:at + n]
                at += n
        self.pool = oracle.Pool(pages)
        self.pool.data[:] = r.randint(0, 65536, self.pool.data.shape).astype(np.uint16)
        sums = r.standard_exponential((len(contexts), layers, 8, self.max_context + extra)).astype(np.float32) ** 3
        if ties:
            sums = np.floor(sums * ties).astype(np.float32)
        self.sums = sums


def _run_evict(pkv, e, budgets, sinks, recent, in_place=False, width=None, bt=None, stream=None, pool=None):
    budgets = np.array(budgets, np.int32)
    width = max(1, int(budgets.max())) if width is None else width
    pool = _pool(pkv, e.pool) if pool is None else pool
    sums = U.to_dev(e.sums)
    new = sums if in_place else torch.full_like(sums, -7.0)
    kept = torch.full((len(e.lens), e.bt.shape[1], 8, width), -1, dtype=torch.int32, device=U.dev())
    lens, status = torch.full((len(e.lens) + 1,), -3, dtype=torch.int32, device=U.dev()), _status()
    bt = U.to_dev(e.bt if bt is None else bt)
    pkv.kv_evict(pool, bt, bt.stride(0), bt.stride(1), U.to_dev(e.lens), U.to_dev(budgets), sums, new, sinks, recent,
                 e.max_context, kept, lens, status, stream=stream)
    torch.cuda.synchronize()
    assert int(lens[-1]) == -3
    return pool, sums, new, kept.cpu().numpy(), lens[:-1].cpu().numpy(), int(status.item())


def _check_evict(pkv, e, budgets, sinks, recent, in_place=False, width=None, bt=None):
    pool, sums, new, kept, lens, status = _run_evict(pkv, e, budgets, sinks, recent, in_place, width, bt)
    want_pool = oracle.Pool(e.pool.num_pages)
    want_pool.data[:] = e.pool.data
    w = max(1, max(budgets)) if width is None else width
    want_new, want_kept, want_lens, err = bounded.evict(want_pool, e.bt if bt is None else bt, e.lens, budgets, e.sums,
                                                        sinks, recent, e.max_context, w)
    assert status == err
    assert lens.tolist() == want_lens.tolist()
    assert np.array_equal(kept, want_kept)
    got = new.cpu().numpy()
    for s in range(len(e.lens)):
        ctx = int(e.lens[s])
        valid = 0 <= ctx <= e.max_context and budgets[s] >= 0 and min(budgets[s], ctx) <= w
        n = ctx if valid else 0
        assert np.array_equal(got[s, :, :, :n], want_new[s, :, :, :n], equal_nan=True)
        rest = e.sums[s, :, :, n:] if in_place else np.full_like(got[s, :, :, n:], -7)
        assert np.array_equal(got[s, :, :, n:], rest, equal_nan=True)
    assert in_place or np.array_equal(sums.cpu().numpy(), e.sums, equal_nan=True)
    assert np.array_equal(U.bits(pool.view()), want_pool.data)


@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 0), (0, 7), (3, 20), (40, 40), (0, 1 << 30), ((1 << 31) - 1, 5)])
@pytest.mark.parametrize("ties", [0, 3])
def test_evict_lengths(pkv, sinks, recent, ties):
    contexts = [0, 1, 2, 15, 16, 17, 33, 64, 100, 130, 257, 300]
    budgets = [5, 1, 1, 15, 3, 16, 20, 0, 99, 70, 128, 301]
    _check_evict(pkv, Evict(contexts, seed=41, ties=ties), budgets, sinks, recent)


@pytest.mark.parametrize("contexts,layers", [([2000], 1), ([5000], 1), ([900, 1300], 3), ([300] * 20, 2), ([130] * 40, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_shares_of_a_unit(pkv, contexts, layers, in_place):
    # one to eight CTAs to a unit, several rounds of the move
    for keep, ties in ((0.5, 0), (0.9, 2), (0.07, 1)):
        e = Evict(contexts, layers, seed=42, ties=ties, extra=9)
        _check_evict(pkv, e, [max(1, int(c * keep)) for c in contexts], 4, 30, in_place)


@pytest.mark.parametrize("contexts,blocks", [([5000], 4200), ([300] * 9 + [700], 4200), ([5000], 25600)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_bounds_far_above_the_lengths(pkv, contexts, blocks, in_place):
    # bounds that leave the block tables, or the sums as well, in global memory, in clusters and without
    e = Evict(contexts, seed=47, ties=2, max_blocks=blocks)
    _check_evict(pkv, e, [c // 2 for c in contexts], 4, 30, in_place)


def test_evict_streams_and_graphs(pkv):
    e = Evict([700, 90], 2, seed=48)
    want = _run_evict(pkv, e, [300, 50], 4, 30)
    side = torch.cuda.Stream()
    got = _run_evict(pkv, e, [300, 50], 4, 30, stream=side)
    assert torch.equal(got[0].buffer.view(torch.int16), want[0].buffer.view(torch.int16)) and np.array_equal(got[3], want[3])
    # captured, and replayed over fresh contents of the same buffers
    pool, fresh = _pool(pkv, e.pool), _pool(pkv, e.pool)
    sums, budgets, lens = U.to_dev(e.sums), U.to_dev(np.array([300, 50], np.int32)), U.to_dev(e.lens)
    bt, kept = U.to_dev(e.bt), torch.full((2, 2, 8, 300), -1, dtype=torch.int32, device=U.dev())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_evict(pool, bt, bt.stride(0), bt.stride(1), lens, budgets, sums, sums, 4, 30, e.max_context, kept)
    for _ in range(3):
        pool.buffer.copy_(fresh.buffer)
        sums.copy_(U.to_dev(e.sums))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool.buffer.view(torch.int16), want[0].buffer.view(torch.int16))
        assert np.array_equal(kept.cpu().numpy(), want[3])
        assert all(torch.equal(sums[s, :, :, :n], want[2][s, :, :, :n]) for s, n in ((0, 700), (1, 90)))


def test_evict_special_sums(pkv):
    e = Evict([300, 90], 2, seed=43)
    r = np.random.RandomState(5)
    values = np.array([0.0, -0.0, 1.0, -1.0, np.inf, -np.inf, np.nan, 1e-45, -1e-45, 3.4e38], np.float32)
    e.sums[:] = values[r.randint(0, len(values), e.sums.shape)]
    e.sums[0, 0, 0] = np.nan
    e.sums[0, 0, 1] = 0
    e.sums[0, 0, 2] = -np.inf
    for budgets in ([100, 45], [299, 1], [2, 89], [260, 80]):
        for in_place in (False, True):
            _check_evict(pkv, e, budgets, 1, 3, in_place)


@pytest.mark.parametrize("contexts", [[2048], [5000], [20000], [3000, 2500]])  # clusters of 4, 4, 8 and 2
def test_evict_special_sums_in_clusters(pkv, contexts):
    """Digits of a cluster divide the range of the keys: the whole range, none at all, one value far from the others, ties."""
    e = Evict(contexts, seed=49)
    r = np.random.RandomState(50)
    plain = e.sums.copy()
    n = plain.shape[-1]
    kinds = [plain * np.where(r.rand(*plain.shape) < 0.5, -1, 1).astype(np.float32), np.full_like(plain, 0.25),
             np.where(r.rand(*plain.shape) < 0.001, np.float32(1e30), np.float32(1e-30)), np.floor(plain * 2),
             r.randint(0, 1 << 32, plain.shape, dtype=np.uint64).astype(np.uint32).view(np.float32)]  # NaN, infinities, all sizes
    one = np.zeros_like(plain)
    one[..., n // 3] = 1
    kinds.append(one)
    for sums in kinds:
        e.sums = np.ascontiguousarray(sums.astype(np.float32))
        for keep in (0, 9, 10, 1501, n):
            _check_evict(pkv, e, [min(keep, c) for c in contexts], 4, 5, in_place=keep % 2 == 1)


def test_evict_other_strides(pkv):
    """Layers outside sequences, in the sums and the tables, and rows of sums longer than the bound."""
    e = Evict([700, 90, 0, 1300], 2, seed=52, extra=3)
    want = _run_evict(pkv, e, [300, 50, 4, 1300], 4, 30)
    pool, status = _pool(pkv, e.pool), _status()
    sums = U.to_dev(np.ascontiguousarray(e.sums.transpose(1, 0, 2, 3))).transpose(0, 1)
    bt = U.to_dev(np.ascontiguousarray(e.bt.transpose(1, 0, 2))).transpose(0, 1)
    kept = torch.full((4, 2, 8, 1300), -1, dtype=torch.int32, device=U.dev())
    pkv.kv_evict(pool, bt, bt.stride(0), bt.stride(1), U.to_dev(e.lens), U.to_dev(np.array([300, 50, 4, 1300], np.int32)), sums,
                 sums, 4, 30, e.max_context, kept, None, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and np.array_equal(kept.cpu().numpy(), want[3])
    assert torch.equal(pool.buffer.view(torch.int16), want[0].buffer.view(torch.int16))
    for s, n in enumerate((700, 90, 0, 1300)):
        assert torch.equal(sums[s, :, :, :n], want[2][s, :, :, :n])
        assert np.array_equal(sums[s, :, :, n:].cpu().numpy(), e.sums[s, :, :, n:])


def test_evict_bad_arguments_on_the_device(pkv):
    e = Evict([100, 200, 64, 33, 50], 2, seed=44)
    e.lens = np.array([-1, 200, e.max_context + 1, 33, 50], np.int32)
    for in_place in (False, True):
        _check_evict(pkv, e, [10, 60, 10, -1, 30], 2, 5, in_place)
        _check_evict(pkv, e, [10, 60, 10, 20, 1000], 2, 5, in_place, width=50)  # 60 are too many, 1000 keep all 50
    bt = e.bt.copy()
    e.lens = np.array([100, 200, 64, 33, 50], np.int32)
    bt[1, 0, 3], bt[1, 1, 1], bt[4, 1, 0] = -7, e.pool.num_pages, e.pool.num_pages + 5
    _check_evict(pkv, e, [40, 60, 10, 20, 30], 2, 5, bt=bt)


def test_evict_rows_past_four_gigabytes(pkv):
    pages = 140000
    pool = pkv.KVPool(pages, device=U.dev())
    pool.buffer.zero_()
    e = Evict([200], 1, seed=45)
    host = e.pool.data
    ids = pages - 1 - np.arange(13)[::-1] * 640                    # 4.3 GB and less apart, the last page among them
    bt = np.full((1, 1, e.bt.shape[2]), -1, np.int32)
    bt[0, 0, :13] = ids[np.random.RandomState(3).permutation(13)]
    pool.view().view(torch.int16)[torch.from_numpy(bt[0, 0, :13].astype(np.int64)).to(U.dev())] = \
        U.to_dev(host[e.bt[0, 0, :13]].view(np.int16))
    got, _, _, kept, _, status = _run_evict(pkv, e, [120], 4, 10, bt=bt, pool=pool)
    want = oracle.Pool(e.pool.num_pages)
    want.data[:] = host
    bounded.evict(want, e.bt, e.lens, [120], e.sums, 4, 10, e.max_context, 120)
    there = got.view().view(torch.int16)[torch.from_numpy(bt[0, 0, :13].astype(np.int64)).to(U.dev())].cpu().numpy()
    assert status == 0 and np.array_equal(there.view(np.uint16), want.data[e.bt[0, 0, :13]])


def test_evict_refusals_of_the_binding(pkv):
    e = Evict([100], 2, seed=46)
    pool, sums = _pool(pkv, e.pool), U.to_dev(e.sums)
    bt, lens, budgets = U.to_dev(e.bt), U.to_dev(e.lens), U.to_dev(np.array([50], np.int32))
    kept = torch.zeros(1, 2, 8, 50, dtype=torch.int32, device=U.dev())

    def call(**kw):
        a = dict(lens=lens, budgets=budgets, sums=sums, new=torch.zeros_like(sums), kept=kept, new_lens=None) | kw
        pkv.kv_evict(pool, bt, bt.stride(0), bt.stride(1), a["lens"], a["budgets"], a["sums"], a["new"], 0, 0, e.max_context,
                     a["kept"], a["new_lens"])

    call()
    for kw in (dict(lens=lens.long()), dict(budgets=budgets.cpu()), dict(sums=sums.half()), dict(sums=sums[:, :, :4]),
               dict(new=torch.zeros_like(sums)[..., :-1]), dict(kept=kept[..., :25]), dict(kept=kept[:, :1]),
               dict(new=sums.transpose(0, 1)), dict(new_lens=lens.float())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(new_lens=lens), dict(new_lens=budgets)):
        with pytest.raises(pkv.PkvError) as err:
            call(**kw)
        assert err.value.code == -2


def test_nothing_cached(pkv):
    """Bounds of 0: zero rows, lengths of 0, and the report where a length is not 0."""
    e = Evict([100, 40], 2, seed=47)
    pool, bt = _pool(pkv, e.pool), U.to_dev(e.bt)
    sums = torch.empty(2, 2, 8, 0, device=U.dev())
    for lens, new, code in (([0, 0], [0, 0], 0), ([0, 40], [0, 40], 2)):
        lens, budgets, status = U.to_dev(np.array(lens, np.int32)), U.to_dev(np.array([7, 0], np.int32)), _status()
        kept = torch.zeros(2, 2, 8, 0, dtype=torch.int32, device=U.dev())
        got = torch.full((2,), -1, dtype=torch.int32, device=U.dev())
        pkv.kv_evict(pool, bt, bt.stride(0), bt.stride(1), lens, budgets, sums, sums, 4, 4, 0, kept, got, status)
        assert got.cpu().tolist() == new and int(status.item()) == code
        q, out, status = torch.zeros(2, 32, 64, dtype=torch.bfloat16, device=U.dev()), torch.ones(2, 32, 64, device=U.dev()), _status()
        pkv.paged_decode_attention_weights(pool, out, q, bt[:, 0], bt.stride(0), lens, 0, 0.125, sums[:, 0], 1.0, None, status)
        assert (out == 0).all() and int(status.item()) == code
        out.fill_(1)
        pkv.paged_window_decode_attention(pool, out, q, bt[:, 0], bt.stride(0), lens, 0, 0.125, 8, 1, status)
        assert (out == 0).all() and int(status.item()) == code
    assert np.array_equal(U.bits(pool.view()), e.pool.data)


def test_attention_refusals_of_the_binding(pkv):
    e = Evict([100, 40], 1, seed=48)
    pool, bt, lens = _pool(pkv, e.pool), U.to_dev(e.bt[:, 0]), U.to_dev(np.array([100, 40], np.int32))
    q, out = torch.zeros(2, 32, 64, dtype=torch.bfloat16, device=U.dev()), torch.ones(2, 32, 64, device=U.dev())
    start, sums = U.to_dev(np.array([0, 1, 2], np.int32)), torch.zeros(2, 8, e.max_context, device=U.dev())
    base = dict(out=out, q=q, bt=bt, lens=lens, start=start, sums=sums, ws=None, status=None)

    def window(**kw):
        a = base | kw
        pkv.paged_window_decode_attention(pool, a["out"], a["q"], a["bt"], 64, a["lens"], e.max_context, 0.125, 8, 1, a["status"])

    def prefill(**kw):
        a = base | kw
        pkv.paged_window_prefill_attention(pool, a["out"], a["q"], a["start"], a["bt"], 64, a["lens"], 1, e.max_context, 0.125, 8,
                                           1, a["status"])

    def weights(**kw):
        a = base | kw
        pkv.paged_decode_attention_weights(pool, a["out"], a["q"], a["bt"], 64, a["lens"], e.max_context, 0.125, a["sums"], 1.0,
                                           a["ws"], a["status"])

    common = (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :, ::2]), dict(q=q.view(64, 64)), dict(out=out.half()),
              dict(out=out.cpu()), dict(out=out[:, :16]), dict(out=out[..., :32].contiguous()), dict(lens=lens.long()),
              dict(lens=lens.cpu()), dict(bt=bt.long()), dict(bt=bt[:, ::2]), dict(bt=bt.cpu()), dict(status=start.long()))
    for call in (window, prefill, weights):
        for kw in common:
            with pytest.raises(ValueError):
                call(**kw)
    for call in (window, weights):
        for kw in (dict(q=q[:1]), dict(out=out[:1])):
            with pytest.raises(ValueError):
                call(**kw)
    for kw in (dict(start=start.long()), dict(start=start[:2]), dict(start=start.cpu())):
        with pytest.raises(ValueError):
            prefill(**kw)
    for kw in (dict(sums=sums.double()), dict(sums=sums[:1]), dict(sums=sums[:, :4]), dict(sums=sums[..., :-1]),
               dict(sums=sums.transpose(1, 2)), dict(sums=sums.cpu()), dict(ws=torch.zeros(16))):
        with pytest.raises(ValueError):
            weights(**kw)
    for kw in (dict(sums=sums[:, :1].expand(2, 8, -1)), dict(sums=sums[:1].expand(2, -1, -1))):  # shared elements
        with pytest.raises(pkv.PkvError) as err:
            weights(**kw)
        assert err.value.code == -2
    assert (out == 1).all() and (sums == 0).all()


# ---- together -----------------------------------------------------------------------------------------
def test_a_bounded_cache_from_prompt_to_eviction_and_on(pkv):
    """Two layers: prompts by windowed prefill, decode steps that add up weights, eviction, pages given back, decode steps on
    the smaller caches (plain and windowed), all on one stream, against the oracle."""
    layers, prompts, steps, window, sinks, recent = 2, [75, 40], 6, 32, 2, 8
    r = np.random.RandomState(51)
    alloc = pkv.Allocator(64, num_layers=layers, max_context=160, max_seqs=2, free_order=r.permutation(64).astype(np.int32))
    for s, n in enumerate(prompts):
        assert alloc.admit(s, n, 40)[0] == 0
    host, pool, status = oracle.Pool(64), pkv.KVPool(64, device=U.dev()), _status()
    pool.buffer.copy_(U.to_dev(host.data).view(-1))
    scale = 0.125
    bits = lambda *shape: (r.standard_normal(shape).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)  # noqa: E731
    lens = np.array(prompts, np.int32)
    sums_h = np.zeros((2, layers, 8, 160))
    sums = torch.zeros(2, layers, 8, 160, device=U.dev())
    check = lambda got, ref, tol=3e-5: np.abs(got.double().cpu().numpy() - ref).max() < tol  # noqa: E731

    def append(positions):
        """New rows at (sequence, position) pairs, in every layer."""
        for layer in range(layers):
            k, v = bits(len(positions), 8, 64), bits(len(positions), 8, 64)
            slots = np.array([alloc.page(s, layer, t // 16) * 16 + t % 16 for s, t in positions], np.int32)
            oracle.kv_append(host, k, v, slots)
            pkv.kv_append(pool, U.to_dev(k), U.to_dev(v), U.to_dev(slots), status)

    append([(s, t) for s, n in enumerate(prompts) for t in range(n)])
    starts = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    for layer in range(layers):
        bt = alloc.block_tables()
        q = bits(int(starts[-1]), 32, 64)
        out = torch.empty(int(starts[-1]), 32, 64, device=U.dev())
        dev = U.to_dev(bt)
        pkv.paged_window_prefill_attention(pool, out, U.to_dev(q), U.to_dev(starts), dev[:, layer], dev.stride(0), U.to_dev(lens),
                                           max(prompts), 160, scale, window, sinks, status)
        assert check(out, bounded.paged_window_attention(host, q, starts, bt[:, layer], lens, scale, window, sinks,
                                                         max(prompts), 160)[0])

    def step(weigh):
        nonlocal lens
        append([(s, int(lens[s])) for s in range(2)])
        lens = lens + 1
        bt = alloc.block_tables()
        dev, dl = U.to_dev(bt), U.to_dev(lens)
        for layer in range(layers):
            q, out = bits(2, 32, 64), torch.empty(2, 32, 64, device=U.dev())
            if weigh:
                pkv.paged_decode_attention_weights(pool, out, U.to_dev(q), dev[:, layer], dev.stride(0), dl, 160, scale,
                                                   sums[:, layer], 0.9, None, status)
                ref, _, _, w = bounded.window_decode(host, q, bt[:, layer], lens, scale, 1 << 30, 0, 160)
                for (s, _, g), (t, x) in w.items():
                    sums_h[s, layer, g, :lens[s]] *= 0.9
                    sums_h[s, layer, g, t] += x.sum(0)
            else:
                pkv.paged_window_decode_attention(pool, out, U.to_dev(q), dev[:, layer], dev.stride(0), dl, 160, scale,
                                                  window, sinks, status)
                ref = bounded.window_decode(host, q, bt[:, layer], lens, scale, window, sinks, 160)[0]
            assert check(out, ref)

    for _ in range(steps):
        step(True)
    assert np.abs(sums.double().cpu().numpy() - sums_h).max() < 1e-4
    budgets = np.array([40, 33], np.int32)
    bt = alloc.block_tables()
    kept = torch.full((2, layers, 8, 40), -1, dtype=torch.int32, device=U.dev())
    new_lens = torch.zeros(2, dtype=torch.int32, device=U.dev())
    old = sums.cpu().numpy()
    pkv.kv_evict(pool, U.to_dev(bt), bt.shape[1] * bt.shape[2], bt.shape[2], U.to_dev(lens), U.to_dev(budgets), sums, sums, sinks,
                 recent, 160, kept, new_lens, status)
    _, want_kept, lens, _ = bounded.evict(host, bt, lens, budgets, old, sinks, recent, 160, 40)
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want_kept) and new_lens.cpu().numpy().tolist() == lens.tolist() == [40, 33]
    assert np.array_equal(U.bits(pool.view()), host.data)
    sums_h = sums.double().cpu().numpy()
    assert (sums_h[0, :, :, 40:81] == 0).all()
    for s in range(2):
        alloc.truncate(s, int(lens[s]))
    for weigh in (True, False, True):
        step(weigh)
    assert int(status.item()) == 0
