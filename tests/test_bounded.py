"""Window attention, weight sums and eviction: the calls' refusals and the oracle's pins (no GPU)."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import bounded
from tests import bounded_util as B
from workloads import rng


@pytest.fixture(scope="module")
def b():
    from paged_kv_cache_180_gb300 import build
    build.build()
    from paged_kv_cache_180_gb300 import binding
    return binding


BASE = 1 << 20  # a fake, aligned device address: refused calls never dereference it


def _pool(b):
    return b.kv_pool_create(BASE, BASE + 16384, 0, 8)


def test_window_decode_refusals(b):
    d = _pool(b)
    P = ctypes.c_void_p

    def call(**kw):
        g = lambda k, v: kw.get(k, v)  # noqa: E731
        return b._lib.pkv_paged_window_decode_attention(
            ctypes.byref(d), P(g("out", BASE)), P(g("q", BASE)), g("hq", 32), P(g("bt", BASE)), g("stride", 128),
            P(g("lens", BASE)), g("n", 4), g("max", 2048), g("scale", 0.125), g("window", 64), g("sinks", 4), None,
            g("flags", 0), None)

    for kw, code in [(dict(hq=16), -3), (dict(q=0), -1), (dict(out=0), -1), (dict(bt=0), -1), (dict(lens=0), -1),
                     (dict(scale=float("inf")), -5), (dict(scale=float("nan")), -5), (dict(scale=3e38), -5), (dict(q=BASE + 8), -4),
                     (dict(out=BASE + 8), -4), (dict(lens=BASE + 2), -4), (dict(bt=BASE + 1), -4), (dict(n=-1), -2),
                     (dict(max=-1), -2), (dict(max=0x7fffffff), -2), (dict(stride=-1), -2), (dict(window=0), -2),
                     (dict(window=-5), -2), (dict(sinks=-1), -2), (dict(flags=4), -2), (dict(n=(1 << 24) + 1), -2)]:
        assert call(**kw) == code, kw
    assert call(n=0) == 0
    assert call(n=0, window=0) == -2


def test_window_prefill_refusals(b):
    d = _pool(b)
    P = ctypes.c_void_p

    def call(**kw):
        g = lambda k, v: kw.get(k, v)  # noqa: E731
        return b._lib.pkv_paged_window_prefill_attention(
            ctypes.byref(d), P(g("out", BASE)), P(g("q", BASE)), g("hq", 32), g("rows", 64), P(g("start", BASE)), P(g("bt", BASE)),
            g("stride", 128), P(g("lens", BASE)), g("n", 4), g("mq", 16), g("max", 2048), g("scale", 0.125),
            g("window", 64), g("sinks", 4), None, g("flags", 0), None)

    for kw, code in [(dict(hq=16), -3), (dict(q=0), -1), (dict(out=0), -1), (dict(start=0), -1), (dict(bt=0), -1),
                     (dict(lens=0), -1), (dict(scale=float("inf")), -5), (dict(scale=3e38), -5), (dict(q=BASE + 8), -4),
                     (dict(out=BASE + 4), -4), (dict(start=BASE + 2), -4), (dict(n=-1), -2), (dict(max=-1), -2),
                     (dict(max=0x7fffffff), -2), (dict(stride=-1), -2), (dict(rows=-1), -2), (dict(mq=-1), -2),
                     (dict(mq=(1 << 20) + 1), -2), (dict(window=0), -2), (dict(sinks=-1), -2), (dict(flags=4), -2),
                     (dict(n=1 << 24, mq=1 << 20), -2)]:
        assert call(**kw) == code, kw
    for kw in (dict(n=0), dict(mq=0), dict(rows=0)):
        assert call(**kw) == 0, kw


def test_weights_refusals(b):
    d = _pool(b)
    P = ctypes.c_void_p

    def call(**kw):
        g = lambda k, v: kw.get(k, v)  # noqa: E731
        return b._lib.pkv_paged_decode_attention_weights(
            ctypes.byref(d), P(g("out", BASE)), P(g("q", BASE)), g("hq", 32), P(BASE), 128, P(g("lens", BASE)),
            g("n", 4), g("max", 2048), g("scale", 0.125), P(g("sums", BASE)), g("seq", 8 * 2048), g("head", 2048),
            g("decay", 1.0), P(g("ws", 0)), g("wsb", 0), None, g("flags", 0), None)

    for kw, code in [(dict(hq=16), -3), (dict(q=0), -1), (dict(sums=0), -1), (dict(sums=BASE + 2), -4),
                     (dict(decay=-0.1), -5), (dict(decay=1.5), -5), (dict(decay=float("nan")), -5),
                     (dict(scale=float("inf")), -5), (dict(head=2047), -2), (dict(seq=8 * 2048 - 1), -2), (dict(head=-1), -2),
                     (dict(seq=-1), -2), (dict(flags=8), -2), (dict(max=(1 << 30) + 1, seq=1 << 40, head=1 << 35), -2),
                     (dict(n=-1), -2), (dict(max=57345, seq=8 * 57345, head=57345), -1),
                     (dict(max=57345, seq=8 * 57345, head=57345, ws=BASE + 8, wsb=1 << 30), -4),
                     (dict(max=57345, seq=8 * 57345, head=57345, ws=BASE, wsb=1024), -6)]:
        assert call(**kw) == code, kw
    assert call(n=0) == 0
    assert call(n=0, seq=2048, head=4 * 2048) in (0, -2)
    for kw, code in [(dict(seq=(1 << 38) + 1), -2), (dict(head=1 << 61, seq=0), -2), (dict(max=0, sums=0, lens=0), -1)]:
        assert call(**kw) == code, kw
    assert b.weights_workspace_bytes((1 << 24) + 1, 70000) == 0 and b.weights_workspace_bytes(4, (1 << 30) + 1) == 0
    assert b.weights_workspace_bytes(1 << 24, 1 << 30) == 1 << 61
    assert b.weights_workspace_bytes(4, 57344) == 0 and b.weights_workspace_bytes(-1, 70000) == 0
    assert b.weights_workspace_bytes(4, 57345) == 4 * 8 * 3585 * 16 * 16  # a float4 for every token of every unit


def test_evict_refusals(b):
    d = _pool(b)
    P = ctypes.c_void_p
    far = 1 << 30

    def call(**kw):
        g = lambda k, v: kw.get(k, v)  # noqa: E731
        return b._lib.pkv_kv_evict(
            ctypes.byref(d), P(g("bt", BASE)), g("bts", 256), g("ls", 128), g("layers", 2), P(g("lens", BASE)),
            P(g("budgets", BASE + 64)), g("n", 4), g("max", 2048), g("budget", 1024), g("sinks", 4), g("recent", 16),
            P(g("sums", far)), P(g("new", 2 * far)), g("seq", 2 * 8 * 2048), g("layer", 8 * 2048), g("head", 2048),
            P(g("kept", 3 * far)), g("ks", 1024), P(g("nl", 4 * far)), None, None)

    for kw, code in [(dict(bt=0), -1), (dict(lens=0), -1), (dict(budgets=0), -1), (dict(sums=0), -1), (dict(new=0), -1),
                     (dict(kept=0), -1), (dict(bt=BASE + 2), -4), (dict(kept=3 * far + 1), -4), (dict(nl=4 * far + 2), -4),
                     (dict(n=-1), -2), (dict(layers=0), -2), (dict(max=-1), -2), (dict(max=(1 << 30) + 1), -2),
                     (dict(budget=-1), -2), (dict(ks=1023), -2), (dict(sinks=-1), -2), (dict(recent=-1), -2),
                     (dict(bts=-1), -2), (dict(ls=-1), -2), (dict(head=2047), -2), (dict(layer=8 * 2048 - 1), -2),
                     (dict(seq=2 * 8 * 2048 - 1), -2), (dict(new=far + 4096), -2), (dict(nl=BASE), -2), (dict(nl=BASE + 64), -2),
                     (dict(kept=far), -2), (dict(kept=2 * far + 64), -2), (dict(kept=BASE), -2), (dict(new=BASE), -2),
                     (dict(nl=far + 4), -2), (dict(nl=2 * far), -2), (dict(nl=3 * far + 8), -2),
                     (dict(layers=1 << 25), -2)]:
        assert call(**kw) == code, kw
    assert call(n=0) == 0
    # nothing cached: the sums may be null, not the lengths; far strides do not wrap around
    for kw, code in [(dict(max=0, sums=0, new=0, lens=0), -1), (dict(max=0, sums=0, new=0, budget=4, kept=0), -1),
                     (dict(seq=(1 << 38) + 1), -2), (dict(seq=1 << 62), -2), (dict(n=5, seq=1 << 37), -2),
                     (dict(layer=1 << 62), -2), (dict(layers=6, layer=1 << 37), -2), (dict(head=1 << 61), -2),
                     (dict(ks=(1 << 31) + 1), -2)]:
        assert call(**kw) == code, kw


# ---- the oracle itself -----------------------------------------------------------------------
def test_a_wide_window_is_plain_attention():
    c = B.Cache([40, 17, 1, 0, 16], seed=3)
    plain, err = oracle.paged_decode_attention(c.pool, c.q, c.bt, c.lens, c.scale, c.max_context)
    assert err == 0
    for window, sinks in ((40, 0), (1 << 30, 0), (20, 20), (1, 40)):
        got, err, _, _, weights = c.decode(window, sinks)
        assert err == 0 and np.allclose(got, plain, rtol=0, atol=1e-12)
        assert all(np.allclose(w.sum(1), 1) for _, w in weights.values())


def test_windows_by_a_dense_mask():
    torch = pytest.importorskip("torch")
    c = B.Cache([70, 33], nodes=[50, 33], seed=4)
    for window, sinks in ((1, 0), (1, 3), (7, 0), (16, 16), (20, 5), (64, 64)):
        got, err, _, _ = c.prefill(window, sinks)
        assert err == 0
        for s in range(2):
            ctx, n = int(c.lens[s]), c.nodes[s]
            kv = c.pool.data[c.bt[s, :(ctx + 15) // 16]].transpose(1, 2, 0, 3, 4).reshape(2, 8, -1, 64)[:, :, :ctx]
            K, V = (torch.from_numpy(rng.bf16_bits_to_f64(x)).repeat_interleave(4, 0) for x in kv)
            q = torch.from_numpy(rng.bf16_bits_to_f64(c.q[c.starts[s]:c.starts[s] + n])).transpose(0, 1)
            i, t = torch.arange(ctx - n, ctx)[:, None], torch.arange(ctx)[None]
            hide = (t > i) | ((i - t >= window) & (t >= sinks))
            w = torch.softmax((q @ K.transpose(1, 2) * c.scale).masked_fill(hide, -torch.inf), -1)
            want = (w @ V).transpose(0, 1).numpy()
            assert np.abs(got[c.starts[s]:c.starts[s] + n] - want).max() < 1e-12


def test_evict_by_hand():
    c = B.Cache([5, 20], seed=5)
    sums = np.zeros((2, 1, 8, 64), np.float32)
    sums[0, 0, :, :5] = [9, 1, 3, 3, 0]
    sums[0, 0, 1, :5] = [0, 0, -0.0, np.nan, -1]
    sums[0, 0, 2, :5] = [np.inf, -np.inf, np.nan, np.nan, 2]
    before = c.pool.data.copy()
    new, kept, lens, err = bounded.evict(c.pool, c.bt[:, None], c.lens, [3, 20], sums, 0, 0, 64, 20)
    assert err == 0 and lens.tolist() == [3, 20]
    assert kept[0, 0, 0, :3].tolist() == [0, 2, 3] and kept[0, 0, 1, :3].tolist() == [0, 1, 2]
    assert kept[0, 0, 2, :3].tolist() == [0, 1, 4] and kept[0, 0, 0, 3] == -1
    assert new[0, 0, 0, :6].tolist() == [9, 3, 3, 0, 0, 0] and kept[1, 0, 3].tolist() == list(range(20))
    page = c.bt[0, 0]
    assert np.array_equal(c.pool.data[page, :, 0, 1], before[page, :, 0, 2])
    assert np.array_equal(c.pool.data[page, :, 0, 2], before[page, :, 0, 3])
    assert np.array_equal(c.pool.data[page, :, 1], before[page, :, 1])
    # sinks and recent tokens come first, then the sums
    assert bounded.evict(c.pool, c.bt[:, None], [5, 20], [3, 4], sums, 1, 1, 64, 20)[1][0, 0, 0, :3].tolist() == [0, 2, 4]
    assert bounded.evict(c.pool, c.bt[:, None], [5, 20], [2, 4], sums, 4, 9, 64, 20)[1][0, 0, 0, :2].tolist() == [0, 1]
    _, _, lens, err = bounded.evict(c.pool, c.bt[:, None], [5, 65], [6, 4], sums, 4, 9, 64, 4)
    assert err == 2 | 32 and lens.tolist() == [5, 65]


def test_the_bounds_reject_lost_keys_and_a_lost_term():
    c = B.Cache([900], seed=6)
    for window, sinks in ((300, 4), (1000, 0)):
        ref, _, size, spread, weights = c.decode(window, sinks)
        keys = weights[0, 0, 0][0].size
        lim = B.decode_bound(ref, size, spread, c.scale, keys, False)
        assert lim.max() < 1e-3                       # far below the outputs, which are of the order of 0.3
        for w2, s2 in ((window - 1, sinks), (window, sinks + 1)):
            other = c.decode(w2, s2)[0]
            if window < 900:
                assert (np.abs(other - ref) > lim).mean() > 0.2
        t, w = weights[0, 0, 0]
        V = rng.bf16_bits_to_f64(c.pool.data[c.bt[0, t // 16], 1, 0, t % 16])
        one = (w.astype(np.float32).view(np.uint32) & 0xffff0000).view(np.float32).astype(np.float64)
        assert (np.abs(one @ V - w @ V) > lim[0, :4]).mean() > 0.5
