"""GPU parity of tree attention, path commit and page copies (through the C ABI) against the FP64 oracle.

Tree attention is held to a bound derived from its arithmetic (spec_util.bound); commits and copies are
bit-exact over the whole pool.  Untouched pool slots hold NaN patterns throughout.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import speculative as spec
from tests import gpu_util as U
from tests import spec_util as S
from workloads import configs, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_180_gb300 as p
    return p


def _pool(pkv, host: oracle.Pool):
    pool = pkv.KVPool(host.num_pages, device=U.dev())
    pool.buffer.copy_(U.to_dev(host.data).view(-1))
    return pool


class Run:
    """One tree call on the device for a TreeCase."""

    def __init__(self, pkv, c, bf16=False, scale=None, pool=None, bt=None, guard=3, workspace=None, **kw):
        self.pkv, self.c = pkv, c
        self.scale = c.wl.scale if scale is None else scale
        self.pool = _pool(pkv, c.pool) if pool is None else pool
        self.out = torch.full((max(c.rows, 1) + guard, 32, 64), float("nan"), device=U.dev(),
                              dtype=torch.bfloat16 if bf16 else torch.float32)
        self.q = torch.cat([U.to_dev(c.q), torch.full((guard, 32, 64), float("nan"), dtype=torch.bfloat16,
                                                      device=U.dev())])
        self.mask = torch.cat([U.to_dev(c.mask), torch.full((guard, c.mask.shape[1]), -1, dtype=torch.int32,
                                                            device=U.dev())])
        self.starts, self.lens = U.to_dev(c.starts), U.to_dev(c.lens)
        self.bt = U.to_dev(c.bt if bt is None else bt)
        self.status = torch.zeros(1, dtype=torch.int32, device=U.dev())
        self.ws = pkv.tree_workspace(len(c.nodes), c.max_query) if workspace is None else workspace
        self.kw = kw

    def call(self, **kw):
        self.pkv.paged_tree_attention(self.pool, self.out, self.q, self.starts, self.mask, self.bt, self.bt.shape[1],
                                      self.lens, self.c.max_query, self.c.max_context, self.scale, self.ws, self.status,
                                      **self.kw, **kw)
        return self

    def result(self):
        torch.cuda.synchronize()
        assert torch.isnan(self.out[self.c.rows:]).all(), "rows behind the last sequence were written"
        return self.out[:self.c.rows].double().cpu().numpy(), int(self.status.item())


def _check(pkv, c, bf16=False, scale=None, **kw):
    scale = c.wl.scale if scale is None else scale
    got, status = Run(pkv, c, bf16, scale, **kw).call().result()
    ref, err, size, spread = c.reference(scale)
    assert status == err
    lim = S.bound(ref, size, spread, scale, int(max(c.lens)), bf16)
    S.assert_within(got, ref, lim, "tree attention")
    return got


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("contexts,nodes", [
    ([1], [1]), ([16], [16]), ([17], [1]), ([40], [5]), ([64], [8]), ([65], [9]), ([128], [16]), ([130], [17]),
    ([600], [6]), ([300], [31]), ([300], [32]), ([300], [33]), ([300], [64]), ([300], [65]), ([260], [130]),
    ([200], [200]), ([5000], [20]),
    ([2048, 128, 512, 1024], [16, 16, 16, 16]),
    ([77, 1, 0, 300, 64, 63, 129, 33], [5, 1, 0, 64, 64, 1, 12, 0]),
])
def test_shapes(pkv, contexts, nodes, bf16):
    _check(pkv, S.TreeCase(contexts, nodes, seed=40 + len(nodes) + nodes[0]), bf16)


@pytest.mark.parametrize("bf16", [False, True])
def test_ragged_batch_of_trees(pkv, bf16):
    r = np.random.RandomState(7)
    nodes = r.randint(0, 65, 48).tolist()
    contexts = [int(max(n, x)) for n, x in zip(nodes, r.randint(1, 900, 48))]
    _check(pkv, S.TreeCase(contexts, nodes, seed=50), bf16)


@pytest.mark.parametrize("scale", [1.0, -0.125, -1.0, 0.0, 1e-30])
def test_scales(pkv, scale):
    _check(pkv, S.TreeCase([700, 40, 90], [12, 40, 3], seed=51), scale=scale)


@pytest.mark.parametrize("bf16", [False, True])
def test_scores_that_outgrow_the_first_block(pkv, bf16):
    # later keys score hundreds of times higher (or every later key far lower) than the first 64: a reference taken
    # from those alone would overflow (or vanish), on whole rows and on some of them
    for gain, where in ((64, slice(100, 400)), (256, slice(333, 334)), (1 / 64, slice(70, 600)), (512, slice(590, 600))):
        c = S.TreeCase([600, 70], [20, 9], seed=71)
        for s in range(2):
            for t in range(*where.indices(int(c.lens[s]))):
                k = c.pool.data[c.bt[s, t // 16], 0, :, t % 16]
                k[:] = ((rng.bf16_bits_to_f64(k) * gain).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        _check(pkv, c, bf16)


def test_large_values_stay_finite(pkv):
    # V about 2^101, and a reference below the maximum: sums of 2^x V pass the range of fp32, the output does not
    c = S.TreeCase([400], [10], seed=72)
    for t in range(400):
        v = c.pool.data[c.bt[0, t // 16], 1, :, t % 16]
        v[:] = (v & 0x8000) | 0x7200 | (v & 0x7F)
        if t >= 128:
            k = c.pool.data[c.bt[0, t // 16], 0, :, t % 16]
            k[:] = ((rng.bf16_bits_to_f64(k) * 8).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    got = _check(pkv, c)
    assert np.isfinite(got).all()


def test_wide_mask_rows_and_ignored_bits(pkv):
    c = S.TreeCase([90, 33], [7, 33], seed=52, words=5)
    got = _check(pkv, c)
    c.mask[:7, 1:] = -1
    c.mask[:7, 0] |= np.int32(-128)                 # bits 7 .. 31
    c.mask[7:, 2:] = -1
    c.mask[7:, 1] |= np.int32(-2)                   # bits 33 .. 63
    assert np.array_equal(Run(pkv, c).call().result()[0], got)


def test_rows_that_see_nothing_are_zero(pkv):
    # no prefix and no bits; a prefix alone; a node that does not see itself; nothing but a later block
    def visible(s, n):
        see = np.zeros((n, n), bool)
        if s == 2:
            see[:, n - 1] = True
        if s == 3:
            see[n // 2:, :3] = True
        return see
    c = S.TreeCase([9, 30, 150, 150], [9, 4, 150, 150], seed=53, visible=visible)
    got = _check(pkv, c)
    assert not got[:9].any() and got[9:13].any()


def test_nonfinite_nodes_reach_only_the_rows_that_see_them(pkv):
    # one node's K and another's V hold NaN and infinities; half of the rows see them
    bad_k, bad_v, bad_inf = 2, 5, 70
    def visible(s, n):
        see = S.random_tree(n, np.random.RandomState(s))
        see[:, [bad_k, bad_v, bad_inf]] = False
        see[0::8, bad_k] = see[1::8, bad_v] = see[2::8, bad_inf] = True
        return see
    for bf16 in (False, True):
        c = S.TreeCase([300, 97], [97, 97], seed=54, visible=visible)
        def poke(node, kv, bits):
            for s in range(2):
                t = int(c.lens[s]) - 97 + node
                c.pool.data[c.bt[s, t // 16], kv, :, t % 16, 3::7] = bits
        clean, _, size, spread = c.reference()
        poke(bad_k, 0, 0x7FC0)
        poke(bad_v, 1, 0x7FC0)
        poke(bad_inf, 1, 0xFF80)
        got, status = Run(pkv, c, bf16).call().result()
        assert status == 0
        lim = S.bound(clean, size, spread, c.wl.scale, 300, bf16)
        for s in range(2):
            j = np.arange(97) % 8
            rows = c.starts[s] + np.arange(97)
            fine = rows[j > 2]
            S.assert_within(got[fine], clean[fine], lim[fine], "rows that do not see the bad nodes")
            assert np.isnan(got[rows[j == 0]]).all()                          # a NaN score: the whole row
            for k, test in ((1, np.isnan), (2, np.isneginf)):
                part = got[rows[j == k]]
                assert test(part[:, :, 3::7]).all()
                ok = np.ones(64, bool)
                ok[3::7] = False
                S.assert_within(part[:, :, ok], clean[rows[j == k]][:, :, ok], lim[rows[j == k]][:, :, ok],
                                "other dims of rows that see a bad V")


def test_bad_sequences_beside_good_ones(pkv):
    # more nodes than tokens; a context past the tables; good ones between
    c = S.TreeCase([10, 200, 2049, 70], [11, 20, 3, 9], seed=55, num_pages=40, max_blocks=128)
    got = _check(pkv, c)
    assert not got[:11].any() and not got[31:34].any() and got[34:].any()


def test_rows_past_the_queries_are_refused(pkv):
    c = S.TreeCase([50, 60], [5, 6], seed=56)
    good, _ = Run(pkv, c).call().result()
    r = Run(pkv, c, guard=0)
    r.q, r.out = r.q[:8].contiguous(), r.out[:8].contiguous()
    r.call()
    torch.cuda.synchronize()
    assert int(r.status.item()) == spec.ERR_CONTEXT
    assert np.array_equal(r.out[:5].double().cpu().numpy(), good[:5]) and not r.out[5:].any()


def test_bad_pages_are_left_out(pkv):
    c = S.TreeCase([200, 90, 20], [20, 30, 20], seed=57)
    c.bt[0, 5] = c.wl.num_pages + 7
    c.bt[1, 0] = -1
    c.bt[2, :2] = 1 << 30                             # a sequence without a page
    got = _check(pkv, c)
    assert not got[50:].any()


def test_page_permutation_and_repeats_are_bit_exact(pkv):
    c = S.TreeCase([700, 90, 333], [40, 7, 64], seed=58)
    r = Run(pkv, c)
    first = r.call().result()[0]
    for _ in range(3):
        assert np.array_equal(r.call().result()[0], first)          # the same workspace, call after call
    perm = rng.permutation(rng.stream_key(59, "move"), c.wl.num_pages)
    moved = oracle.Pool(c.wl.num_pages)
    moved.data[perm] = c.pool.data
    bt = np.where(c.bt >= 0, perm[np.maximum(c.bt, 0)], -1).astype(np.int32)
    assert np.array_equal(Run(pkv, c, pool=_pool(pkv, moved), bt=bt).call().result()[0], first)


def test_one_workspace_for_calls_of_many_shapes(pkv):
    ws = pkv.tree_workspace(64, 200)
    for seed, contexts, nodes in [(60, [2000] * 3, [64, 1, 33]), (61, [40] * 64, [3] * 64), (62, [900], [200]),
                                  (63, [1500, 3], [8, 2])]:
        _check(pkv, S.TreeCase(contexts, nodes, seed=seed), workspace=ws)


def test_separate_buffers_and_odd_strides(pkv):
    c = S.TreeCase([300, 45], [20, 5], seed=64)
    pages, half = c.wl.num_pages, 8 * 16 * 64
    k = torch.full((pages, half + 72), float("nan"), dtype=torch.bfloat16, device=U.dev())
    v = torch.full((pages, half + 72), float("nan"), dtype=torch.bfloat16, device=U.dev())
    k[:, :half] = U.to_dev(np.ascontiguousarray(c.pool.k)).view(pages, half)
    v[:, :half] = U.to_dev(np.ascontiguousarray(c.pool.v)).view(pages, half)
    desc = pkv.kv_pool_create(k, v, (half + 72) * 2, pages)
    got = _check(pkv, c, pool=desc)
    # tables inside a multi-layer table, and an output that starts off a 32-byte boundary
    wide = np.full((2, 3, c.bt.shape[1]), -5, np.int32)
    wide[:, 1] = c.bt
    r = Run(pkv, c, pool=desc)
    flat, blocks = U.to_dev(wide).view(-1), c.bt.shape[1]
    store = torch.empty(c.rows * 2048 + 4, dtype=torch.float32, device=U.dev())
    out = store[4:].view(c.rows, 32, 64)
    pkv.paged_tree_attention(desc, out, r.q, r.starts, r.mask, flat[blocks:], 3 * blocks, r.lens, c.max_query,
                             c.max_context, c.wl.scale, r.ws, r.status)
    assert np.array_equal(out.double().cpu().numpy(), got) and int(r.status.item()) == 0


def test_overlap_with_the_append_of_the_nodes(pkv):
    # the nodes' K/V arrive by kv_append right before the overlapped call, six times with other values
    c = S.TreeCase([500, 64, 90], [20, 64, 3], seed=65)
    r = Run(pkv, c)
    slots = np.concatenate([c.wl.slot_mapping(s, 0, int(c.lens[s]) - n, int(c.lens[s])) for s, n in enumerate(c.nodes)])
    for i in range(6):
        kv = [rng.normal_bf16(rng.stream_key(70 + i, tag), 0, c.rows * 8 * 64).reshape(c.rows, 8, 64) for tag in "kv"]
        oracle.kv_append(c.pool, kv[0], kv[1], slots)
        ref, err, size, spread = c.reference()
        dk, dv, ds = U.to_dev(kv[0]), U.to_dev(kv[1]), U.to_dev(slots)
        torch.cuda.synchronize()
        pkv.kv_append(r.pool, dk, dv, ds, r.status)
        got, status = r.call(overlap_previous=True).result()
        assert status == err == 0
        S.assert_within(got, ref, S.bound(ref, size, spread, c.wl.scale, 500, False), f"overlapped call {i}")


def test_graph_replays_follow_their_inputs(pkv):
    c = S.TreeCase([400, 90], [16, 40], seed=66)
    r = Run(pkv, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.call()
    want = r.result()[0]
    r.out[:c.rows].fill_(7)
    graph.replay()
    assert np.array_equal(r.result()[0], want)
    c.q = np.ascontiguousarray(c.q[::-1])
    r.q[:c.rows].copy_(U.to_dev(c.q))
    graph.replay()
    got, status = r.result()
    ref, _, size, spread = c.reference()
    S.assert_within(got, ref, S.bound(ref, size, spread, c.wl.scale, 400, False), "replay with other queries")
    assert status == 0


def test_chain_tree_agrees_with_prefill(pkv):
    chain = lambda s, n: np.tril(np.ones((n, n), bool))  # noqa: E731
    c = S.TreeCase([600, 70, 33], [50, 70, 1], seed=67, visible=chain)
    r = Run(pkv, c).call()
    got, _ = r.result()
    out = torch.empty(c.rows, 32, 64, dtype=torch.float32, device=U.dev())
    pkv.paged_prefill_attention(r.pool, out, r.q[:c.rows], r.starts, r.bt, r.bt.shape[1], r.lens, c.max_query,
                                c.max_context, c.wl.scale, r.status)
    ref, _, size, spread = c.reference()
    lim = 2 * S.bound(ref, size, spread, c.wl.scale, 600, False)
    S.assert_within(got, out.double().cpu().numpy(), lim, "chain tree against prefill")


def test_binding_refuses_what_the_kernel_would_misread(pkv):
    c = S.TreeCase([50], [5], seed=68)
    r = Run(pkv, c)
    for name, bad in (("q", r.q.float()), ("out", r.out.half()), ("mask", r.mask.long()), ("starts", r.starts.long()),
                      ("q", r.q.transpose(1, 2)), ("out", r.out.cpu()), ("starts", r.starts[:1])):
        good = getattr(r, name)
        setattr(r, name, bad)
        with pytest.raises(ValueError):
            r.call()
        setattr(r, name, good)
    with pytest.raises(ValueError):
        pkv.kv_copy_pages(r.pool, r.starts.long(), r.starts)
    with pytest.raises(ValueError):
        pkv.kv_copy_pages(r.pool, r.starts, r.starts[:1])
    with pytest.raises(ValueError):
        pkv.tree_commit(r.pool, r.bt, r.bt.shape[1], 0, 1, r.starts, r.lens, r.mask[:1, 0], r.lens, 64)


# ---- commits and copies ----------------------------------------------------------------------------
def _commit_case(seqs, layers, seed, nodes_hi=40, prefix_hi=50, width=9):
    r = np.random.RandomState(seed)
    n = r.randint(0, nodes_hi + 1, seqs)
    prefix = r.randint(0, prefix_hi + 1, seqs)
    count = np.minimum(r.randint(0, width + 1, seqs), n)
    path = np.full((seqs, width), -7, np.int32)
    for s in range(seqs):
        path[s, :count[s]] = np.sort(r.permutation(int(n[s]))[:count[s]])
    blocks = int((prefix + n).max() + 15) // 16 + 1
    per = np.repeat((prefix + n + 15) // 16, layers)
    used = np.arange(blocks)[None] < per[:, None]
    table = np.full(used.shape, -1, np.int32)
    table[used] = r.permutation(int(used.sum()))
    pool = oracle.Pool(int(used.sum()))
    pool.data[:] = r.randint(0, 1 << 16, pool.data.shape)
    return (pool, table.reshape(seqs, layers, blocks), np.concatenate([[0], np.cumsum(n)]).astype(np.int32),
            (prefix + n).astype(np.int32), path, count.astype(np.int32))


def _commit(pkv, case, max_context=None, with_new=True):
    pool, table, starts, lens, path, count = case
    dpool = _pool(pkv, pool)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    new = torch.full((len(lens) + 1,), -9, dtype=torch.int32, device=U.dev()) if with_new else None
    max_context = table.shape[2] * 16 if max_context is None else max_context
    pkv.tree_commit(dpool, U.to_dev(table), table.shape[1] * table.shape[2], table.shape[2], table.shape[1],
                    U.to_dev(starts), U.to_dev(lens), U.to_dev(path), U.to_dev(count), max_context, new, status)
    torch.cuda.synchronize()
    want, err = spec.tree_commit(pool, table, starts, lens, path, count, max_context)
    assert int(status.item()) == err
    if with_new:
        assert new[:-1].cpu().numpy().tolist() == want.tolist() and int(new[-1]) == -9
    assert np.array_equal(U.bits(dpool.buffer).reshape(pool.data.shape), pool.data)
    return err


@pytest.mark.parametrize("seqs,layers,width,nodes_hi", [(1, 1, 1, 1), (1, 16, 5, 8), (7, 3, 9, 40), (64, 2, 12, 64),
                                                        (3, 2, 200, 300)])
def test_commit_moves_the_path(pkv, seqs, layers, width, nodes_hi):
    for seed in range(3):
        assert _commit(pkv, _commit_case(seqs, layers, 80 + seed, nodes_hi, width=width), with_new=seed != 1) == 0


def test_commit_of_faulty_sequences_moves_nothing_of_them(pkv):
    case = _commit_case(12, 2, 90, nodes_hi=20, width=6)
    pool, table, starts, lens, path, count = case
    n = np.diff(starts)
    ok = [s for s in range(12) if n[s] >= 6]
    assert len(ok) >= 6
    a, b, c, d, e, f = ok[:6]
    for s, row in ((a, [0, 2, 2, 3, 4, 5]), (b, [0, 1, 2, 3, 4, n[b]]), (c, [-1, 2, 3, 4, 5, 6]), (d, [5, 4, 3, 2, 1, 0])):
        path[s], count[s] = row, 6
    count[e] = 7                                      # wider than the list
    lens[f] = 1 << 20                                 # past max_context
    assert _commit(pkv, case) == spec.ERR_PATH | spec.ERR_CONTEXT


def test_commit_leaves_rows_of_bad_pages(pkv):
    case = _commit_case(6, 2, 91, nodes_hi=60, prefix_hi=3, width=20)
    pool, table = case[0], case[1]
    table[:, 0, 1] = pool.num_pages
    table[2:4, 1, 0] = -1
    assert _commit(pkv, case) == spec.ERR_PAGE


@pytest.mark.parametrize("pairs", [1, 3, 16, 151, 700])
def test_copies_move_whole_pages(pkv, pairs):
    r = np.random.RandomState(pairs)
    pool = oracle.Pool(2 * pairs + 3)
    pool.data[:] = r.randint(0, 1 << 16, pool.data.shape)
    ids = r.permutation(pool.num_pages).astype(np.int32)
    src, dst = ids[:pairs].copy(), ids[pairs:2 * pairs].copy()
    if pairs > 2:
        src[0] = src[1]                               # one source, two destinations
        src[2] = -1                                   # padding
    if pairs > 10:
        dst[5] = -3
        src[7] = pool.num_pages
        dst[8] = 1 << 30
        dst[9] = src[9]
    dpool = _pool(pkv, pool)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    pkv.kv_copy_pages(dpool, U.to_dev(src), U.to_dev(dst), status)
    torch.cuda.synchronize()
    assert int(status.item()) == spec.copy_pages(pool, src, dst)
    assert np.array_equal(U.bits(dpool.buffer).reshape(pool.data.shape), pool.data)


def test_copies_with_separate_buffers_and_mapped_ids(pkv):
    r = np.random.RandomState(5)
    pages, half = 40, 8 * 16 * 64
    k, v = (torch.from_numpy(r.randint(-32768, 32768, (pages, half + 8)).astype(np.int16)).to(U.dev()) for _ in "kv")
    want = [x.clone() for x in (k, v)]
    ids = torch.from_numpy(r.permutation(pages).astype(np.int32))
    src, dst = ids[:20].contiguous().pin_memory(), ids[20:].contiguous().pin_memory()
    desc = pkv.kv_pool_create(k, v, (half + 8) * 2, pages)
    pkv.kv_copy_pages(desc, src, dst)
    torch.cuda.synchronize()
    for x, w in zip((k, v), want):
        w[dst.long(), :half] = w[src.long(), :half]
        assert torch.equal(x, w)


def test_a_speculative_step_end_to_end(pkv):
    """Two layers: a prompt, a fork, a tree for both branches, its attention, the accepted path committed, the pages
    behind it freed, a defragmented pool, one more decode step - each against the oracle on the host's pool."""
    layers, prompt, tree, r = 2, 70, 20, np.random.RandomState(9)
    alloc = pkv.Allocator(64, layers, 16, 256, 2, free_order=r.permutation(64).astype(np.int32))
    host = oracle.Pool(64)
    dpool = _pool(pkv, host)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())

    def append(seq, layer, t0, t1):
        n = t1 - t0
        k, v = (rng.normal_bf16(rng.stream_key(r.randint(1 << 20), tag), 0, n * 512).reshape(n, 8, 64) for tag in "kv")
        slots = []
        for t in range(t0, t1):
            page, copy = alloc.write_page(seq, layer, t // 16)
            assert copy == -1
            slots.append(page * 16 + t % 16)
        slots = np.array(slots, np.int32)
        oracle.kv_append(host, k, v, slots)
        pkv.kv_append(dpool, U.to_dev(k), U.to_dev(v), U.to_dev(slots), status)

    assert alloc.admit(0, prompt, 64)[0] == alloc.OK
    for layer in range(layers):
        append(0, layer, 0, prompt)
    rc, src, dst = alloc.fork(0, 1, prompt, 64)
    assert rc == alloc.OK and len(src) == layers
    pkv.kv_copy_pages(dpool, U.to_dev(src), U.to_dev(dst), status)
    spec.copy_pages(host, src, dst)

    lens = np.array([prompt + tree] * 2, np.int32)
    starts = np.array([0, tree, 2 * tree], np.int32)
    see = [S.random_tree(tree, np.random.RandomState(s), 3) for s in range(2)]
    mask = spec.mask_words(np.concatenate(see))
    for seq in range(2):
        for layer in range(layers):
            append(seq, layer, prompt, prompt + tree)
    ws = pkv.tree_workspace(2, tree)

    def tables():
        return alloc.block_tables()

    for layer in range(layers):
        bt = tables()
        q = rng.normal_bf16(rng.stream_key(900 + layer, "q"), 0, 2 * tree * 2048).reshape(-1, 32, 64)
        out = torch.empty(2 * tree, 32, 64, dtype=torch.float32, device=U.dev())
        dbt = U.to_dev(bt)
        pkv.paged_tree_attention(dpool, out, U.to_dev(q), U.to_dev(starts), U.to_dev(mask), dbt[0, layer:],
                                 layers * bt.shape[2], U.to_dev(lens), tree, 256, 0.125, ws, status)
        args = (host, q, starts, mask, bt[:, layer], lens, 0.125, tree, 256)
        ref, err, _ = spec.paged_tree_attention(*args)
        size, _, spread = spec.paged_tree_attention(*args, absolute=True)
        S.assert_within(out.double().cpu().numpy(), ref, S.bound(ref, size, spread, 0.125, 90, False), f"layer {layer}")
        assert err == 0

    # accept a root-to-node path of each tree
    paths = [np.flatnonzero(see[0][tree - 1]), np.flatnonzero(see[1][7])]
    width = max(map(len, paths))
    accepted = np.full((2, width), -1, np.int32)
    for s, p in enumerate(paths):
        accepted[s, :len(p)] = p
    counts = np.array([len(p) for p in paths], np.int32)
    new = torch.zeros(2, dtype=torch.int32, device=U.dev())
    bt = tables()
    pkv.tree_commit(dpool, U.to_dev(bt), layers * bt.shape[2], bt.shape[2], layers, U.to_dev(starts), U.to_dev(lens),
                    U.to_dev(accepted), U.to_dev(counts), 256, new, status)
    want, err = spec.tree_commit(host, bt, starts, lens, accepted, counts, 256)
    assert err == 0 and new.cpu().numpy().tolist() == want.tolist()
    free = alloc.state()[0]
    for seq in range(2):
        alloc.truncate(seq, int(want[seq]))
    assert alloc.state()[0] > free
    src, dst = alloc.compact()
    assert len(src)
    pkv.kv_copy_pages(dpool, U.to_dev(src), U.to_dev(dst), status)
    spec.copy_pages(host, src, dst)

    # one more token by the decode step
    for layer in range(layers):
        k, v = (rng.normal_bf16(rng.stream_key(950 + layer, tag), 0, 2 * 512).reshape(2, 8, 64) for tag in "kv")
        slots = []
        for seq in range(2):
            t = int(want[seq])
            page, copy = alloc.write_page(seq, layer, t // 16)
            assert copy == -1
            slots.append(page * 16 + t % 16)
        slots = np.array(slots, np.int32)
        bt = tables()
        q = rng.normal_bf16(rng.stream_key(960 + layer, "q"), 0, 2 * 2048).reshape(2, 32, 64)
        out = torch.empty(2, 32, 64, dtype=torch.float32, device=U.dev())
        dbt = U.to_dev(bt)
        pkv.decode_step(dpool, U.to_dev(k), U.to_dev(v), U.to_dev(slots), out, U.to_dev(q), dbt[0, layer:],
                        layers * bt.shape[2], new + 1, 256, 0.125, pkv.decode_workspace(2), status)
        oracle.kv_append(host, k, v, slots)
        ref, err = oracle.paged_decode_attention(host, q, np.ascontiguousarray(bt[:, layer]), want + 1, 0.125, 256)
        U.assert_close(out.double().cpu().numpy(), ref, "decode after the commit")
    torch.cuda.synchronize()
    assert int(status.item()) == 0


# ---- the ends of the ranges ------------------------------------------------------------------------
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("gain", [1, 256])
def test_infinities_in_the_prefix(pkv, gain, bf16):
    """A key whose score is -infinity has no weight, an infinite V of the prefix is infinite in the output; in the
    fast path and (scores that grow behind the first keys) in rows that are computed again."""
    c = S.TreeCase([300, 90], [20, 9], seed=73)
    c.q[:, :, 7] = np.maximum(c.q[:, :, 7] & 0x7FFF, 0x3C00)  # q_7 > 0 everywhere
    for s in range(2):
        for t in range(70, 270 if s == 0 else 81):
            k = c.pool.data[c.bt[s, t // 16], 0, :, t % 16]
            k[:] = ((rng.bf16_bits_to_f64(k) * gain).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    ref, err, size, spread = c.reference()
    bt = c.bt
    for t in (0, 37):                                         # gone: left out of what the oracle sums
        c.pool.data[bt[0, t // 16], 0, :, t % 16, 7] = 0xFF80
    want = []
    for s in range(2):
        k, v = (np.concatenate([rng.bf16_bits_to_f64(c.pool.data[bt[s, b], i]).transpose(1, 0, 2)
                                for b in range(-(-int(c.lens[s]) // 16))])[:c.lens[s]] for i in (0, 1))
        n, base = c.nodes[s], int(c.lens[s]) - c.nodes[s]
        keep = np.ones(int(c.lens[s]), bool)
        if s == 0:
            keep[[0, 37]] = False
        for j in range(n):
            word = int(np.uint32(c.mask[c.starts[s] + j, 0]))
            see = np.flatnonzero(keep & np.r_[np.ones(base, bool), [(word >> i) & 1 == 1 for i in range(n)]])
            q = rng.bf16_bits_to_f64(c.q[c.starts[s] + j]).reshape(8, 4, 64)
            x = np.einsum("ghd,tgd->ght", q, k[see]) * c.wl.scale
            w = np.exp(x - x.max(-1, keepdims=True))
            want.append(np.einsum("ght,tgd->ghd", w / w.sum(-1, keepdims=True), v[see]).reshape(32, 64))
    want = np.array(want)
    lim = S.bound(want, np.maximum(size, 8.0), spread, c.wl.scale, 300, bf16)
    got, status = Run(pkv, c, bf16).call().result()
    assert status == 0
    S.assert_within(got, want, lim, "keys of score -infinity")
    if gain == 1:                                             # (every weight is far from 0 here)
        for t, bits in ((5, 0x7F80), (200, 0xFF80)):
            c.pool.data[bt[0, t // 16], 1, :, t % 16, t % 64] = bits
        got, status = Run(pkv, c, bf16).call().result()
        first = got[:20]
        assert np.isposinf(first[:, :, 5]).all() and np.isneginf(first[:, :, 200 % 64]).all()
        dims = np.delete(np.arange(64), [5, 200 % 64])
        S.assert_within(first[:, :, dims], want[:20][:, :, dims], lim[:20][:, :, dims], "the other dims")
        S.assert_within(got[20:], want[20:], lim[20:], "the other sequence")


def test_a_row_whose_scores_are_all_minus_infinity_is_zero(pkv):
    c = S.TreeCase([30], [6], seed=74)
    c.q[:, :, 7] = 0x3F80
    for t in range(30):
        c.pool.data[c.bt[0, t // 16], 0, :, t % 16, 7] = 0xFF80
    got, status = Run(pkv, c).call().result()
    assert status == 0 and not got.any()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("contexts,nodes", [([9000], [3]), ([30000, 700], [40, 64]), ([20000, 64], [8, 64])])
def test_long_contexts_split_over_many_parts(pkv, contexts, nodes, bf16):
    # units in tens of parts (merged in groups), and units cut into parts of many blocks
    _check(pkv, S.TreeCase(contexts, nodes, seed=75), bf16)


def test_segments_of_several_runs(pkv):
    # as many units as there are CTAs and more: whole units of 47 blocks, their products added up in runs
    c = S.TreeCase([3000, 2990, 2500, 3000] * 10, [2, 8, 1, 3] * 10, seed=76)
    got = _check(pkv, c)
    ref, _, size, _ = c.reference()
    # weights in two bf16 terms (2^-18), 16 truncating blocks a run (16 * 1.4e-7 = 2^-18.8), 3 runs and the scores in fp32
    # (of exponents below 2^4: 2^-19): below 2^-16 of the size of the values
    assert (np.abs(got - ref) <= size * 2.0 ** -16).all()


@pytest.mark.parametrize("bf16", [False, True])
def test_batches_larger_than_a_block(pkv, bf16):
    # more sequences than the kernel has threads, one in three without nodes, some with two tiles
    r = np.random.RandomState(11)
    nodes = [0 if s % 3 == 1 else int(r.randint(1, 70 if s % 17 == 0 else 6)) for s in range(900)]
    contexts = [n + int(r.randint(0, 60)) for n in nodes]
    _check(pkv, S.TreeCase(contexts, nodes, seed=77), bf16)


def test_pages_past_four_gigabytes(pkv):
    """Tree attention (the fast path and rows computed again), commit and copies on pages whose byte offsets need
    more than 32 bits."""
    pages = 140_000                                            # 4.6 GB
    pool = pkv.KVPool(pages, device=U.dev())
    c = S.TreeCase([90, 40], [20, 7], seed=78)
    used = c.wl.num_pages
    view = pool.buffer.view(pages, -1)
    for gain in (1, 256):
        for s in range(2):
            for t in range(65, int(c.lens[s])):
                k = c.pool.data[c.bt[s, t // 16], 0, :, t % 16]
                k[:] = ((rng.bf16_bits_to_f64(k) * gain).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        view[pages - used:].copy_(U.to_dev(c.pool.data).view(used, -1))
        bt = np.where(c.bt >= 0, c.bt + pages - used, -1).astype(np.int32)
        small = Run(pkv, c).call().result()[0]
        got, status = Run(pkv, c, pool=pool, bt=bt).call().result()
        assert status == 0 and np.array_equal(got, small)
    path, count = np.array([[1, 4, 19], [0, 6, -1]], np.int32), np.array([3, 2], np.int32)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    new = torch.zeros(2, dtype=torch.int32, device=U.dev())
    pkv.tree_commit(pool, U.to_dev(bt), bt.shape[1], 0, 1, U.to_dev(c.starts), U.to_dev(c.lens), U.to_dev(path),
                    U.to_dev(count), c.max_context, new, status)
    spec.tree_commit(c.pool, c.bt[:, None], c.starts, c.lens, path, count, c.max_context)
    high = np.arange(pages - used, pages, dtype=np.int32)
    assert np.array_equal(U.bits(view[pages - used:]).reshape(c.pool.data.shape), c.pool.data)
    pkv.kv_copy_pages(pool, U.to_dev(high), U.to_dev(high - used), status)
    torch.cuda.synchronize()
    assert torch.equal(view[pages - used:].view(torch.int16), view[pages - 2 * used:pages - used].view(torch.int16))
    assert int(status.item()) == 0


def test_calls_on_two_streams_at_once(pkv):
    # each with its own workspace and output; the results are those of a call alone, bit for bit
    cases = [S.TreeCase([2000] * 4, [40, 3, 64, 1], seed=79), S.TreeCase([5000, 17], [9, 17], seed=80)]
    runs = [Run(pkv, c) for c in cases]
    want = [r.call().result()[0] for r in runs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for r in runs:
        r.out[:r.c.rows].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for r, s in zip(runs, streams):
            r.call(stream=s)
    for r, w in zip(runs, want):
        got, status = r.result()
        assert status == 0 and np.array_equal(got, w)


def test_two_graphs_of_one_workspace_in_turn(pkv):
    # replayed one after the other on one stream: each leaves the workspace ready for the other
    cases = [S.TreeCase([900, 33], [64, 33], seed=81), S.TreeCase([70] * 5, [2, 9, 1, 0, 70], seed=82)]
    ws = pkv.tree_workspace(8, 70)
    runs = [Run(pkv, c, workspace=ws) for c in cases]
    want = [r.call().result()[0] for r in runs]
    graphs = []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.call()
        graphs.append(g)
        r.out[:r.c.rows].zero_()
    for _ in range(5):
        for g in graphs:
            g.replay()
    for r, w in zip(runs, want):
        got, status = r.result()
        assert status == 0 and np.array_equal(got, w)


def test_binding_refuses_tables_and_workspaces_of_the_wrong_kind(pkv):
    c = S.TreeCase([50], [5], seed=83)
    r = Run(pkv, c)
    for name, bad in (("bt", r.bt.long()), ("bt", r.bt.cpu()), ("ws", r.ws.cpu())):
        good = getattr(r, name)
        setattr(r, name, bad)
        with pytest.raises(ValueError):
            r.call()
        setattr(r, name, good)
    with pytest.raises(ValueError):
        pkv.tree_commit(r.pool, r.bt.long(), r.bt.shape[1], 0, 1, r.starts, r.lens, r.mask[:, :1], r.lens, 64)
    with pytest.raises(ValueError):                            # host memory that is not pinned
        pkv.kv_copy_pages(r.pool, torch.zeros(1, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    with pytest.raises(pkv.PkvError):
        c.max_context = 0x7FFFFFFF
        r.call()
    assert r.status.item() == 0


def test_claimed_units_are_bit_exact_call_after_call(pkv):
    # many short units: the CTAs claim them in whatever order they get free; the workspace serves other calls between
    r = np.random.RandomState(12)
    nodes = [int(r.randint(1, 64)) for _ in range(72)]
    contexts = [n + int(r.randint(0, 1600)) for n in nodes]
    c = S.TreeCase(contexts, nodes, seed=84)
    assert sum(8 * -(-n // 32) for n in nodes) >= 2 * 304
    ws = pkv.tree_workspace(72, 64)
    run, other = Run(pkv, c, workspace=ws), Run(pkv, S.TreeCase([700, 30], [5, 30], seed=85), workspace=ws)
    first, alone = run.call().result()[0], other.call().result()[0]
    ref, err, size, spread = c.reference()
    S.assert_within(first, ref, S.bound(ref, size, spread, c.wl.scale, max(contexts), False), "claimed units")
    for _ in range(6):
        run.out[:c.rows].zero_()
        got, status = run.call().result()
        assert status == err == 0 and np.array_equal(got, first)
        assert np.array_equal(other.call().result()[0], alone)


@pytest.mark.parametrize("bf16", [False, True])
def test_one_long_sequence_among_many_short_ones(pkv, bf16):
    # units enough to be claimed whole, but one that is longer than a CTA's share: cut
    r = np.random.RandomState(13)
    contexts = [20000] + [int(r.randint(8, 200)) for _ in range(90)]
    _check(pkv, S.TreeCase(contexts, [8] + [int(r.randint(1, 8)) for _ in range(90)], seed=86), bf16)


def test_overlapped_calls_that_claim_units(pkv):
    # the next call starts while the last CTAs of the one before are at work on the same counters
    c = S.TreeCase([130 + s % 90 for s in range(80)], [1 + s % 9 for s in range(80)], seed=87)
    r = Run(pkv, c)
    want = r.call().result()[0]
    for _ in range(10):
        r.call(overlap_previous=True)
    got, status = r.result()
    assert status == 0 and np.array_equal(got, want)


# ---- calls the interface allows ---------------------------------------------------------------------
@pytest.mark.parametrize("seqs", [3, 80])
def test_bounds_far_above_what_is_there(pkv, seqs):
    # max_query and max_context are bounds: results do not depend on them
    nodes, contexts = [1 + s % 7 for s in range(seqs)], [20 + 13 * (s % 11) for s in range(seqs)]
    c = S.TreeCase(contexts, nodes, seed=88, words=32)
    got = _check(pkv, c)
    c.max_query, c.max_context = 1000, c.max_context * 1000
    assert np.array_equal(Run(pkv, c).call().result()[0], got)


def test_a_batch_without_nodes_writes_nothing(pkv):
    c = S.TreeCase([30, 0, 17], [0, 0, 0], seed=89)
    r = Run(pkv, c)
    r.call()
    torch.cuda.synchronize()
    assert torch.isnan(r.out).all() and int(r.status.item()) == 0
    r.c.max_query = 0
    r.call()


def test_faults_without_a_status_word(pkv):
    c = S.TreeCase([10, 200, 70], [11, 20, 9], seed=90, num_pages=40)
    c.bt[1, 3] = -1
    want, _, size, spread = c.reference()
    r = Run(pkv, c)
    r.status = None
    r.call()
    torch.cuda.synchronize()
    S.assert_within(r.out[:c.rows].double().cpu().numpy(), want, S.bound(want, size, spread, c.wl.scale, 200, False),
                    "without a status word")


def test_a_query_that_is_not_finite_stays_in_its_row(pkv):
    c = S.TreeCase([300, 90], [20, 9], seed=91)
    good = _check(pkv, c)
    c.q[3, 5, 7], c.q[22, 0, 1] = 0x7FC0, 0x7F80
    got, status = Run(pkv, c).call().result()
    assert status == 0 and np.isnan(got[3, 5]).all() and not np.isfinite(got[22, 0]).any()
    keep = np.ones(got.shape[:2], bool)
    keep[3, 5] = keep[22, 0] = False
    assert np.array_equal(got[keep], good[keep])


def test_commit_of_nothing_and_of_everything(pkv):
    pool, table, starts, lens, path, count = _commit_case(5, 3, 92, nodes_hi=30, width=30)
    count[:] = 0
    assert _commit(pkv, (pool, table, starts, lens, path, count)) == 0          # only the lengths change
    n = np.diff(starts)
    for s in range(5):
        path[s, :n[s]] = np.arange(n[s])
    assert _commit(pkv, (pool, table, starts, lens, path, n.astype(np.int32))) == 0  # every row stays
    assert _commit(pkv, (pool, table, starts, lens, np.zeros((5, 0), np.int32), count)) == 0
