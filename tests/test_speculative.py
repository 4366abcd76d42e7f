"""Speculative decoding on the CPU: the FP64 oracle's pins, the allocator's forks, copy on write, cuts and
defragmentation, and the host checks of the operators (no call here reaches a kernel launch)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import speculative as spec
from tests import spec_util as S
from workloads import configs, rng


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_180_gb300 import build
    build.build()
    import paged_kv_cache_180_gb300 as p
    return p


# ---- the oracle ----------------------------------------------------------------------------------
def test_oracle_tree_is_torch_attention_under_the_mask():
    c = S.TreeCase([37, 9, 64], [5, 9, 1], seed=11)
    ref, err, _, _ = c.reference()
    assert err == 0
    for s in range(3):
        k, v = (torch.from_numpy(rng.bf16_bits_to_f64(x)) for x in c.wl.kv_tokens(s))
        a, b = c.starts[s], c.starts[s + 1]
        n, ctx = b - a, int(c.lens[s])
        q = torch.from_numpy(rng.bf16_bits_to_f64(c.q[a:b]))
        see = np.ones((n, ctx), bool)
        bits = c.mask[a:b].view(np.uint32)
        for j in range(n):
            see[:, ctx - n + j] = (bits[:, j // 32] >> np.uint32(j % 32)) & 1
        x = torch.einsum("nhd,thd->hnt", q, k.repeat_interleave(4, 1)) / math.sqrt(64)
        x = x.masked_fill(~torch.from_numpy(see), -math.inf)
        want = torch.einsum("hnt,thd->nhd", torch.softmax(x, -1), v.repeat_interleave(4, 1)).numpy()
        assert np.abs(ref[a:b] - want).max() < 1e-12


def test_oracle_chain_tree_is_causal_prefill():
    # a chain (every node's parent is the one before) is a causal chunk
    chain = lambda s, n: np.tril(np.ones((n, n), bool))  # noqa: E731
    c = S.TreeCase([50, 20, 7], [13, 20, 3], seed=12, visible=chain)
    ref, err, _, _ = c.reference()
    want, werr = oracle.paged_prefill_attention(c.pool, c.q, c.starts, c.bt, c.lens, c.wl.scale, c.max_context)
    assert err == werr == 0 and np.abs(ref - want).max() < 1e-12


def test_oracle_empty_rows_ignored_bits_and_faults():
    # no prefix and no bit: zeros; bits at or past n are ignored; lengths that do not fit
    c = S.TreeCase([4, 40, 3, 9], [4, 2, 5, 2], seed=13, num_pages=8)
    c.mask[0] = 0
    c.mask[c.starts[1]] |= np.int32(-4)                    # bits 2 .. 31 of a tree of two nodes
    ref, err, _, _ = c.reference()
    assert err == spec.ERR_CONTEXT                         # sequence 2: five nodes, three tokens
    assert not ref[0].any() and ref[1].any() and not ref[c.starts[2]:c.starts[3]].any()
    plain = c.mask.copy()
    plain[c.starts[1]] &= 3
    assert np.array_equal(c.reference(mask=plain)[0], ref)
    bt = c.bt.copy()
    bt[3, 0] = 99
    ref2, err2, _, _ = c.reference(block_tables=bt)
    assert err2 & spec.ERR_PAGE and not ref2[c.starts[3]:].any()    # its only page


def test_oracle_commit_and_copies():
    pool = oracle.Pool(6)
    pool.data[:] = np.arange(pool.data.size, dtype=np.uint32).reshape(pool.data.shape).astype(np.uint16)
    before = pool.data.copy()
    bt = np.array([[[4, 1], [0, 5]], [[2, -1], [3, -1]]], np.int32)
    new, err = spec.tree_commit(pool, bt, [0, 6, 8], [20, 3], np.array([[0, 2, 5], [1, 0, 0]]), [3, 1], 32)
    assert err == 0 and new.tolist() == [17, 2]
    for layer in range(2):      # base 14: rows 14, 16, 19 -> 14, 15, 16
        a, b = bt[0, layer]
        assert np.array_equal(pool.data[a, :, :, 14], before[a, :, :, 14])
        assert np.array_equal(pool.data[a, :, :, 15], before[b, :, :, 0])
        assert np.array_equal(pool.data[b, :, :, 0], before[b, :, :, 3])
        assert np.array_equal(pool.data[b, :, :, 1:], before[b, :, :, 1:])
        p = bt[1, layer, 0]     # base 1: row 2 -> 1
        assert np.array_equal(pool.data[p, :, :, 1], before[p, :, :, 2])
    for path, count in (([1, 1, 0], 2), ([0, 6, 0], 2), ([0, 1, 2], 4), ([0, -1, 2], 2), ([0, 1, 2], -1)):
        got = oracle.Pool(6)
        got.data[:] = before
        new, err = spec.tree_commit(got, bt, [0, 6, 8], [20, 3], np.array([path, [0, 0, 0]]), [count, 0], 32)
        assert err == spec.ERR_PATH and new.tolist() == [20, 1] and np.array_equal(got.data, before)
    got = oracle.Pool(6)
    got.data[:] = before
    assert spec.copy_pages(got, [0, -1, 3, 6], [1, 2, 5, 4]) == spec.ERR_PAGE
    assert np.array_equal(got.data[1], before[0]) and np.array_equal(got.data[5], before[3])
    assert np.array_equal(got.data[[0, 2, 3, 4]], before[[0, 2, 3, 4]])


# ---- allocator -----------------------------------------------------------------------------------
def _invariants(a):
    """Every page is free or named as often as its count says; returns the table."""
    bt = a.block_tables()
    named = np.bincount(bt[bt >= 0], minlength=a.num_pages)
    assert named.tolist() == [a.page_refs(p) for p in range(a.num_pages)]
    free, credits = a.state()
    assert free == int((named == 0).sum())
    assert int((bt >= 0).sum()) <= credits
    return bt


def _fill(a, seq, tokens):
    for layer in range(a.num_layers):
        for b in range(-(-tokens // 16)):
            a.page(seq, layer, b)


def test_fork_shares_full_pages_and_copies_the_last_one(pkv):
    a = pkv.Allocator(64, 2, 16, 128, 4)
    assert a.admit(0, 40, 8)[0] == a.OK
    _fill(a, 0, 40)
    rc, src, dst = a.fork(0, 1, 40, 8)
    assert rc == a.OK
    bt = _invariants(a)
    for layer in range(2):
        assert bt[1, layer, :2].tolist() == bt[0, layer, :2].tolist()
        assert src[layer] == bt[0, layer, 2] and dst[layer] == bt[1, layer, 2] != src[layer]
    # on a page boundary nothing is copied
    rc, src, dst = a.fork(0, 2, 32, 1)
    assert rc == a.OK and len(src) == 0 and a.page_refs(int(bt[0, 0, 0])) == 3
    # pages go back when the last holder lets go
    free = a.state()[0]
    a.free_seq(0)
    assert a.state()[0] == free + 2                          # only its two own last pages
    a.free_seq(2)
    assert a.state()[0] == free + 2
    a.free_seq(1)
    assert a.state() == (64, 0)
    _invariants(a)


def test_fork_refusals_change_nothing(pkv):
    a = pkv.Allocator(16, 1, 16, 64, 4)
    assert a.admit(0, 40, 8)[0] == a.OK
    _fill(a, 0, 40)
    before, state = a.block_tables(), a.state()
    for args, code in [((0, 0, 40, 1), -2), ((0, 4, 40, 1), -2), ((-1, 1, 40, 1), -2), ((0, 1, 0, 1), -2),
                       ((0, 1, 65, 1), -2), ((0, 1, 40, 0), -2), ((2, 1, 40, 1), -11)]:
        with pytest.raises(pkv.PkvError) as e:
            a.fork(*args)
        assert e.value.code == code, args
    lib, n = pkv.binding._lib, ctypes.c_int32(7)
    assert lib.pkv_alloc_fork(a._h, 0, 1, 40, 1, None, None, 0, ctypes.byref(n)) == -2 and n.value == 1
    assert lib.pkv_alloc_fork(a._h, 0, 1, 40, 1, None, None, 1, ctypes.byref(n)) == -1
    assert lib.pkv_alloc_fork(a._h, 0, 1, 40, 1, None, None, 1, None) == -1
    assert lib.pkv_alloc_fork(None, 0, 1, 40, 1, None, None, 1, ctypes.byref(n)) == -1
    assert np.array_equal(a.block_tables(), before) and a.state() == state
    for seq in (1, 2, 3):
        assert a.admit(seq, 50, 15)[0] == a.OK              # 4 credits each: 15 of 16 held
    a.free_seq(3)
    assert a.fork(0, 3, 40, 40)[0] == a.OK                  # clamped to 64 tokens: 4 credits
    a.free_seq(3)
    assert a.admit(3, 64, 1)[0] == a.OK
    with pytest.raises(pkv.PkvError) as e:
        a.fork(0, 3, 40, 1)                                 # admitted already
    assert e.value.code == -11
    b = pkv.Allocator(5, 1, 16, 64, 2)
    assert b.admit(0, 40, 1)[0] == b.OK
    _fill(b, 0, 40)
    rc, src, dst = b.fork(0, 1, 40, 1)
    assert rc == b.NO_CREDIT and len(src) == 0 and b.state() == (2, 3)


def test_write_page_copies_a_shared_page_once(pkv):
    a = pkv.Allocator(16, 1, 16, 64, 3)
    assert a.admit(0, 40, 1)[0] == a.OK
    _fill(a, 0, 40)
    assert a.fork(0, 1, 32, 9)[0] == a.OK                    # room for a third block
    shared = int(a.block_tables()[0, 0, 1])
    page, copy = a.write_page(1, 0, 1)                       # rewriting token 20 of the fork
    assert copy == shared and page != shared and a.page_refs(shared) == 1 and a.page_refs(page) == 1
    assert a.write_page(1, 0, 1) == (page, -1)               # its own now
    assert a.write_page(0, 0, 1) == (shared, -1)
    fresh, copy = a.write_page(1, 0, 2)                      # a block not assigned yet
    assert copy == -1 and a.page_refs(fresh) == 1
    _invariants(a)
    for args, code in [((0, 1, 0), -2), ((0, 0, 4), -2), ((3, 0, 0), -2), ((2, 0, 0), -11)]:
        with pytest.raises(pkv.PkvError) as e:
            a.write_page(*args)
        assert e.value.code == code


def test_truncate_gives_back_the_pages_behind(pkv):
    a = pkv.Allocator(32, 2, 16, 128, 2)
    assert a.admit(0, 100, 20)[0] == a.OK
    _fill(a, 0, 100)
    credits = a.state()[1]
    a.truncate(0, 65)
    bt = _invariants(a)
    assert (bt[0, :, :5] >= 0).all() and (bt[0, :, 5:] == -1).all() and a.state() == (22, credits)
    a.truncate(0, 64)
    assert (a.block_tables()[0, :, 4:] == -1).all()
    a.truncate(0, 128)
    assert a.state() == (24, credits)
    a.truncate(0, 0)
    assert a.state() == (32, credits)
    _fill(a, 0, 128)                                          # still within its credits
    for args, code in [((0, -1), -2), ((0, 129), -2), ((1, 5), -11), ((2, 5), -2)]:
        with pytest.raises(pkv.PkvError) as e:
            a.truncate(*args)
        assert e.value.code == code


def test_compact_moves_used_pages_to_the_front(pkv):
    order = np.random.RandomState(3).permutation(24).astype(np.int32)
    a = pkv.Allocator(24, 1, 16, 128, 4, free_order=order)
    for seq, tokens in ((0, 60), (1, 90), (2, 30)):
        assert a.admit(seq, tokens, 1)[0] == a.OK
        _fill(a, seq, tokens)
    assert a.fork(2, 3, 16, 1)[0] == a.OK
    a.free_seq(1)
    before = a.block_tables()
    refs = {p: a.page_refs(p) for p in range(24)}
    used = sum(r > 0 for r in refs.values())
    lib, n = pkv.binding._lib, ctypes.c_int32(0)
    assert lib.pkv_alloc_compact(a._h, None, None, 0, ctypes.byref(n)) == -2 and n.value > 0
    assert lib.pkv_alloc_compact(a._h, None, None, n.value, ctypes.byref(n)) == -1
    assert np.array_equal(a.block_tables(), before)
    src, dst = a.compact()
    after = _invariants(a)
    assert len(src) == n.value and not set(src) & set(dst) and len(set(src)) == len(set(dst)) == len(src)
    assert set(after[after >= 0]) == set(range(used))
    move = dict(zip(src.tolist(), dst.tolist()))
    assert np.array_equal(after, np.vectorize(lambda p: move.get(int(p), int(p)))(before))
    assert all(refs[p] == a.page_refs(move.get(p, p)) for p in refs if refs[p])
    assert a.page(2, 0, 1) < used and a.admit(1, 1, 1)[0] == a.OK and a.page(1, 0, 0) == used
    assert len(a.compact()[0]) == 0
    assert a.page_refs(24) == a.page_refs(-1) == -1


def test_random_forks_cuts_and_frees_keep_the_books(pkv):
    """Random calls against a model of pages by content: a page's content is the (sequence history, block) that
    wrote it, and after every call each sequence still reads what it wrote."""
    r = np.random.RandomState(5)
    a = pkv.Allocator(60, 2, 16, 96, 6, free_order=r.permutation(60).astype(np.int32))
    pages = {}                       # page -> content of its 16 tokens (list), per physical page
    seqs = {}                        # seq -> list of token ids
    fresh = iter(range(1 << 30))

    def write(seq, pos, token):
        for layer in range(2):
            page, copy = a.write_page(seq, layer, pos // 16)
            if copy >= 0:
                pages[page] = list(pages[copy])
            pages.setdefault(page, [None] * 16)[pos % 16] = (token, layer)

    for _ in range(600):
        what = r.randint(6)
        live = sorted(seqs)
        free = [s for s in range(6) if s not in seqs]
        if what == 0 and free:
            if a.admit(free[0], int(r.randint(1, 60)), 96)[0] == a.OK:
                seqs[free[0]] = []
        elif what in (1, 2) and live:
            s = live[r.randint(len(live))]
            for _ in range(r.randint(1, 20)):
                if len(seqs[s]) < 96:
                    token = next(fresh)
                    write(s, len(seqs[s]), token)
                    seqs[s].append(token)
        elif what == 3 and live and free:
            s = live[r.randint(len(live))]
            if seqs[s]:
                tokens = r.randint(1, len(seqs[s]) + 1)
                rc, src, dst = a.fork(s, free[0], int(tokens), 96)
                if rc == a.OK:
                    for x, y in zip(src.tolist(), dst.tolist()):
                        pages[y] = list(pages[x])
                    seqs[free[0]] = seqs[s][:tokens]
        elif what == 4 and live:
            s = live[r.randint(len(live))]
            keep = r.randint(0, len(seqs[s]) + 1)
            a.truncate(s, int(keep))
            seqs[s] = seqs[s][:keep]
        elif what == 5 and live:
            if r.rand() < 0.4:
                s = live[r.randint(len(live))]
                a.free_seq(s)
                del seqs[s]
            else:
                src, dst = a.compact()
                held = [list(pages[x]) for x in src.tolist()]
                for y, data in zip(dst.tolist(), held):
                    pages[y] = data
        bt = _invariants(a)
        for s, tokens in seqs.items():
            for layer in range(2):
                for t, token in enumerate(tokens):
                    assert pages[int(bt[s, layer, t // 16])][t % 16] == (token, layer)


# ---- host checks ---------------------------------------------------------------------------------
def test_tree_attention_refusals(pkv):
    b = pkv.binding
    lib, P, base = b._lib, ctypes.c_void_p, 1 << 20
    d = b.kv_pool_create(base, base + 16384, 0, 8)
    need = b.tree_workspace_bytes(4, 16)

    def call(**kw):
        g = lambda name, default=base: P(kw.get(name, default))  # noqa: E731
        return lib.pkv_paged_tree_attention(
            ctypes.byref(kw.get("pool", d)), g("out"), g("q"), kw.get("hq", 32), kw.get("rows", 64), g("qs"), g("mask"),
            kw.get("ms", 1), g("bt"), kw.get("bs", 128), g("lens"), kw.get("n", 4), kw.get("mq", 16), kw.get("mc", 2048),
            kw.get("scale", 0.125), g("ws"), kw.get("wsb", need), None, kw.get("flags", 0), None)

    for kw, code in [(dict(flags=4), -2), (dict(hq=16), -3), (dict(n=-1), -2), (dict(mq=-1), -2), (dict(mc=-1), -2),
                     (dict(rows=-1), -2), (dict(bs=-1), -2), (dict(ms=-1), -2), (dict(ms=0), -2), (dict(mq=33), -2),
                     (dict(out=0), -1), (dict(q=0), -1), (dict(qs=0), -1), (dict(mask=0), -1), (dict(bt=0), -1),
                     (dict(lens=0), -1), (dict(ws=0), -1), (dict(scale=float("nan")), -5),
                     (dict(scale=float("inf")), -5), (dict(out=base + 8), -4), (dict(q=base + 2), -4),
                     (dict(ws=base + 8), -4), (dict(qs=base + 2), -4), (dict(mask=base + 1), -4),
                     (dict(bt=base + 2), -4), (dict(lens=base + 3), -4), (dict(wsb=need - 1), -6),
                     (dict(n=5), -6), (dict(pool=b.PkvPool()), -1)]:
        if "n" in kw and kw["n"] == 5 and b.tree_workspace_bytes(5, 16) == need:
            continue                       # the same rounded size
        assert call(**kw) == code, kw
    for kw in (dict(n=0), dict(mq=0, ms=0), dict(rows=0)):
        assert call(**kw) == 0             # nothing to do
    assert b.tree_workspace_bytes(-1, 16) == b.tree_workspace_bytes(4, -1) == 0
    assert b.tree_workspace_bytes(4, 16, 16) == b.tree_workspace_bytes(4, 16, 32, 128) == 0
    assert b.tree_workspace_bytes(4000, 256) > need


def test_tree_attention_refuses_contexts_whose_last_block_passes_32_bits(pkv):
    b = pkv.binding
    d = b.kv_pool_create(1 << 20, (1 << 20) + 16384, 0, 8)
    p, need = ctypes.c_void_p(1 << 20), b.tree_workspace_bytes(1, 1)
    call = lambda mc, wsb: b._lib.pkv_paged_tree_attention(  # noqa: E731
        ctypes.byref(d), p, p, 32, 1, p, p, 1, p, 1 << 27, p, 1, 1, mc, 0.125, p, wsb, None, 0, None)
    assert call(2 ** 31 - 1, need) == call(2 ** 31 - 63, need) == -2
    assert call(2 ** 31 - 64, need - 1) == -6          # the largest one passes on to the next check


def test_commit_and_copy_refusals(pkv):
    b = pkv.binding
    lib, P, base = b._lib, ctypes.c_void_p, 1 << 20
    d = b.kv_pool_create(base, base + 16384, 0, 8)
    far = base + (1 << 16)

    def commit(**kw):
        g = lambda name, default=base: P(kw.get(name, default))  # noqa: E731
        return lib.pkv_tree_commit(ctypes.byref(kw.get("pool", d)), g("bt"), kw.get("bs", 128), kw.get("ls", 0),
                                   kw.get("layers", 1), g("qs"), g("lens"), g("path"), kw.get("ps", 8), g("counts"),
                                   kw.get("n", 4), kw.get("ma", 8), kw.get("mc", 2048), g("new", far), None, None)

    for kw, code in [(dict(n=-1), -2), (dict(layers=0), -2), (dict(ma=-1), -2), (dict(mc=-1), -2), (dict(bs=-1), -2),
                     (dict(ls=-1), -2), (dict(ps=7), -2), (dict(n=1 << 20, layers=1 << 12), -2), (dict(bt=0), -1),
                     (dict(qs=0), -1), (dict(lens=0), -1), (dict(path=0), -1), (dict(counts=0), -1),
                     (dict(bt=base + 2), -4), (dict(new=far + 1), -4), (dict(new=base), -2), (dict(new=base + 12), -2),
                     (dict(new=base - 12), -2), (dict(path=far, new=far + 4 * (3 * 8 + 7)), -2),
                     (dict(pool=b.PkvPool()), -1)]:
        assert commit(**kw) == code, kw
    assert commit(n=0) == 0
    copy = lambda n=4, src=base, dst=base, pool=d: lib.pkv_kv_copy_pages(  # noqa: E731
        ctypes.byref(pool), P(src), P(dst), n, None, None)
    assert copy(n=0) == 0 and copy(n=-1) == -2 and copy(n=1 << 30) == -2
    assert copy(src=0) == -1 and copy(dst=0) == -1 and copy(src=base + 2) == -4
    assert copy(pool=b.PkvPool()) == -1
