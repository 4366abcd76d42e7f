"""Helpers of the speculative-decoding tests: random trees, a workload of ragged trees, error bounds."""
from __future__ import annotations

import numpy as np

import oracle
from oracle import speculative as spec
from workloads import configs, rng


def random_tree(n: int, r: np.random.RandomState, window: int = 0) -> np.ndarray:
    """Boolean [n, n]: the ancestors of each node and itself; ``window``: parents at most that far back (0: anywhere)."""
    see = np.zeros((n, n), bool)
    for k in range(n):
        if k:
            lo = max(0, k - window) if window else 0
            see[k] = see[r.randint(lo, k)]
        see[k, k] = True
    return see


class TreeCase:
    """A pool with every sequence's tokens (the nodes last), queries, masks; host side only."""

    def __init__(self, contexts, nodes, seed=1, num_pages=None, words=None, visible=None, max_blocks=None):
        blocks = max(8, max((c + 15) // 16 for c in contexts)) if max_blocks is None else max_blocks
        self.wl = configs.custom(seed, contexts, num_pages=num_pages, max_blocks=blocks, name="tree")
        self.max_context = blocks * 16
        self.nodes = list(nodes)
        self.starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.rows = int(self.starts[-1])
        self.max_query = max(max(nodes), 1)
        r = np.random.RandomState(seed)
        words = max((self.max_query + 31) // 32, 1) if words is None else words
        self.mask = np.zeros((max(self.rows, 1), words), np.int32)
        for s, n in enumerate(nodes):
            if n:
                see = random_tree(n, r, window=(0, 1, 3)[s % 3]) if visible is None else visible(s, n)
                m = spec.mask_words(see)
                self.mask[self.starts[s]:self.starts[s] + n, :m.shape[1]] = m
        self.q = rng.normal_bf16(rng.stream_key(seed, "tree-q"), 0, max(self.rows, 1) * 32 * 64).reshape(-1, 32, 64)
        self.bt = np.ascontiguousarray(self.wl.block_tables[:, 0, :])
        self.lens = self.wl.context_lens
        self.pool = oracle.Pool(self.wl.num_pages)      # untouched slots hold a NaN pattern
        for s in range(self.wl.num_seqs):
            if self.wl.has_pages(s):
                k, v = self.wl.kv_tokens(s, 0)
                oracle.kv_append(self.pool, k, v, self.wl.slot_mapping(s, 0, 0, int(self.lens[s])))

    def reference(self, scale=None, **over):
        scale = self.wl.scale if scale is None else scale
        args = dict(pool=self.pool, q=self.q, query_start=self.starts, mask=self.mask, block_tables=self.bt,
                    context_lens=self.lens, scale=scale, max_query=self.max_query, max_context=self.max_context)
        args.update(over)
        out, err, _ = spec.paged_tree_attention(**args)
        size, _, spread = spec.paged_tree_attention(absolute=True, **args)
        return out, err, size, spread


def bound(ref, size, spread, scale, keys, bf16):
    """Elementwise bound of |gpu - ref|, with size = sum_t w_t |V_t| and u = 2^-23 (an addition that may truncate).

    Score: products of bf16 are exact in fp32; 64 additions err by at most 64 u sum|q_d K_d| (<= spread),
    two multiplications and the subtraction of the reference by 4 u of the exponent (<= |scale| spread, twice
    for the difference): e = (64 + 8) u |scale| spread.  A weight and the sum it is divided by carry e each,
    the exponential 2^-22 and the split into two bf16 terms 2^-16 each.  Sums over `keys` keys: one addition
    per 16 keys and term in the product with V, one per key at most in the row sum, 64 in merges, each u of
    what has been added so far (<= size).  The last division u.  A bf16 output rounds by half a step (2^-8),
    and its single-term weights by 2^-8 each above and below the fraction."""
    u = 2.0 ** -23
    rel = 2 * ((64 + 8) * u * abs(scale) * spread + 2.0 ** -22 + 2.0 ** -16) + (3 * keys / 16 + keys + 128) * u + u
    if bf16:
        rel += 2 * 2.0 ** -8
        return size * rel + np.abs(ref) * 2.0 ** -8 + 1e-30
    return size * rel + 1e-30


def assert_within(got, ref, lim, what=""):
    got = np.asarray(got, np.float64)
    err = np.abs(got - ref)
    bad = ~(err <= lim)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first {i} got {got[i]} "
                             f"ref {ref[i]} bound {lim[i]}")
