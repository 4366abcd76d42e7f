"""Helpers of the tests of window attention, weight sums and eviction: a ragged pool, error bounds."""
from __future__ import annotations

import numpy as np

import oracle
from oracle import bounded
from workloads import configs, rng


class Cache:
    """A pool with every sequence's tokens, its tables and queries; host side only.  Untouched slots hold NaN patterns.
    ``nodes``: query tokens of every sequence (1 each without), the last cached ones."""

    def __init__(self, contexts, nodes=None, seed=1, layers=1, max_blocks=None):
        blocks = max(4, max((c + 15) // 16 for c in contexts)) if max_blocks is None else max_blocks
        self.wl = configs.custom(seed, contexts, max_blocks=blocks, name="bounded")
        self.max_context = blocks * 16
        self.nodes = [1] * len(contexts) if nodes is None else list(nodes)
        self.starts = np.concatenate([[0], np.cumsum(self.nodes)]).astype(np.int32)
        self.rows = int(self.starts[-1])
        self.max_query = max(max(self.nodes), 1)
        self.lens = np.array(contexts, np.int32)
        # twice normal: a softmax as peaked as trained heads have it
        q = rng.normal_bf16(rng.stream_key(seed, "bounded-q"), 0, max(self.rows, 1) * 32 * 64).reshape(-1, 32, 64)
        self.q = np.where((q & 0x7f80) != 0, q + 0x80, q).astype(np.uint16)
        self.bt = np.ascontiguousarray(self.wl.block_tables[:, 0, :])
        self.pool = oracle.Pool(self.wl.num_pages)
        self.scale = self.wl.scale
        for s in range(self.wl.num_seqs):
            if self.wl.has_pages(s):
                k, v = self.wl.kv_tokens(s, 0)
                oracle.kv_append(self.pool, k, v, self.wl.slot_mapping(s, 0, 0, int(self.lens[s])))

    def token(self, s, t, kv):
        """The 8 x 64 bf16 bits of token t of sequence s, K (0) or V (1), for writing."""
        return self.pool.data[self.bt[s, t // 16], kv, :, t % 16]

    def hide(self, window, sinks):
        """Tables without the pages that no query of ``nodes`` sees."""
        bt = self.bt.copy()
        for s, ctx in enumerate(self.lens):
            seen = set()
            for p in range(int(ctx) - max(self.nodes[s], 1), int(ctx)):
                if p >= 0:
                    seen |= set((bounded.seen_by(p, window, sinks) // 16).tolist())
            bt[s, [b for b in range(bt.shape[1]) if b not in seen]] = -1
        return bt

    def decode(self, window, sinks, scale=None, bt=None, max_context=None):
        """(reference, error bits, |w| |V| sums, spread, weights)."""
        args = (self.pool, self.q, self.bt if bt is None else bt, self.lens, self.scale if scale is None else scale,
                window, sinks, self.max_context if max_context is None else max_context)
        out, err, _, weights = bounded.window_decode(*args)
        size, _, spread, _ = bounded.window_decode(*args, absolute=True)
        return out, err, size, spread, weights

    def prefill(self, window, sinks, scale=None, bt=None, max_query=None, starts=None, lens=None):
        args = (self.pool, self.q, self.starts if starts is None else starts, self.bt if bt is None else bt,
                self.lens if lens is None else lens, self.scale if scale is None else scale, window, sinks,
                self.max_query if max_query is None else max_query, self.max_context)
        out, err, _, _ = bounded.paged_window_attention(*args)
        size, _, spread, _ = bounded.paged_window_attention(*args, absolute=True)
        return out, err, size, spread


def weight_error(spread, scale, keys):
    """Relative error of a normalised weight in window decode and in the weight sums; u = 2^-23 (an addition of the tensor
    cores may truncate).

    Score: products of bf16 are exact in fp32; 64 additions err by at most 64 u sum |q_d K_d| (<= spread), two
    multiplications and the subtraction of the reference by 4 u of the exponent (<= |scale| spread, twice for the
    difference): (64 + 8) u |scale| spread; the exponential 2^-22.  The sum that divides it carries the same and an
    addition for every four keys of a thread and for every warp and CTA, and 2^-22 in each of two changes of reference."""
    u = 2.0 ** -23
    return 2 * ((64 + 8) * u * abs(scale) * spread + 2.0 ** -22) + (keys / 4 + 64) * u + 2 * 2.0 ** -22


def decode_bound(ref, size, spread, scale, keys, bf16):
    """Elementwise bound of |gpu - ref| of the decode operators, with size = sum_t w_t |V_t|: the weight's error, three bf16
    terms of it (2^-24), a page's products of 16 keys and 3 terms in the tensor core (16 u) and one addition and one
    multiplication a page; merges of 8 warps and 8 CTAs with two factors of 2^-22; a division.  A bf16 output rounds by half a step."""
    u = 2.0 ** -23
    lim = size * (weight_error(spread, scale, keys) + u + 16 * u + 2 * keys / 16 * u + 32 * u + 2 * 2.0 ** -22 + u)
    return lim + (np.abs(ref) * 2.0 ** -8 if bf16 else 0) + 1e-30
