"""FP64 oracle of the speculative-decoding operators (plain numpy; test infrastructure only).

Shares nothing with the CUDA path.  Tree attention takes the two-pass form of the softmax (maximum
first, then weights) over an explicit list of the positions each node may see; the commit and the page
copies move rows of the host pool one by one, reading everything before writing anything.
"""
from __future__ import annotations

import numpy as np

ERR_CONTEXT = 2
ERR_PAGE = 4
ERR_PATH = 16


def _values(bits: np.ndarray) -> np.ndarray:
    """bf16 bit patterns -> float64 values."""
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def mask_words(visible: np.ndarray) -> np.ndarray:
    """A boolean [rows, nodes] matrix as int32 words, bit j of a row in word j // 32."""
    rows, nodes = visible.shape
    words = max((nodes + 31) // 32, 1)
    out = np.zeros((rows, words), np.uint32)
    for j in range(nodes):
        out[:, j // 32] |= visible[:, j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


def paged_tree_attention(pool, q, query_start, mask, block_tables, context_lens, scale, max_query, max_context,
                         absolute=False):
    """(out float64 [rows, heads, dim], error bits, largest sum |q_d K_d| of any score).

    ``mask``: int32 words [rows, words].  A page id outside the pool is left out.  ``absolute``: take
    |V| for V, for error bounds (the weights stay what they are)."""
    rows, heads, dim = q.shape
    group = heads // pool.num_kv_heads
    words = np.ascontiguousarray(mask).view(np.uint32)
    out = np.zeros((rows, heads, dim))
    err, spread = 0, 0.0
    P = pool.page_tokens
    for s in range(len(context_lens)):
        q0, n, ctx = int(query_start[s]), int(query_start[s + 1] - query_start[s]), int(context_lens[s])
        if n == 0:
            continue
        if n < 0 or n > max_query or ctx < 0 or ctx > max_context or n > ctx or q0 < 0 or q0 + n > rows:
            err |= ERR_CONTEXT
            continue
        base = ctx - n
        here = np.ones(ctx, bool)
        pages = np.asarray(block_tables[s][:(ctx + P - 1) // P]).copy()
        for b, p in enumerate(pages):
            if p < 0 or p >= pool.num_pages:
                err |= ERR_PAGE
                here[b * P:(b + 1) * P] = False
                pages[b] = 0
        kv = pool.data[pages]                                       # [block, K|V, head, row, dim]
        K, V = (_values(kv[:, i].transpose(1, 0, 2, 3).reshape(pool.num_kv_heads, -1, dim)[:, :ctx]) for i in (0, 1))
        if absolute:
            V = np.abs(V)
        for j in range(n):
            node = (words[q0 + j, np.arange(n) // 32] >> (np.arange(n) % 32).astype(np.uint32)) & 1
            see = np.flatnonzero(here & np.concatenate([np.ones(base, bool), node.astype(bool)]))
            if see.size == 0:
                continue
            for g in range(pool.num_kv_heads):
                qg = _values(q[q0 + j, g * group:(g + 1) * group])
                x = qg @ K[g, see].T * scale
                w = np.exp(x - x.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                out[q0 + j, g * group:(g + 1) * group] = w @ V[g, see]
                if absolute:
                    spread = max(spread, float((np.abs(qg) @ np.abs(K[g, see]).T).max()))
    return out, err, spread


def tree_commit(pool, block_tables, query_start, context_lens, accepted, accept_counts, max_context):
    """Moves rows of ``pool`` in place; ``block_tables`` is [seqs, layers, blocks].  (new lengths, error bits)"""
    seqs, layers, _ = block_tables.shape
    new, err = np.array(context_lens, np.int32).copy(), 0
    P = pool.page_tokens
    for s in range(seqs):
        n, ctx, c = int(query_start[s + 1] - query_start[s]), int(context_lens[s]), int(accept_counts[s])
        if n < 0 or ctx < 0 or ctx > max_context or n > ctx:
            err |= ERR_CONTEXT
            continue
        path = [int(p) for p in accepted[s][:max(c, 0)]]
        if c < 0 or c > n or c > accepted.shape[1] or any(not 0 <= p < n for p in path) or \
                any(b <= a for a, b in zip(path, path[1:])):
            err |= ERR_PATH
            continue
        base = ctx - n
        new[s] = base + c
        for layer in range(layers):
            table = block_tables[s, layer]
            held = []
            for k, p in enumerate(path):
                if p == k:
                    continue
                a, b = table[(base + p) // P], table[(base + k) // P]
                if not (0 <= a < pool.num_pages and 0 <= b < pool.num_pages):
                    err |= ERR_PAGE
                    continue
                held.append((b, (base + k) % P, pool.data[a, :, :, (base + p) % P].copy()))
            for page, row, data in held:
                pool.data[page, :, :, row] = data
    return new, err


def copy_pages(pool, src, dst):
    """Copies whole pages of ``pool`` in place (distinct destinations, none of them a source)."""
    err = 0
    for a, b in zip(src, dst):
        if a < 0 or b < 0:
            continue
        if a >= pool.num_pages or b >= pool.num_pages:
            err |= ERR_PAGE
            continue
        pool.data[b] = pool.data[a]
    return err
