"""FP64 oracle of the operators that bound a cache (plain numpy; test infrastructure only).

Shares nothing with the CUDA path: attention takes the two-pass form of the softmax over an explicit list of the
positions a query sees, eviction sorts a list of (sum, position) pairs and moves rows one by one, reading everything
before writing anything.
"""
from __future__ import annotations

import numpy as np

ERR_CONTEXT = 2
ERR_PAGE = 4
ERR_BUDGET = 32


def _values(bits: np.ndarray) -> np.ndarray:
    """bf16 bit patterns -> float64 values."""
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def seen_by(position: int, window: int, sinks: int) -> np.ndarray:
    """Positions that the query at ``position`` attends to, ascending."""
    t = np.arange(position + 1)
    return t[(t < sinks) | (t > position - window)]


def paged_window_attention(pool, q, query_start, block_tables, context_lens, scale, window, sinks, max_query,
                           max_context, absolute=False):
    """(out float64 [rows, heads, dim], error bits, largest sum |q_d K_d| of any score, weights by (sequence, row, kv head)).

    ``weights``: a dict of (s, row, g) -> (positions, weights [group, positions]).  ``absolute``: take |V| for V, for
    error bounds (the weights stay what they are)."""
    rows, heads, dim = q.shape
    group, P = heads // pool.num_kv_heads, pool.page_tokens
    out, err, spread, weights = np.zeros((rows, heads, dim)), 0, 0.0, {}
    for s in range(len(context_lens)):
        q0, n, ctx = int(query_start[s]), int(query_start[s + 1] - query_start[s]), int(context_lens[s])
        if n == 0:
            continue
        if n < 0 or n > max_query or ctx < 0 or ctx > max_context or n > ctx or q0 < 0 or q0 + n > rows:
            err |= ERR_CONTEXT
            continue
        for j in range(n):
            t = seen_by(ctx - n + j, window, sinks)
            page = np.asarray(block_tables[s])[t // P]
            good = (page >= 0) & (page < pool.num_pages)
            if not good.all():
                err |= ERR_PAGE
            t, page = t[good], page[good]
            if t.size == 0:
                continue
            for g in range(pool.num_kv_heads):
                K, V = _values(pool.data[page, 0, g, t % P]), _values(pool.data[page, 1, g, t % P])
                qg = _values(q[q0 + j, g * group:(g + 1) * group])
                x = qg @ K.T * scale
                w = np.exp(x - x.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                out[q0 + j, g * group:(g + 1) * group] = w @ (np.abs(V) if absolute else V)
                weights[s, j, g] = t, w
                if absolute:
                    spread = max(spread, float((np.abs(qg) @ np.abs(K).T).max()))
    return out, err, spread, weights


def decode_queries(context_lens, max_context):
    """query_start and lengths that make decode of these contexts a prefill of one token each: a sequence without (valid)
    tokens has no query; (starts, rows in the order of sequences)."""
    has = np.array([0 < int(c) <= max_context for c in context_lens])
    return np.concatenate([[0], np.cumsum(has)]).astype(np.int32), np.flatnonzero(has)


def window_decode(pool, q, block_tables, context_lens, scale, window, sinks, max_context, absolute=False):
    """As paged_window_attention, one query per sequence (zero rows where the context is empty or invalid)."""
    starts, rows = decode_queries(context_lens, max_context)
    lens = np.where((np.asarray(context_lens) > 0) & (np.asarray(context_lens) <= max_context), context_lens, 0)
    got, err, spread, weights = paged_window_attention(pool, q[rows], starts, block_tables, lens, scale, window, sinks, 1,
                                                       max_context, absolute)
    out = np.zeros(q.shape)
    out[rows] = got
    if any(int(c) < 0 or int(c) > max_context for c in context_lens):
        err |= ERR_CONTEXT
    return out, err, spread, weights


def evict(pool, block_tables, context_lens, budgets, sums, sinks, recent, max_context, max_budget):
    """Moves rows of ``pool`` in place; ``block_tables`` [seqs, layers, blocks], ``sums`` [seqs, layers, heads, tokens].
    (new sums, kept positions [seqs, layers, heads, max_budget], -1 where not written, new lengths, error bits)"""
    seqs, layers, _ = block_tables.shape
    heads, P = pool.num_kv_heads, pool.page_tokens
    new, kept = np.array(sums), np.full((seqs, layers, heads, max_budget), -1, np.int32)
    lens, err = np.array(context_lens, np.int32).copy(), 0
    for s in range(seqs):
        ctx, budget = int(context_lens[s]), int(budgets[s])
        if ctx < 0 or ctx > max_context:
            err |= ERR_CONTEXT
            continue
        if budget < 0 or min(budget, ctx) > max_budget:
            err |= ERR_BUDGET
            continue
        keep = min(budget, ctx)
        lens[s] = keep
        first = min(sinks, keep)
        last = min(recent, keep - first)
        held = []
        for layer in range(layers):
            table = block_tables[s, layer]
            for g in range(heads):
                row = [float(x) for x in sums[s, layer, g, :ctx]]
                order = sorted(range(first, ctx - last),
                               key=lambda t: (0, t) if np.isnan(row[t]) else (1, row[t], -t), reverse=True)
                # (NaN last; among them, too, the earlier position first)
                nans = sorted(t for t in order if np.isnan(row[t]))
                order = [t for t in order if not np.isnan(row[t])] + nans
                chosen = sorted([*range(first), *range(ctx - last, ctx), *order[:keep - first - last]])
                kept[s, layer, g, :keep] = chosen
                new[s, layer, g, :ctx] = 0
                new[s, layer, g, :keep] = np.asarray(sums[s, layer, g])[chosen] if keep else []
                for k, t in enumerate(chosen):
                    if t == k:
                        continue
                    a, b = int(table[t // P]), int(table[k // P])
                    if not (0 <= a < pool.num_pages and 0 <= b < pool.num_pages):
                        err |= ERR_PAGE
                        continue
                    held.append((b, g, k % P, pool.data[a, :, g, t % P].copy()))
        for page, g, r, data in held:
            pool.data[page, :, g, r] = data
    return new, kept, lens, err
