"""Model of how tree attention splits a batch over its CTAs: which key blocks of which units make up each CTA's segments.

Written from the rule that ``csrc/tree_attention.cu`` states, so that a test can pick (and prove that it picked) a layout."""
from __future__ import annotations

import math

TOK, KEYS, HEADS, UNIT_COST = 32, 64, 8, 5
MERGE_COST, MERGE_COST_OCTET, LAST_ROUND = 7.0, 6.0, 0.5625
MIN_ENTRIES, MOST_ENTRIES, MERGE_GROUP = 2, 6, 5


def split(contexts, nodes, sms=152):
    """(whole units?, per CTA its segments (sequence, head, tile, first block, end block, unit's blocks)).
    With whole units the list holds each CTA's first unit only (the others are claimed as they come)."""
    G = 2 * sms
    seqs = [(s, -(-n // TOK), (c - 1) // KEYS + 1) for s, (c, n) in enumerate(zip(contexts, nodes)) if n]
    if not seqs:
        return True, []
    units = sum(HEADS * t for _, t, _ in seqs)
    T = sum(HEADS * t * (nb + UNIT_COST) for _, t, nb in seqs)
    longest = max(4 * nb + (min(nodes[s], TOK) - 1) // 8 for s, _, nb in seqs)
    merge = MERGE_COST + MERGE_COST_OCTET * ((longest & 3) + 1)
    length = (longest >> 2) + UNIT_COST
    least = min(max(length // (2 * MERGE_GROUP - 1) + 1, MIN_ENTRIES), MOST_ENTRIES)
    rounds = units / G
    idle = math.ceil(rounds) - rounds
    whole = length - merge <= max(T / G, least) and (rounds <= 1 or idle * length * LAST_ROUND <= merge)
    if whole:
        listed = [(s, g, t, 0, nb, nb) for s, tiles, nb in seqs for g in range(HEADS) for t in range(tiles)]
        return True, [[u] for u in listed[:min(units, G)]]
    ctas = min(G, max(1, T // least))
    units_in_order, at = [], 0          # even tiles of all sequences, then the odd ones
    for part in (0, 1):
        for s, tiles, nb in seqs:
            for g in range(HEADS):
                for t in range(part, tiles, 2):
                    units_in_order.append((at, s, g, t, nb))
                    at += nb + UNIT_COST
    shares = []
    for i in range(ctas):
        a, b, segments = i * T // ctas, (i + 1) * T // ctas, []
        for first, s, g, t, nb in units_in_order:
            v0, v1 = max(a - first, 0), min(b - first, nb + UNIT_COST)
            if v0 < v1 and v1 > UNIT_COST:
                segments.append((s, g, t, max(v0 - UNIT_COST, 0), v1 - UNIT_COST, nb))
        shares.append(segments)
    return False, shares


def parts_of_units(shares):
    """(sequence, head, tile) -> number of CTAs that have a part of it."""
    count = {}
    for segments in shares:
        for s, g, t, *_ in segments:
            count[s, g, t] = count.get((s, g, t), 0) + 1
    return count
