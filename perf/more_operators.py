"""Cases of the operators that bound the paged KV cache, with their plain forms.

Four operators over the paged cache (32 query heads share 8 K/V heads of dim 64; pages hold 16 tokens):

* ``window_decode``: one new token per sequence attends to the last ``window`` tokens of its cache (itself
  included) and to its first ``sinks`` tokens.
* ``window_prefill``: the same for a chunk of query tokens per sequence, each with a window of its own.
* ``weights``: decode attention over the whole cache that also adds what weight each cached token received from
  the query heads of its K/V head to a running sum per token.
* ``evict``: per sequence, layer and K/V head the tokens of the largest sums are kept (with the first few and
  the most recent ones); their K/V rows move together at the front of the sequence, in order, in place.

``run`` takes the plain form (elementary torch operations, 32 bits) where ``own`` is false, and the framework's
calls where it is true.  Sizes of a case (lengths, budgets) come from the case alone, values from the seed.
"""
import math

import numpy as np
import torch

own = False

PAGE, HEADS, KV_HEADS, DIM = 16, 32, 8, 64
GROUP = HEADS // KV_HEADS
ROW = 2 * KV_HEADS * DIM * 2            # bytes of one token's K and V
SCALE = 1.0 / math.sqrt(DIM)

# The most that a drawn case may cost, which is what the largest listed cases cost.
MAX_VISIBLE = 256 * 2048                # tokens that a window_decode case reads
MAX_SCORES = 4 * 2048 * 4096            # (query, key) pairs that a window_prefill case may hold
MAX_TOKENS = 256 * 2048                 # cached tokens of a weights case
MAX_ROWS = 64 * 16 * 2048               # (layer, token) pairs of an evict case


def listed():
    return [
        # One user of a long chat: a small window over a cache whose older pages are gone.  The latency of a call.
        {"name": "wdecode-single", "op": "window_decode", "seqs": 1, "ctx_lo": 2048, "ctx_hi": 2048, "window": 512,
         "sinks": 4, "out": "f32", "sizes": 1},
        # Continuous batching: lengths anywhere up to 8192, some shorter than the window.
        {"name": "wdecode-ragged64", "op": "window_decode", "seqs": 64, "ctx_lo": 1, "ctx_hi": 8192, "window": 1000,
         "sinks": 5, "out": "bf16", "sizes": 2},
        # A full batch of long contexts: 1 GiB of K/V inside the windows.
        {"name": "wdecode-256", "op": "window_decode", "seqs": 256, "ctx_lo": 2048, "ctx_hi": 65536, "window": 2032,
         "sinks": 16, "out": "f32", "sizes": 3},
        # One prompt's next chunk of 200 tokens, in a small window.
        {"name": "wprefill-chunk", "op": "window_prefill", "seqs": 1, "query_lo": 200, "query_hi": 200, "ctx_lo": 600,
         "ctx_hi": 600, "window": 256, "sinks": 4, "out": "f32", "sizes": 4},
        # Sixteen prompts of up to 512 tokens, whole, windows of 128.
        {"name": "wprefill-16x512", "op": "window_prefill", "seqs": 16, "query_lo": 300, "query_hi": 512, "ctx_lo": 300,
         "ctx_hi": 512, "window": 128, "sinks": 1, "out": "f32", "sizes": 5},
        # Four long documents, a chunk of 2048 tokens each, windows of 2000.
        {"name": "wprefill-4x2048", "op": "window_prefill", "seqs": 4, "query_lo": 2048, "query_hi": 2048,
         "ctx_lo": 2048, "ctx_hi": 16384, "window": 2000, "sinks": 16, "out": "bf16", "sizes": 6},
        # One user's step while its cache grows towards an eviction.
        {"name": "weights-single", "op": "weights", "seqs": 1, "ctx_lo": 2048, "ctx_hi": 2048, "decay": 1.0,
         "out": "f32", "sizes": 7},
        # Continuous batching, older steps fading out.
        {"name": "weights-ragged64", "op": "weights", "seqs": 64, "ctx_lo": 1, "ctx_hi": 2048, "decay": 0.95,
         "out": "bf16", "sizes": 8},
        # The 256 x 2048 decode batch: 1 GiB of K/V read once.
        {"name": "weights-256x2048", "op": "weights", "seqs": 256, "ctx_lo": 2048, "ctx_hi": 2048, "decay": 1.0,
         "out": "f32", "sizes": 9},
        # One sequence of 16 layers, 2048 tokens down to half.
        {"name": "evict-single", "op": "evict", "seqs": 1, "layers": 16, "ctx_lo": 2048, "ctx_hi": 2048, "keep": 0.5,
         "sinks": 4, "recent": 64, "sizes": 10},
        # Two long documents, a layer at a time: few units, each with a long axis.
        {"name": "evict-long2", "op": "evict", "seqs": 2, "layers": 1, "ctx_lo": 50001, "ctx_hi": 65536, "keep": 0.25,
         "sinks": 16, "recent": 1000, "sizes": 11},
        # A batch of 64 with all of 16 layers, ragged lengths, to 60 %.
        {"name": "evict-64x16", "op": "evict", "seqs": 64, "layers": 16, "ctx_lo": 1024, "ctx_hi": 2048, "keep": 0.6,
         "sinks": 4, "recent": 128, "sizes": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("window_decode", "window_prefill", "weights", "evict"))
    sizes = rng.randrange(1 << 30)
    out = rng.choice(("f32", "bf16"))
    if op == "window_decode":
        seqs = _log(rng, 1, 256)
        window = _log(rng, 1, min(16384, MAX_VISIBLE // seqs))
        sinks = rng.choice((0, 1, 4, rng.randrange(0, 65)))
        sinks = min(sinks, MAX_VISIBLE // seqs - window)
        ctx_hi = _log(rng, 1, 65536)
        return {"op": op, "seqs": seqs, "ctx_lo": rng.randrange(0, ctx_hi + 1), "ctx_hi": ctx_hi, "window": window,
                "sinks": sinks, "out": out, "sizes": sizes}
    if op == "window_prefill":
        seqs = _log(rng, 1, 32)
        query_hi = _log(rng, 1, 2048)
        sinks = rng.choice((0, 1, 4, rng.randrange(0, 65)))
        most = max(1, MAX_SCORES // (seqs * query_hi) - query_hi - sinks)
        window = _log(rng, 1, min(4096, most))
        query_hi = max(1, min(query_hi, MAX_SCORES // (seqs * (window + sinks + query_hi))))
        ctx_hi = _log(rng, query_hi, 16384)
        return {"op": op, "seqs": seqs, "query_lo": rng.randrange(0, query_hi + 1), "query_hi": query_hi,
                "ctx_lo": rng.randrange(0, ctx_hi + 1), "ctx_hi": ctx_hi, "window": window, "sinks": sinks,
                "out": out, "sizes": sizes}
    if op == "weights":
        seqs = _log(rng, 1, 256)
        ctx_hi = _log(rng, 1, min(131072, MAX_TOKENS // seqs))
        return {"op": op, "seqs": seqs, "ctx_lo": rng.randrange(0, ctx_hi + 1), "ctx_hi": ctx_hi,
                "decay": rng.choice((1.0, 0.9, 0.0)), "out": out, "sizes": sizes}
    layers = rng.choice((1, 2, 7, 16))
    seqs = _log(rng, 1, 64)
    ctx_hi = _log(rng, 2, min(65536, MAX_ROWS // (seqs * layers)))
    return {"op": op, "seqs": seqs, "layers": layers, "ctx_lo": rng.randrange(1, ctx_hi + 1), "ctx_hi": ctx_hi,
            "keep": rng.choice((0.1, 0.25, 0.5, 0.9, 1.0)), "sinks": rng.randrange(0, 17),
            "recent": rng.choice((0, 1, 32, 200)), "sizes": sizes}


# ---- sizes, from the case alone ----------------------------------------------------------------
def _sizes(case):
    """(query tokens, cached tokens) of every sequence, the query tokens being the last cached ones."""
    r = np.random.RandomState(case["sizes"] % (1 << 31))
    ctx = r.randint(case["ctx_lo"], case["ctx_hi"] + 1, case["seqs"]).astype(np.int64)
    if case["op"] == "window_prefill":
        n = r.randint(case["query_lo"], case["query_hi"] + 1, case["seqs"]).astype(np.int64)
        return n, np.maximum(ctx, n)
    return np.ones_like(ctx), ctx


def _budgets(case, ctx):
    return np.maximum(1, np.round(case["keep"] * ctx).astype(np.int64))


def _span(case):
    """Sizes, and per sequence the first key of the window of its first query token (none before the sinks)."""
    n, ctx = _sizes(case)
    return n, ctx, np.maximum(case["sinks"], ctx - n - case["window"] + 1)


def work(case):
    n, ctx = _sizes(case)
    out = 4 if case.get("out") == "f32" else 2
    if case["op"] == "evict":
        budget = _budgets(case, ctx)
        moved = np.where(budget < ctx, np.maximum(budget - case["sinks"], 0), 0)
        per_unit = int((moved * 512 + ctx * 8 + np.minimum(budget, ctx) * 4).sum())
        return {"bytes": per_unit * KV_HEADS * case["layers"] + 12 * case["seqs"], "flops": 0}
    if case["op"] == "weights":
        tokens = int(ctx.sum())
        return {"bytes": tokens * (ROW + KV_HEADS * 8) + case["seqs"] * (HEADS * DIM * (2 + out) + 4) +
                int(((ctx + PAGE - 1) // PAGE).sum()) * 4, "flops": 4.0 * DIM * HEADS * tokens}
    window, sinks = case["window"], case["sinks"]
    pairs = keys = 0
    for a, c in zip(n.tolist(), ctx.tolist()):
        if a == 0 or c == 0:
            continue
        p = np.arange(c - a, c)
        lo = np.maximum(p - window + 1, 0)
        pairs += int((p + 1 - lo + np.minimum(sinks, lo)).sum())
        keys += c - int(lo[0]) + min(sinks, int(lo[0]))
    rows = int(np.where(ctx > 0, n, 0).sum())
    return {"bytes": keys * ROW + rows * HEADS * DIM * (2 + out) + keys // PAGE * 4 + case["seqs"] * 4,
            "flops": 4.0 * DIM * HEADS * pairs}


# ---- inputs -------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _normal_pool(pages, g):
    """[page][K|V][kv_head][row][dim] bf16, standard normal, in steps that stay small."""
    pool = torch.empty(max(pages, 1), 2, KV_HEADS, PAGE, DIM, dtype=torch.bfloat16, device="cuda")
    for i in range(0, pool.shape[0], 8192):
        part = pool[i:i + 8192]
        part.copy_(torch.randn(part.shape, device="cuda", generator=g, dtype=torch.float32))
    return pool


def _sums(shape, ctx, g):
    """Running sums of attention weights after some 64 steps: many small, some large, the newest tokens' still at zero."""
    w = torch.rand(shape, device="cuda", generator=g).log_().neg_().pow_(3)
    w *= (43.0 / ctx.clamp(min=1)).view(shape[0], *([1] * (len(shape) - 1)))
    t = torch.arange(shape[-1], device="cuda")
    new = (t >= (ctx - 4)[:, None]).view(shape[0], *([1] * (len(shape) - 2)), shape[-1])
    return w.masked_fill_(new, 0.0)


def _inputs(case, seed):
    r = np.random.RandomState(int(seed) % (1 << 31))
    g = _gen(seed)
    n, ctx = _sizes(case)
    seqs = case["seqs"]
    blocks = max(1, int((ctx.max() + PAGE - 1) // PAGE))
    block = np.arange(blocks)[None, :]
    here = block < ((ctx + PAGE - 1) // PAGE)[:, None]          # blocks that have a page
    if case["op"].startswith("window"):                         # pages behind every window are given back
        first = _span(case)[2] // PAGE
        here &= (block * PAGE < case["sinks"]) | (block >= first[:, None])
    if case["op"] == "evict":
        here = np.repeat(here, case["layers"], axis=0)
    table = np.full(here.shape, -1, np.int32)
    pages = int(here.sum())
    table[here] = r.permutation(pages).astype(np.int32)
    s = {"lens": _dev(ctx, torch.int32), "max_context": max(1, int(ctx.max()))}
    if case["op"] == "evict":
        budget = _budgets(case, ctx)
        s["tables"] = _dev(table.reshape(seqs, case["layers"], blocks))
        s["pool"] = torch.randint(-32768, 32768, (pages, 2, KV_HEADS, PAGE, DIM), dtype=torch.int16, device="cuda",
                                  generator=g)
        s["sums"] = _sums((seqs, case["layers"], KV_HEADS, blocks * PAGE), s["lens"], g)
        s["new_sums"] = torch.zeros_like(s["sums"])
        s["budgets"] = _dev(budget, torch.int32)
        s["kept"] = torch.full((seqs, case["layers"], KV_HEADS, int(budget.max())), -1, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        return s | {"sinks": case["sinks"], "recent": case["recent"]}
    s["tables"], s["pool"] = _dev(table), _normal_pool(pages, g)
    rows = int(n.sum())
    # queries of a spread that makes the softmax as peaked as trained heads have it
    s["q"] = (2.0 * torch.randn(rows, HEADS, DIM, device="cuda", generator=g)).bfloat16()
    s["out"] = torch.empty(rows, HEADS, DIM, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16,
                           device="cuda")
    s["start"] = _dev(np.concatenate([[0], np.cumsum(n)]), torch.int32)
    s["max_query"] = int(n.max())
    if case["op"] == "weights":
        s["sums"] = _sums((seqs, KV_HEADS, blocks * PAGE), s["lens"], g)
        return s | {"decay": case["decay"]}
    return s | {"window": case["window"], "sinks": case["sinks"]}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"] = case["op"]
    if own:  # what a program of the framework keeps from call to call: the pool's handle, the status word, a workspace
        import paged_kv_cache_180_gb300 as pkv
        s["pkv"] = pkv
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["handle"] = pkv.KVPool(s["pool"].shape[0], buffer=s["pool"].view(torch.bfloat16).view(-1))
        if case["op"] == "weights":
            s["workspace"] = pkv.weights_workspace(case["seqs"], s["max_context"])
    return s


# ---- one pass -----------------------------------------------------------------------------------
def run(s):
    if s["op"] == "window_decode":
        return _own_window_decode(s) if own else _plain_window(s)
    if s["op"] == "window_prefill":
        return _own_window_prefill(s) if own else _plain_window(s)
    if s["op"] == "weights":
        return _own_weights(s) if own else _plain_weights(s)
    return _own_evict(s) if own else _plain_evict(s)


def _own_window_decode(s):
    s["pkv"].paged_window_decode_attention(s["handle"], s["out"], s["q"], s["tables"], s["tables"].shape[1], s["lens"],
                                           s["max_context"], SCALE, s["window"], s["sinks"], s["status"])
    return s["out"]


def _own_window_prefill(s):
    s["pkv"].paged_window_prefill_attention(s["handle"], s["out"], s["q"], s["start"], s["tables"],
                                            s["tables"].shape[1], s["lens"], s["max_query"], s["max_context"], SCALE,
                                            s["window"], s["sinks"], s["status"])
    return s["out"]


def _own_weights(s):
    s["pkv"].paged_decode_attention_weights(s["handle"], s["out"], s["q"], s["tables"], s["tables"].shape[1],
                                            s["lens"], s["max_context"], SCALE, s["sums"], s["decay"],
                                            s["workspace"], s["status"])
    return s["out"], s["sums"]


def _own_evict(s):
    t = s["tables"]
    s["pkv"].kv_evict(s["handle"], t, t.shape[1] * t.shape[2], t.shape[2], s["lens"], s["budgets"], s["sums"],
                      s["new_sums"], s["sinks"], s["recent"], s["max_context"], s["kept"], s["new_lens"], s["status"])
    return s["pool"], s["new_sums"], s["kept"], s["new_lens"]


def _attend(s, keys, vals, seen):
    """Softmax attention of every sequence's queries over its own list of keys ([seq, head, key, dim]) where
    ``seen`` [seq, query, key] is true; (outputs [rows, heads, dim], weights [seq, kv_head, query, head, key])."""
    start, most, rows = s["start"].long(), max(s["max_query"], 1), s["q"].shape[0]
    seqs, count = keys.shape[0], keys.shape[2]
    idx = torch.minimum(start[:-1, None] + torch.arange(most, device="cuda"), start[-1] - 1).clamp(min=0)
    q = s["q"][idx].float().view(seqs, most, KV_HEADS, GROUP, DIM).permute(0, 2, 1, 3, 4)
    score = (q.reshape(seqs, KV_HEADS, most * GROUP, DIM) @ keys.transpose(2, 3)).mul_(SCALE)
    score = score.view(seqs, KV_HEADS, most, GROUP, count).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    o = (p.view(seqs, KV_HEADS, most * GROUP, count) @ vals).view(seqs, KV_HEADS, most, GROUP, DIM)
    o = o.permute(0, 2, 1, 3, 4).reshape(seqs, most, HEADS, DIM)
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(start, row, right=True) - 1
    return o[seq, row - start[seq]].to(s["out"].dtype), p


def _plain_window(s):
    if s["q"].shape[0] == 0:
        return s["out"].clone()
    lens, tables, sinks, window = s["lens"].long(), s["tables"].long(), s["sinks"], s["window"]
    n = (s["start"][1:] - s["start"][:-1]).long()
    first = (lens - n - window + 1).clamp(min=sinks)
    front = min(sinks, s["max_context"])
    k = torch.arange(front + min(window + s["max_query"] - 1, s["max_context"]), device="cuda")
    pos = torch.where(k < front, k, first[:, None] + k - front)     # the sinks, then everything from the first window on
    own_key = pos < lens[:, None]
    place = torch.where(own_key, pos, torch.zeros_like(pos))
    page = torch.gather(tables, 1, place // PAGE).clamp(min=0)
    kv = s["pool"][page, :, :, place % PAGE]                        # [seq, key, K|V, kv_head, dim]
    keys, vals = kv[:, :, 0].transpose(1, 2).float(), kv[:, :, 1].transpose(1, 2).float()
    vals = torch.where(own_key[:, None, :, None], vals, torch.zeros_like(vals))
    at = ((lens - n)[:, None] + torch.arange(max(s["max_query"], 1), device="cuda"))[:, :, None]
    t = pos[:, None, :]
    seen = own_key[:, None, :] & (t <= at) & ((t < sinks) | (t > at - window))
    return _attend(s, keys, vals, seen)[0]


def _plain_weights(s):
    lens, tables = s["lens"].long(), s["tables"].long()
    kv = s["pool"][tables.clamp(min=0)]                             # [seq, block, K|V, kv_head, row, dim]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, tables.shape[0], KV_HEADS, -1, DIM).float()
    cached = torch.arange(kv.shape[3], device="cuda") < lens[:, None]
    vals = torch.where(cached[:, None, :, None], kv[1], torch.zeros_like(kv[1]))
    out, p = _attend(s, kv[0], vals, cached[:, None, :])
    given = p[:, :, 0].sum(2)                                       # over the query heads of a K/V head
    s["sums"].copy_(torch.where(cached[:, None, :], s["decay"] * s["sums"] + given, s["sums"]))
    return out, s["sums"]


def _plain_evict(s):
    lens, sums, tables = s["lens"].long(), s["sums"], s["tables"].long()
    keep = torch.minimum(s["budgets"].long(), lens)
    seqs, layers, _, width = sums.shape
    t = torch.arange(width, device="cuda")
    first = keep.clamp(max=s["sinks"])
    last = torch.minimum(keep - first, torch.full_like(keep, s["recent"]))
    sure = (t < first[:, None]) | ((t >= (lens - last)[:, None]) & (t < lens[:, None]))
    key = torch.where(sure[:, None, None, :], torch.full_like(sums, math.inf), sums)
    key = torch.where((t < lens[:, None])[:, None, None, :], key, torch.full_like(sums, -math.inf))
    rank = key.argsort(dim=-1, descending=True, stable=True).argsort(dim=-1)   # ties: the lower index first
    kept = rank < keep[:, None, None, None]
    at = kept.nonzero(as_tuple=True)                                # (seq, layer, head, position), positions ascending
    to = (kept.cumsum(-1) - 1)[at]
    s["new_sums"][:] = torch.where((t < lens[:, None])[:, None, None, :], torch.zeros_like(sums), s["new_sums"])
    s["new_sums"][at[0], at[1], at[2], to] = sums[at]
    s["kept"][at[0], at[1], at[2], to] = at[3].int()
    from_page, to_page = tables[at[0], at[1], at[3] // PAGE], tables[at[0], at[1], to // PAGE]
    pool = s["pool"].permute(0, 2, 3, 1, 4)                         # [page, kv_head, row, K|V, dim]
    pool[to_page, at[2], to % PAGE] = pool[from_page, at[2], at[3] % PAGE]
    s["new_lens"].copy_(keep)
    return s["pool"], s["new_sums"], s["kept"], s["new_lens"]


# ---- the definition in 64 bits ------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    lens, tables = s["lens"].tolist(), s["tables"].cpu().numpy()
    if case["op"] == "evict":
        return _exact_evict(s, lens)
    start = s["start"].tolist()
    parts, sums = [torch.zeros(0, HEADS, DIM, dtype=torch.float64, device="cuda")], None
    if case["op"] == "weights":
        sums = s["sums"].double()
    for i, ctx in enumerate(lens):
        a, b = start[i], start[i + 1]
        if a == b:
            continue
        if ctx == 0:
            parts.append(torch.zeros(b - a, HEADS, DIM, dtype=torch.float64, device="cuda"))
            continue
        p = np.arange(ctx - (b - a), ctx)
        t = np.arange(ctx)
        if case["op"] != "weights":
            t = t[(t < case["sinks"]) | (t > p[0] - case["window"])]
        page = torch.from_numpy(tables[i][t // PAGE].astype(np.int64)).cuda()
        kv = s["pool"][page, :, :, torch.from_numpy(t % PAGE).cuda()].double()      # [key, K|V, kv_head, dim]
        rows = []
        for q0 in range(a, b, 512):                                 # query tokens in steps that stay small
            q1 = min(b, q0 + 512)
            pos = p[q0 - a:q1 - a, None]
            allowed = t[None, :] <= pos
            if case["op"] != "weights":
                allowed &= (t[None, :] < case["sinks"]) | (pos - t[None, :] < case["window"])
            hide = torch.from_numpy(~allowed).cuda()
            heads = []
            for h in range(HEADS):
                x = s["q"][q0:q1, h].double() @ kv[:, 0, h // GROUP].T / math.sqrt(DIM)
                w = torch.softmax(x.masked_fill(hide, -math.inf), -1)
                heads.append(w @ kv[:, 1, h // GROUP])
                if sums is not None:
                    if h % GROUP == 0:
                        sums[i, h // GROUP, :ctx] *= case["decay"]
                    sums[i, h // GROUP, :ctx] += w[0]
            rows.append(torch.stack(heads, 1))
        parts.append(torch.cat(rows))
    out = torch.cat(parts)
    return out if sums is None else (out, sums)


def _exact_evict(s, lens):
    sums, kept = s["sums"].cpu().numpy().astype(np.float64), s["kept"].cpu().numpy()
    budgets, new = s["budgets"].tolist(), np.zeros_like(sums)
    new_lens = []
    for i, ctx in enumerate(lens):
        keep = min(budgets[i], ctx)
        first = min(s["sinks"], keep)
        last = min(s["recent"], keep - first)
        middle = sums[i, :, :, first:ctx - last]
        best = np.argsort(-middle, axis=-1, kind="stable")[..., :keep - first - last] + first
        ends = np.concatenate([np.arange(first), np.arange(ctx - last, ctx)])
        chosen = np.sort(np.concatenate([best, np.broadcast_to(ends, (*best.shape[:2], ends.size))], -1), -1)
        kept[i, :, :, :keep] = chosen
        new[i, :, :, :keep] = np.take_along_axis(sums[i], chosen, -1)
        new_lens.append(keep)
    return None, torch.from_numpy(new), torch.from_numpy(kept), torch.tensor(new_lens, dtype=torch.int32)
