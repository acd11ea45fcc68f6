"""Cases of what a paged cache needs besides append, gather and attend, and their plain forms.

Four operators work on the paged key/value cache (pages of `page` tokens per kv
head, fp16 or bf16 entries, or e4m3 entries with one power-of-two exponent per
token and head), in two loops of serving:

  verifying drafts      tree      attention of a tree of drafted tokens over the cache: a token
                                  sees what came before the tree and its own ancestors
                        compact   the tokens of the accepted path move together
  a bounded cache       weigh     attention that also adds up the softmax weight that each
                                  cached token of each kv head gets
                        select    the tokens to keep of every sequence and kv head: the first,
                                  the latest, and those of largest weight in between
                        compact   the kept tokens (and their weights) move together

`run` computes the plain form with elementary torch operations, or (own) makes
the calls of the package.  Head width 128, the width of the package's caches.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
DT = {"float16": torch.float16, "bfloat16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"float16": 2, "bfloat16": 2, "e4m3": 1}


# ------------------------------------------------------------------- cases

def _tree(name, batch, q_lo, q_hi, heads_q, heads, len_lo, len_hi, dtype, cache, page, window, sinks, mix):
    return {"name": name, "op": "tree", "batch": batch, "q_lo": q_lo, "q_hi": q_hi, "heads_q": heads_q,
            "heads": heads, "len_lo": len_lo, "len_hi": len_hi, "dtype": dtype, "cache": cache, "page": page,
            "window": window, "sinks": sinks, "mix": mix}


def _weigh(name, batch, chunks, q_lo, q_hi, heads_q, heads, len_lo, len_hi, dtype, cache, page, window, sinks,
           observe, decay, mix):
    return {"name": name, "op": "weigh", "batch": batch, "chunks": chunks, "q_lo": q_lo, "q_hi": q_hi,
            "heads_q": heads_q, "heads": heads, "len_lo": len_lo, "len_hi": len_hi, "dtype": dtype, "cache": cache,
            "page": page, "window": window, "sinks": sinks, "observe": observe, "decay": decay, "mix": mix}


def _select(name, batch, heads, len_lo, len_hi, page, budget, recent, sinks, mix):
    return {"name": name, "op": "select", "batch": batch, "heads": heads, "len_lo": len_lo, "len_hi": len_hi,
            "page": page, "budget": budget, "recent": recent, "sinks": sinks, "mix": mix}


def _compact(name, kind, batch, heads, len_lo, len_hi, dtype, cache, page, keep_lo, keep_hi, mix):
    return {"name": name, "op": "compact", "kind": kind, "batch": batch, "heads": heads, "len_lo": len_lo,
            "len_hi": len_hi, "dtype": dtype, "cache": cache, "page": page, "keep_lo": keep_lo, "keep_hi": keep_hi,
            "mix": mix}


def listed():
    return [
        # a single sequence's draft of four tokens: latency
        _tree("tree_1x4_of_1029", 1, 4, 4, 32, 8, 1029, 1029, "float16", "float16", 16, 0, 0, 31),
        # a serving batch's small trees over caches of 1k to 16k
        _tree("tree_64x16_bf16", 64, 16, 16, 32, 8, 1024, 16384, "bfloat16", "bfloat16", 64, 0, 0, 32),
        # larger trees of several sizes over the 8-bit cache
        _tree("tree_32x64_e4m3", 32, 33, 64, 32, 8, 1024, 16384, "float16", "e4m3", 32, 0, 0, 33),
        # odd trees under a window with first tokens kept; seven query heads to a kv head
        _tree("tree_window_9x127", 9, 1, 127, 28, 4, 5001, 12288, "bfloat16", "bfloat16", 16, 4096, 4, 34),
        # a single sequence's next token, weights added up: latency
        _weigh("weigh_1x1029", 1, 0, 1, 1, 32, 8, 1029, 1029, "float16", "float16", 16, 0, 0, 0, 1.0, 41),
        # a serving batch's next tokens, caches of 1k to 16k
        _weigh("weigh_64x16k_bf16", 64, 0, 1, 1, 32, 8, 1024, 16384, "bfloat16", "bfloat16", 64, 0, 0, 0, 1.0, 42),
        # prompt chunks, of which the last 32 tokens count, and decodes, over the 8-bit cache; older weights fade
        _weigh("weigh_mixed_16_e4m3", 16, 4, 129, 512, 32, 8, 600, 8192, "bfloat16", "e4m3", 32, 0, 0, 32, 0.97, 43),
        # a prompt's chunk whose tokens all count: bound by the products
        _weigh("weigh_chunk_2048_of_8192", 1, 1, 2048, 2048, 32, 8, 8192, 8192, "bfloat16", "bfloat16", 64, 0, 0, 0,
               1.0, 44),
        # a serving batch that keeps 2048 tokens of each sequence and head
        _select("select_64x16k", 64, 8, 1024, 16384, 64, 2048, 256, 4, 51),
        # one long prompt: few rows, all of them long
        _select("select_1x131072", 1, 8, 131072, 131072, 128, 8192, 512, 16, 52),
        # accepted paths of 64 trees: a few tokens of each, the smallest moves
        _compact("accept_64x16", "accept", 64, 8, 1024, 4096, "bfloat16", "bfloat16", 16, 1, 16, 61),
        # what is kept of 16 long sequences moves together, head by head, with its weights
        _compact("evict_16x16k_bf16", "evict", 16, 8, 5000, 16384, "bfloat16", "bfloat16", 32, 4096, 4096, 62),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["tree", "tree", "weigh", "weigh", "select", "compact"])
        dtype = rng.choice(["float16", "bfloat16"])
        cache = rng.choice([dtype, "e4m3"])
        page = rng.choice([16, 32, 64, 128, 256])
        heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
        mix = rng.randrange(1 << 30)
        window = rng.choice([0, 0, 0, _log(rng, 32, 4096)])
        sinks = rng.choice([0, 1, 4, 16, 130]) if window else 0
        if op == "tree":
            q = _log(rng, 1, 256)
            hi = max(_log(rng, 64, 32768), q)
            c = _tree("", _log(rng, 1, 64), max(1, q // 3), q, heads * group, heads, max(q, hi // 8), hi, dtype, cache,
                      page, window, sinks, mix)
        elif op == "weigh":
            hi = _log(rng, 64, 32768)
            decay = rng.choice([1.0, 1.0, 0.97, 0.5, 0.0])
            if rng.random() < 0.5:
                c = _weigh("", _log(rng, 1, 64), 0, 1, 1, heads * group, heads, max(1, hi // 8), hi, dtype, cache, page,
                           window, sinks, 0, decay, mix)
            else:
                batch, q = _log(rng, 1, 16), min(_log(rng, 2, 2048), hi)
                c = _weigh("", batch, rng.randint(1, batch), max(1, q // 2), q, heads * group, heads, max(q, hi // 4),
                           hi, dtype, cache, page, window, sinks, rng.choice([0, 0, 1, 16, 32, 100]), decay, mix)
        elif op == "select":
            hi = _log(rng, 64, 131072)
            budget = min(hi, _log(rng, 16, 8192))
            c = _select("", _log(rng, 1, 64), heads, max(1, hi // 8), hi, page, budget, rng.randint(0, budget // 2),
                        rng.randint(0, min(16, budget // 2)), mix)
        else:
            hi = _log(rng, 64, 32768)
            if rng.random() < 0.5:
                n = min(hi, _log(rng, 1, 256))
                c = _compact("", "accept", _log(rng, 1, 64), heads, max(n, hi // 8), hi, dtype, cache, page, 1, n, mix)
            else:
                n = _log(rng, 16, max(16, hi // 2))
                c = _compact("", "evict", _log(rng, 1, 64), heads, max(1, hi // 8), hi, dtype, cache, page, n, n, mix)
        w = work(c)
        if w["bytes"] > 2.2e9 or w["flops"] > 3.5e11:
            continue
        lens, news = _lengths(c)
        if op == "select" and max(lens) <= c["budget"]:  # nothing to choose
            continue
        if c["batch"] * c["heads"] * max(lens) * D * 4 > 5.0e9:
            continue
        # the plain form's padded scores stay within the card
        if op in ("tree", "weigh") and c["batch"] * max(news) * c["heads_q"] * max(lens) * 4 > 1.0e10:
            continue
        del c["name"]
        return c


def _lengths(case):
    """(cache lengths, new tokens) of the case's sequences, the new ones counted in the lengths;
    of `compact` the tokens that are kept."""
    r = random.Random(case["mix"])
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    op = case["op"]
    if op == "select":
        return lens, None
    if op == "compact":
        return lens, [min(n, r.randint(case["keep_lo"], case["keep_hi"])) for n in lens]
    chunks = case["batch"] if op == "tree" else case["chunks"]
    news = [r.randint(case["q_lo"], case["q_hi"]) if i < chunks else 1 for i in range(case["batch"])]
    r.shuffle(news)  # prompts and decodes come in any order
    return lens, [min(q, n) for q, n in zip(news, lens)]


def _parents(case, news):
    """Each drafted token's parent among the new tokens of its sequence, -1: the last cached token."""
    r = random.Random(case["mix"] + 1)
    out = []
    for n in news:
        wide = r.choice([1.5, 3.0, 8.0])  # chains, small trees, broad ones
        out += [max(-1, i - 1 - int(r.expovariate(1.0) * (wide - 1.0))) for i in range(n)]
    return out


def _depths(parents, news):
    """The number of ancestors of each drafted token."""
    out, t = [], 0
    for n in news:
        for i in range(n):
            p = parents[t + i]
            out.append(0 if p < 0 else out[t + p] + 1)
        t += n
    return out


def _visible(pos, window, sinks):
    """Positions up to `pos` that a token there sees."""
    if not window:
        return pos + 1
    return min(pos + 1, window) + max(0, min(sinks, pos + 1 - window))


def work(case):
    op = case["op"]
    lens, news = _lengths(case)
    if op == "select":
        b = [min(n, case["budget"]) for n in lens]
        mid = [max(0, n - case["recent"] - case["sinks"]) if n > case["budget"] else 0 for n in lens]
        return {"bytes": 4 * case["heads"] * (sum(mid) + case["batch"] * case["budget"]) + 8 * sum(x > 0 for x in b),
                "flops": 0}
    cb = SIZE[case["cache"]]
    entry = 2 * (D * cb + (1 if case["cache"] == "e4m3" else 0))  # a token's key and value of one head
    if op == "compact":
        one, keeps = (0, 1) if case["kind"] == "accept" else (4, case["heads"])
        return {"bytes": sum(news) * (2 * case["heads"] * (entry + one) + 4 * keeps), "flops": 0}
    pairs = scored = keys = updated = 0
    depth = _depths(_parents(case, news), news) if op == "tree" else None
    w, s, t = case["window"], case["sinks"], 0
    for n, q in zip(lens, news):
        lo = n - q  # the position of the first new token
        for i in range(q):
            seen = _visible(lo + (depth[t + i] if depth else i), w, s)
            pairs += seen
            if op == "weigh" and (case["observe"] == 0 or i >= q - case["observe"]):
                scored += seen
        first = max(0, lo - w + 1) if w else 0
        keys += n - first + min(s, first)
        t += q
    updated = keys if op == "weigh" else 0
    tokens = sum(news)
    flops = 4 * D * case["heads_q"] * pairs
    if op == "weigh" and case["chunks"]:
        flops += 2 * D * case["heads_q"] * scored  # chunks' scores are computed twice, their sums have to be known first
    return {"bytes": keys * case["heads"] * entry + 2 * tokens * case["heads_q"] * D * 2 + updated * case["heads"] * 8,
            "flops": flops}


# ------------------------------------------------------------------ inputs

def _pow2(k):
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(x):
    """(e4m3 entries, exponents + 127) of rows of x: x = entry * 2^exponent, the exponent the
    least in [-32, 64] that holds the row's largest magnitude below 448 (0 for a zero row)."""
    top = x.abs().amax(-1)
    bits = top.view(torch.int32)
    k = (bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    k = torch.where(top == 0, torch.zeros_like(k), k.clamp(-32, 64))
    y = (x * _pow2(-k)[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), (k + 127).to(torch.uint8)


def _pool(gen, count, case, dtype):
    """Pages with keys or values: channels of different size, as projections give."""
    shape = (count, case["heads"], case["page"], D)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if case["cache"] == "e4m3" else dtype)
    x *= torch.exp2(torch.rand((case["heads"], 1, D), generator=gen, device="cuda") * 2 - 1).to(x.dtype)
    return _quantise(x) if case["cache"] == "e4m3" else (x, None)


def _cache(gen, count, case, dtype):
    k, ke = _pool(gen, count, case, dtype)
    v, ve = _pool(gen, count, case, dtype)
    return {"k_pages": k, "v_pages": v, "k_exp": ke, "v_exp": ve}


def _table(gen, lens, kept, page):
    """(block table, pages in the pool): pages of all sequences shuffled in the pool, -1 where a
    sequence holds none; kept(b, p) says whether sequence b still holds its page p."""
    width = max(-(-n // page) for n in lens)
    rows = [[kept(b, p) for p in range(-(-n // page))] + [False] * (width - -(-n // page)) for b, n in enumerate(lens)]
    held = torch.tensor(rows, device="cuda")
    used = sum(sum(r) for r in rows)
    count = used + used // 16 + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[held] = torch.randperm(count, generator=gen, device="cuda")[:used].to(torch.int32)
    return table, count


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _weights(gen, count, case):
    """Accumulated softmax weights: a few large, most small, some that underflowed to zero."""
    shape = (count, case["heads"], case["page"])
    w = torch.exp(2.0 * torch.randn(shape, generator=gen, device="cuda")) / 4096
    return w * (torch.rand(shape, generator=gen, device="cuda") > 0.02)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    page, heads, op = case["page"], case["heads"], case["op"]
    lens, news = _lengths(case)
    if op == "select":
        table, count = _table(gen, lens, lambda b, p: True, page)
        return {"op": op, "weights": _weights(gen, count, case), "table": table, "lens": _int32(lens),
                "budget": case["budget"], "recent": case["recent"], "sinks": case["sinks"]}
    dtype = DT[case["dtype"]]
    if op == "compact":
        table, count = _table(gen, lens, lambda b, p: True, page)
        state = {"op": op, "table": table, "counts": _int32(news), "cache": _cache(gen, count, case, dtype),
                 "first": None, "weights": None}
        accept = case["kind"] == "accept"
        keep = torch.full((case["batch"], 1 if accept else heads, max(news)), -1, dtype=torch.int32, device="cuda")
        first = []
        for b, (n, m) in enumerate(zip(lens, news)):
            if accept:  # some m of the last tokens, in order: a path from the root down
                q = min(n, 2 * case["keep_hi"])
                m = min(m, q)
                first.append(n - q)
                keep[b, 0, :m] = n - q + _subset(gen, 1, q, m)[0]
            else:  # each head keeps the first four tokens and others
                keep[b, :, :m] = _subset(gen, heads, n, m, 4)
        if accept:
            state["first"] = _int32(first)
        else:
            state["weights"] = _weights(gen, count, case)
        state["keep"] = keep
        return state
    window, sinks = case["window"], case["sinks"]

    def kept(b, p):  # pages that no new token sees any more were given back
        return not window or p * page < sinks or (p + 1) * page > lens[b] - news[b] - window + 1

    table, count = _table(gen, lens, kept, page)
    tokens = sum(news)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    q = torch.randn((tokens, (case["heads_q"] + 2 * heads) * D), generator=gen, device="cuda", dtype=dtype)
    q = q[:, :case["heads_q"] * D].view(tokens, case["heads_q"], D)  # the queries' part of a fused projection
    state = {"op": op, "q": q, "table": table, "lens": _int32(lens), "cu": _int32(cu), "max_q": max(news),
             "scale": 1.0 / math.sqrt(D), "window": window, "sinks": sinks, "cache": _cache(gen, count, case, dtype)}
    if op == "tree":
        state["parents"] = _int32(_parents(case, news))
    else:
        state.update(weights=_weights(gen, count, case), observe=case["observe"], decay=case["decay"])
    return state


def _subset(gen, rows, n, m, first=0):
    """m of the numbers below n in ascending order, each row its own; the `first` lowest always."""
    x = torch.rand((rows, n), generator=gen, device="cuda")
    x[:, :first] = 2.0
    return x.argsort(-1, descending=True)[:, :m].sort(-1).values.to(torch.int32)


# --------------------------------------------------------------------- run

def run(state):
    op = state["op"]
    if own:
        from kv_cache_quantization_turboquantrvq_gb300 import api
        if op == "tree":
            return api.vq_paged_attend_tree(state["q"], state["cache"], state["table"], state["cu"], state["lens"],
                                            state["parents"], state["scale"], max_q=state["max_q"],
                                            window=state["window"], sinks=state["sinks"])
        if op == "weigh":
            out = api.vq_paged_attend_weigh(state["q"], state["cache"], state["weights"], state["table"], state["cu"],
                                            state["lens"], state["scale"], max_q=state["max_q"],
                                            window=state["window"], sinks=state["sinks"], observe=state["observe"],
                                            decay=state["decay"])
            return {"out": out, "weights": state["weights"]}
        if op == "select":
            keep, counts = api.vq_paged_select(state["weights"], state["table"], state["lens"], state["budget"],
                                               recent=state["recent"], sinks=state["sinks"])
            return {"keep": keep, "counts": counts}
        api.vq_paged_compact(state["cache"], state["table"], state["keep"], state["counts"], first=state["first"],
                             weights=state["weights"])
        return _moved(state)
    if op == "tree":
        return _attend_plain(state)[0]
    if op == "weigh":
        return _weigh_plain(state)
    if op == "select":
        return _select_plain(state)
    return _compact_plain(state)


def _moved(state):
    c = state["cache"]
    out = {"k": c["k_pages"], "v": c["v_pages"]}
    if c["k_exp"] is not None:
        out["k_exp"], out["v_exp"] = c["k_exp"], c["v_exp"]
    if state["weights"] is not None:
        out["weights"] = state["weights"]
    return out


def _rows(pages, exps, table, tokens):
    """Values [B, S, heads, D] of the tokens [B, S] (indices into each sequence), 0 where no page is held."""
    page, width = pages.shape[2], table.shape[1]
    p = table.long().gather(1, (tokens // page).clamp(max=width - 1))
    held = (p >= 0) & (tokens // page < width)
    at = (p.clamp(min=0), slice(None), tokens % page)
    if exps is None:
        x = pages[at].float()
    else:
        x = pages.view(torch.uint8)[at].view(pages.dtype).float() * _pow2(exps[at].to(torch.int32) - 127)[..., None]
    return x, held


def _tree_masks(parents, cu, n):
    """(ancestors [B, n, n], the token itself among them; depths [B, n]) of the sequences' trees."""
    i = torch.arange(n, device="cuda")
    p = parents.long()[(cu[:-1, None] + i).clamp(max=parents.numel() - 1)]
    inside = i < (cu[1:] - cu[:-1])[:, None]
    up = ((p[..., None] == i) & inside[..., None]).float()  # one step
    reach = up + torch.eye(n, device="cuda")
    steps = 1
    while steps < n:  # twice as many steps a product
        reach = (torch.matmul(reach, reach) > 0).float()
        steps *= 2
    return reach > 0, reach.sum(-1).long() - 1


def _attend_plain(state):
    """(outputs, softmax weights [B, heads, n, group, S], which keys a token sees [B, n, S])."""
    c, q, lens, cu = state["cache"], state["q"], state["lens"].long(), state["cu"].long()
    heads, page = c["k_pages"].shape[1:3]
    tokens, heads_q, _ = q.shape
    batch, n, group = lens.numel(), state["max_q"], heads_q // heads
    base = lens - (cu[1:] - cu[:-1])
    j = torch.arange(state["table"].shape[1] * page, device="cuda")
    i = torch.arange(n, device="cuda")
    if state["op"] == "tree":
        reach, depth = _tree_masks(state["parents"], cu, n)
        pos = base[:, None] + depth
        a = (j - base[:, None]).clamp(0, n - 1)  # a key's place in the tree
        new = j >= base[:, None]
        at = torch.where(new, base[:, None] + depth.gather(1, a), j)  # positions
        see = (~new)[:, None] | reach.gather(2, a[:, None].expand(-1, n, -1))
    else:
        pos = base[:, None] + i
        at = j.expand(batch, -1)
        see = j <= pos[..., None]
    see = see & (j < lens[:, None])[:, None]
    if state["window"]:
        see &= (at[:, None] > pos[..., None] - state["window"]) | (at[:, None] < state["sinks"])
    k, _ = _rows(c["k_pages"], c["k_exp"], state["table"], j.expand(batch, -1))
    v, held = _rows(c["v_pages"], c["v_exp"], state["table"], j.expand(batch, -1))
    v = v.masked_fill(~(held & (j < lens[:, None]))[..., None, None], 0.0)
    at = (cu[:-1, None] + i).clamp(max=tokens - 1)
    x = q[at].float().view(batch, n, heads, group, D).permute(0, 2, 1, 3, 4).reshape(batch, heads, n * group, D)
    s = torch.matmul(x, k.permute(0, 2, 3, 1)) * state["scale"]
    s = s.view(batch, heads, n, group, -1).masked_fill_(~see[:, None, :, None], float("-inf"))
    s -= s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = s.exp_()
    p /= p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.view(batch, heads, n * group, -1), v.transpose(1, 2)).view(batch, heads, n, group, D)
    o = o.permute(0, 2, 1, 3, 4).reshape(batch, n, heads_q, D)
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    return o[b, t - cu[b]].to(q.dtype), p, see


def _weigh_plain(state):
    out, p, see = _attend_plain(state)
    cu, lens, table, w = state["cu"].long(), state["lens"].long(), state["table"].long(), state["weights"]
    page = w.shape[2]
    n = (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(state["max_q"], device="cuda")
    inside = i < n
    counted = inside & (i >= n - state["observe"]) if state["observe"] else inside
    j = torch.arange(see.shape[2], device="cuda")
    new = p.sum(3).masked_fill_(~counted[:, None, :, None], 0.0).sum(2).transpose(1, 2)  # [B, S, heads]
    b, s = ((see & inside[..., None]).any(1) & (table.repeat_interleave(page, 1) >= 0)).nonzero(as_tuple=True)
    at = (table[b, s // page], slice(None), s % page)
    old = torch.where((j >= lens[:, None] - n)[b, s][:, None], torch.zeros_like(w[at]), w[at] * state["decay"])
    w[at] = old + new[b, s]
    return {"out": out, "weights": w}


def _select_plain(state):
    w, table, lens = state["weights"], state["table"].long(), state["lens"].long()
    page, budget, recent, sinks = w.shape[2], state["budget"], state["recent"], state["sinks"]
    batch, heads = lens.numel(), w.shape[1]
    j = torch.arange(table.shape[1] * page, device="cuda")
    x = w[table.clamp(min=0)].permute(0, 2, 1, 3).reshape(batch, heads, -1)
    inside = (j < lens[:, None])[:, None]
    x = x.masked_fill((j < sinks) | (j >= lens[:, None] - recent)[:, None], float("inf")).masked_fill(~inside, float("-inf"))
    order = x.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    counts = lens.clamp(max=budget)
    order = order.masked_fill(torch.arange(order.shape[-1], device="cuda") >= counts[:, None, None], 1 << 30).sort(-1).values
    keep = torch.full((batch, heads, budget), -1, dtype=torch.int32, device="cuda")
    keep[..., :order.shape[-1]] = order.masked_fill(order == 1 << 30, -1).to(torch.int32)
    return {"keep": keep, "counts": counts.to(torch.int32)}


def _compact_plain(state):
    c, keep, counts, table = state["cache"], state["keep"].long(), state["counts"].long(), state["table"].long()
    heads, page = c["k_pages"].shape[1:3]
    keep = keep.expand(-1, heads, -1)
    i = torch.arange(keep.shape[2], device="cuda")
    b, h, r = (i < counts[:, None, None]).expand_as(keep).nonzero(as_tuple=True)
    src = keep[b, h, r]
    dst = r if state["first"] is None else state["first"].long()[b] + r
    at = (table[b, dst // page], h, dst % page)
    of = (table[b, src // page], h, src % page)
    for x in "kv":
        pages = c[x + "_pages"]
        pages = pages.view(torch.uint8) if c[x + "_exp"] is not None else pages
        pages[at] = pages[of]
        if c[x + "_exp"] is not None:
            c[x + "_exp"][at] = c[x + "_exp"][of]
    if state["weights"] is not None:
        state["weights"][at] = state["weights"][of]
    return _moved(state)


# ------------------------------------------------------- from the definition

def _two_to(e):
    """2^e in float64 for whole e in [-128, 128], from a table: exact on every device."""
    return torch.tensor([2.0 ** i for i in range(-128, 129)], dtype=torch.float64, device=e.device)[e.long() + 128]


def _exact_rows(c, x, table_row, n):
    """Float64 values [n, heads, D] of a sequence's first n tokens; pages given back count as zeros."""
    pages = c[x + "_pages"]
    p = table_row[:-(-n // pages.shape[2])].long()
    if c["k_exp"] is None:
        r = pages[p.clamp(min=0)].double()
    else:
        r = pages.view(torch.uint8)[p.clamp(min=0)].view(pages.dtype).double()
        r = r * _two_to(c[x + "_exp"][p.clamp(min=0)].long() - 127)[..., None]
    r[p < 0] = 0
    return r.transpose(1, 2).reshape(-1, pages.shape[1], D)[:n]


def exact(case, seed):
    op = case["op"]
    state = prepare(case, seed)
    lens, news = _lengths(case)
    if op == "select":
        return _select_exact(case, state, lens)
    if op == "compact":
        return _compact_exact(case, state, news)
    if work(case)["flops"] > 1e12:
        return None
    c, table, page = state["cache"], state["table"], case["page"]
    parents = state["parents"].tolist() if op == "tree" else None
    out, t, group = [], 0, case["heads_q"] // case["heads"]
    w = state["weights"].double() if op == "weigh" else None
    for b, (n, m) in enumerate(zip(lens, news)):
        k, v = _exact_rows(c, "k", table[b], n), _exact_rows(c, "v", table[b], n)
        base = n - m
        hide = np.zeros((m, n), dtype=bool)
        for i in range(m):
            if op == "tree":
                path = [i]
                while parents[t + path[-1]] >= 0:
                    path.append(parents[t + path[-1]])
                hide[i, base:] = True
                pos = base + len(path) - 1
                for up, a in enumerate(path):
                    key = pos - up
                    hide[i, base + a] = case["window"] and key <= pos - case["window"] and key >= case["sinks"]
            else:
                pos = base + i
                hide[i, pos + 1:] = True
            if case["window"]:
                hide[i, min(base, case["sinks"]):max(min(base, case["sinks"]), min(base, pos - case["window"] + 1))] = True
                if op == "weigh":  # the chunk's own earlier tokens
                    hide[i, max(base, case["sinks"]):max(base, case["sinks"], pos - case["window"] + 1)] = True
        hide = torch.from_numpy(hide).cuda()
        o = torch.empty((m, case["heads_q"], D), dtype=torch.float64, device="cuda")
        added = torch.zeros((n, case["heads"]), dtype=torch.float64, device="cuda")
        for h in range(case["heads_q"]):
            s = state["q"][t:t + m, h].double() @ k[:, h // group].T * state["scale"]
            s[hide] = -math.inf
            p = torch.softmax(s, -1)
            o[:, h] = p @ v[:, h // group]
            if w is not None:
                added[:, h // group] += p[max(0, m - case["observe"]) if case["observe"] else 0:].sum(0)
        if w is not None:
            j = (~hide).any(0).nonzero()[:, 0]
            at = (table[b].long()[j // page], slice(None), j % page)
            w[at] = w[at] * ((j < base).double() * case["decay"])[:, None] + added[j]
        out.append(o)
        t += m
    out = torch.cat(out)
    return out if op == "tree" else {"out": out, "weights": w}


def _select_exact(case, state, lens):
    w, table = state["weights"].cpu().numpy(), state["table"].cpu().numpy()
    budget, recent, sinks, page = case["budget"], case["recent"], case["sinks"], case["page"]
    keep = np.full((case["batch"], case["heads"], budget), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for h in range(case["heads"]):
            if n <= budget:
                keep[b, h, :n] = np.arange(n)
                continue
            mid = np.arange(sinks, n - recent)
            x = w[table[b, mid // page], h, mid % page].astype(np.float64)
            best = mid[np.argsort(-x, kind="stable")[:budget - sinks - recent]]
            keep[b, h] = np.concatenate([np.arange(sinks), np.sort(best), np.arange(n - recent, n)])
    return {"keep": torch.from_numpy(keep).cuda(), "counts": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32).cuda()}


def _compact_exact(case, state, news):
    table, keep, page = state["table"].long(), state["keep"].long(), case["page"]
    names = {"k": "k_pages", "v": "v_pages", "k_exp": "k_exp", "v_exp": "v_exp"}
    src = {k: state["cache"][n] for k, n in names.items() if state["cache"][n] is not None}
    if state["weights"] is not None:
        src["weights"] = state["weights"]
    wide = {k: x if x.dtype == torch.uint8 else x.double() for k, x in src.items()}
    out = {k: x.clone() for k, x in wide.items()}
    counts = state["counts"].tolist()
    for b, m in enumerate(counts):
        first = 0 if state["first"] is None else int(state["first"][b])
        place = first + torch.arange(m, device="cuda")
        for h in range(case["heads"]):
            j = keep[b, h if keep.shape[1] > 1 else 0, :m]
            for k in out:
                out[k][table[b, place // page], h, place % page] = wide[k][table[b, j // page], h, j % page]
    return out
