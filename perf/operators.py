"""Cases of the paged-cache operators and their plain forms.

Three operators work on one paged key/value cache (pages of `page` tokens per
kv head, fp16 or bf16 entries, or e4m3 entries with one power-of-two exponent
per token and head):

  append  writes the keys and values of new tokens into their slots
  gather  reads a range of tokens of every sequence back, contiguous
  attend  attention of each sequence's new tokens (one or a chunk) over its
          pages, causal, optionally with a sliding window and a few first
          tokens that stay visible

`run` computes the plain form with elementary torch operations, or (own) makes
the calls of the package.  Head width 128, the width of the package's caches.
"""
import math
import random

import torch

own = False

D = 128
DT = {"float16": torch.float16, "bfloat16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"float16": 2, "bfloat16": 2, "e4m3": 1}


# ------------------------------------------------------------------- cases

def _append(name, tokens, heads, dtype, cache, page, skip=0, decode=False):
    return {"name": name, "op": "append", "tokens": tokens, "heads": heads, "dtype": dtype, "cache": cache,
            "page": page, "skip": skip, "decode": decode}


def _gather(name, batch, heads, out_len, len_lo, len_hi, cache, out, page, mix, first):
    return {"name": name, "op": "gather", "batch": batch, "heads": heads, "out_len": out_len, "len_lo": len_lo,
            "len_hi": len_hi, "cache": cache, "out": out, "page": page, "mix": mix, "first": first}


def _attend(name, batch, chunks, q_lo, q_hi, heads_q, heads, len_lo, len_hi, dtype, cache, page, window, sinks, mix):
    return {"name": name, "op": "attend", "batch": batch, "chunks": chunks, "q_lo": q_lo, "q_hi": q_hi,
            "heads_q": heads_q, "heads": heads, "len_lo": len_lo, "len_hi": len_hi, "dtype": dtype,
            "cache": cache, "page": page, "window": window, "sinks": sinks, "mix": mix}


def listed():
    return [
        # one decode step of 64 sequences: one new token each, the smallest write
        _append("append_step_64", 64, 8, "bfloat16", "e4m3", 16, decode=True),
        # a prompt chunk written in 8 bits, keys and values cut out of a fused projection
        _append("append_chunk_8192_e4m3", 8192, 8, "float16", "e4m3", 64),
        # packed prompts of odd length with padding tokens that have no slot, kept in 16 bits
        _append("append_packed_16411_bf16", 16411, 8, "bfloat16", "bfloat16", 32, skip=37),
        # the decode-time flush: a block of 128 tokens of each of 64 sequences comes out of the pages
        _gather("gather_flush_64x128", 64, 8, 128, 1024, 16384, "float16", "float16", 16, 11, "tail"),
        # the long-context cache read back whole for the codecs
        _gather("gather_long_4x32768_e4m3", 4, 32, 32768, 30011, 32768, "e4m3", "float16", 128, 12, "start"),
        # a single sequence's next token: latency
        _attend("decode_1x1029", 1, 0, 1, 1, 32, 8, 1029, 1029, "float16", "float16", 16, 0, 0, 21),
        # a serving batch's next tokens, caches of 1k to 16k
        _attend("decode_64x16k_bf16", 64, 0, 1, 1, 32, 8, 1024, 16384, "bfloat16", "bfloat16", 64, 0, 0, 22),
        # the same batch over the 8-bit cache
        _attend("decode_64x16k_e4m3", 64, 0, 1, 1, 32, 8, 1024, 16384, "float16", "e4m3", 32, 0, 0, 22),
        # long sequences under a window, their first tokens kept, the pages between given back
        _attend("decode_window_32x32k", 32, 0, 1, 1, 64, 8, 8192, 32768, "bfloat16", "bfloat16", 16, 4096, 4, 23),
        # a step that mixes prompt chunks with decodes over the 8-bit cache
        _attend("mixed_16_e4m3", 16, 4, 129, 512, 32, 8, 600, 8192, "bfloat16", "e4m3", 32, 0, 0, 24),
        # a prompt's last chunk over everything before it: the largest, bound by the products
        _attend("chunk_4096_of_16384", 1, 1, 4096, 4096, 32, 8, 16384, 16384, "bfloat16", "bfloat16", 64, 0, 0, 25),
        # chunks under a window with first tokens kept; seven query heads to a kv head, odd lengths
        _attend("chunk_window_2x2048", 2, 2, 1531, 2048, 28, 4, 9001, 12288, "float16", "float16", 16, 1024, 16, 26),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["append", "gather", "attend", "attend", "attend"])
        dtype = rng.choice(["float16", "bfloat16"])
        cache = rng.choice([dtype, "e4m3"])
        page = rng.choice([16, 32, 64, 128])
        if op == "append":
            c = _append("", _log(rng, 1, 32768), rng.choice([1, 2, 4, 8]), dtype, cache, page,
                        skip=rng.choice([0, 0, 5, 37]), decode=rng.random() < 0.3)
        elif op == "gather":
            hi = _log(rng, 64, 32768)
            c = _gather("", _log(rng, 1, 64), rng.choice([1, 4, 8, 32]), _log(rng, 16, hi), max(1, hi // 8), hi,
                        cache, dtype, page, rng.randrange(1 << 30), rng.choice(["start", "tail"]))
        else:
            heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
            hi = _log(rng, 64, 32768)
            window = rng.choice([0, 0, _log(rng, 32, 4096)])
            sinks = rng.choice([0, 1, 4, 16, 130]) if window else 0
            if rng.random() < 0.5:
                c = _attend("", _log(rng, 1, 64), 0, 1, 1, heads * group, heads, max(1, hi // 8), hi, dtype, cache,
                            page, window, sinks, rng.randrange(1 << 30))
            else:
                batch, q = _log(rng, 1, 16), min(_log(rng, 2, 4096), hi)
                c = _attend("", batch, rng.randint(1, batch), max(1, q // 2), q, heads * group, heads, max(q, hi // 4),
                            hi, dtype, cache, page, window, sinks, rng.randrange(1 << 30))
        w = work(c)
        if w["bytes"] > 3.2e9 or w["flops"] > 9.0e11:
            continue
        if op == "attend":
            lens, news = _lengths(c)
            # the plain form's padded scores and caches stay within the card
            if c["batch"] * max(news) * c["heads_q"] * max(lens) * 4 > 1.0e10:
                continue
            if c["batch"] * c["heads"] * max(lens) * D * 4 > 5.0e9:
                continue
        del c["name"]
        return c


def _lengths(case):
    """(cache lengths, new tokens) of the case's sequences, the new ones counted in the lengths."""
    r = random.Random(case["mix"])
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    if case["op"] == "gather":
        return lens, None
    news = [r.randint(case["q_lo"], case["q_hi"]) if i < case["chunks"] else 1 for i in range(case["batch"])]
    order = list(range(case["batch"]))
    r.shuffle(order)  # prompts and decodes come in any order
    news = [min(news[i], n) for i, n in zip(order, lens)]
    return lens, news


def _slots_used(case):
    return case["tokens"] - (case["tokens"] // case["skip"] if case["skip"] else 0)


def work(case):
    cb = SIZE[case["cache"]]
    entry = 2 * (D * cb + (1 if case["cache"] == "e4m3" else 0))  # a token's key and value of one head
    if case["op"] == "append":
        n = _slots_used(case) * case["heads"]
        return {"bytes": n * (2 * D * 2 + entry) + 8 * case["tokens"], "flops": 0}
    lens, news = _lengths(case)
    if case["op"] == "gather":
        held = sum(min(case["out_len"], n - s) for n, s in zip(lens, _first(case, lens)))
        return {"bytes": case["heads"] * (held * entry + case["batch"] * case["out_len"] * 2 * D * 2), "flops": 0}
    pairs = keys = 0
    for n, q in zip(lens, news):
        lo = n - q  # position of the first new token
        if case["window"]:
            w, s = case["window"], case["sinks"]
            pairs += sum(min(p + 1, w) + max(0, min(s, p + 1 - w)) for p in range(lo, n))
            first = max(0, lo - w + 1)
            keys += n - first + min(s, first)
        else:
            pairs += q * lo + q * (q + 1) // 2
            keys += n
    tokens = sum(news)
    return {"bytes": keys * case["heads"] * entry + 2 * tokens * case["heads_q"] * D * 2,
            "flops": 4 * D * case["heads_q"] * pairs}


# ------------------------------------------------------------------ inputs

def _first(case, lens):
    """The first token that a gather reads of each sequence."""
    if case["first"] == "start":
        return [0] * len(lens)
    return [max(0, (n - case["out_len"]) // 16 * 16) for n in lens]  # the last whole block or so


def _pow2(k):
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(x):
    """(e4m3 entries, exponents + 127) of rows of x: x = entry * 2^exponent, the exponent the
    least in [-32, 64] that holds the row's largest magnitude below 448 (0 for a zero row)."""
    x = x.float()
    top = x.abs().amax(-1)
    bits = top.view(torch.int32)
    k = (bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    k = torch.where(top == 0, torch.zeros_like(k), k.clamp(-32, 64))
    y = (x * _pow2(-k)[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), (k + 127).to(torch.uint8)


def _entries(pages, exps):
    """The values that pages of the cache stand for, in 32 bits."""
    if exps is None:
        return pages.float()
    return pages.float() * _pow2(exps.to(torch.int32) - 127)[..., None]


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


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    page, heads = case["page"], case["heads"]
    if case["op"] == "append":
        n, dtype = case["tokens"], DT[case["dtype"]]
        count = n + 8 if case["decode"] else -(-n // page) + 2
        qkv = torch.randn((n, 6 * heads * D), generator=gen, device="cuda", dtype=dtype)
        k = qkv[:, 4 * heads * D:5 * heads * D].view(n, heads, D)
        v = qkv[:, 5 * heads * D:].view(n, heads, D)
        if case["decode"]:  # every token goes to a page of its own, at any place in it
            slots = torch.randperm(count, generator=gen, device="cuda")[:n] * page
            slots += torch.randint(0, page, (n,), generator=gen, device="cuda")
        else:
            i = torch.arange(n, device="cuda")
            slots = torch.randperm(count, generator=gen, device="cuda")[i // page] * page + i % page
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1
        return {"op": "append", "k": k, "v": v, "slots": slots, "cache": _cache(gen, count, case, dtype)}
    lens, news = _lengths(case)
    if case["op"] == "gather":
        first = _first(case, lens)
        table, count = _table(gen, lens, lambda b, p: True, page)
        dtype = DT[case["out"]]
        return {"op": "gather", "table": table, "lens": _int32(lens), "first": _int32(first),
                "out_len": case["out_len"], "dtype": dtype, "cache": _cache(gen, count, case, dtype)}
    window, sinks, dtype = case["window"], case["sinks"], DT[case["dtype"]]

    def kept(b, p):  # pages that no new token sees any more were given back
        return not window or p * page < sinks or (p + 1) * page > lens[b] - news[b] - window + 1

    table, count = _table(gen, lens, kept, page)
    tokens = sum(news)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    q = torch.randn((tokens, (case["heads_q"] + 2 * heads) * D), generator=gen, device="cuda", dtype=dtype)
    q = q[:, :case["heads_q"] * D].view(tokens, case["heads_q"], D)  # the queries' part of a fused projection
    return {"op": "attend", "q": q, "table": table, "lens": _int32(lens), "cu": _int32(cu), "max_q": max(news),
            "scale": 1.0 / math.sqrt(D), "window": window, "sinks": sinks, "cache": _cache(gen, count, case, dtype)}


# --------------------------------------------------------------------- run

def run(state):
    if own:
        from kv_cache_quantization_turboquantrvq_gb300 import api
        c = state["cache"]
        if state["op"] == "append":
            api.vq_paged_append(state["k"], state["v"], c, state["slots"])
            return _written(c)
        if state["op"] == "gather":
            return api.vq_paged_gather(c, state["table"], state["lens"], state["out_len"], first=state["first"],
                                       dtype=state["dtype"])
        return api.vq_paged_attend(state["q"], c, state["table"], state["cu"], state["lens"], state["scale"],
                                   max_q=state["max_q"], window=state["window"], sinks=state["sinks"])
    if state["op"] == "append":
        return _append_plain(state)
    if state["op"] == "gather":
        return _gather_plain(state)
    return _attend_plain(state)


def _written(c):
    out = {"k": c["k_pages"], "v": c["v_pages"]}
    if c["k_exp"] is not None:
        out["k_exp"], out["v_exp"] = c["k_exp"], c["v_exp"]
    return out


def _store(rows, pages, exps, at):
    """Rows [T, heads, D] into a flat view of the pages at the tokens' places; place count + 0 is dropped."""
    if exps is None:
        data = rows.to(pages.dtype)
    else:
        data, e = _quantise(rows)
        data, pages = data.view(torch.uint8), pages.view(torch.uint8)
        flat = torch.cat([exps.reshape(-1), exps.new_zeros(1)])
        flat[at] = e
        exps.copy_(flat[:-1].view_as(exps))
    flat = torch.cat([pages.reshape(-1, D), pages.new_zeros((1, D))])
    flat[at] = data
    pages.copy_(flat[:-1].view_as(pages))


def _append_plain(state):
    c, slots = state["cache"], state["slots"]
    count, heads, page, _ = c["k_pages"].shape
    h = torch.arange(heads, device="cuda")
    at = ((slots // page)[:, None] * heads + h) * page + (slots % page)[:, None]
    at = torch.where((slots < 0)[:, None], count * heads * page, at)
    _store(state["k"], c["k_pages"], c["k_exp"], at)
    _store(state["v"], c["v_pages"], c["v_exp"], at)
    return _written(c)


def _rows(pages, exps, table, tokens):
    """Values [B, S, heads, D] of the tokens [B, S] (indices into each sequence), 0 where no page is held."""
    page, width = pages.shape[2], table.shape[1]
    p = table.long().gather(1, (tokens // page).clamp(max=width - 1))
    held = (p >= 0) & (tokens // page < width)
    at = (p.clamp(min=0), slice(None), tokens % page)
    if exps is None:
        x = pages[at].float()
    else:
        x = _entries(pages.view(torch.uint8)[at].view(pages.dtype), exps[at])
    return x, held


def _gather_plain(state):
    c, lens = state["cache"], state["lens"].long()
    tokens = state["first"].long()[:, None] + torch.arange(state["out_len"], device="cuda")
    outs = []
    for x in "kv":
        r, held = _rows(c[x + "_pages"], c[x + "_exp"], state["table"], tokens)
        r = r.masked_fill(~(held & (tokens < lens[:, None]))[..., None, None], 0.0)
        outs.append(r.transpose(1, 2).to(state["dtype"]).contiguous())
    return tuple(outs)


def _attend_plain(state):
    c, q, lens, cu = state["cache"], state["q"], state["lens"].long(), state["cu"].long()
    heads, page = c["k_pages"].shape[1:3]
    tokens, heads_q, _ = q.shape
    batch, n, group = lens.numel(), state["max_q"], heads_q // heads
    j = torch.arange(state["table"].shape[1] * page, device="cuda")
    k, _ = _rows(c["k_pages"], c["k_exp"], state["table"], j.expand(batch, -1))
    v, held = _rows(c["v_pages"], c["v_exp"], state["table"], j.expand(batch, -1))
    v = v.masked_fill(~(held & (j < lens[:, None]))[..., None, None], 0.0)
    i = torch.arange(n, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=tokens - 1)
    x = q[at].float().view(batch, n, heads, group, D).permute(0, 2, 1, 3, 4).reshape(batch, heads, n * group, D)
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + i
    see = (j <= pos[..., None]) & (j < lens[:, None, None])
    if state["window"]:
        see &= (j > pos[..., None] - state["window"]) | (j < state["sinks"])
    s = torch.matmul(x, k.permute(0, 2, 3, 1)) * state["scale"]
    s = s.view(batch, heads, n, group, -1).masked_fill_(~see[:, None, :, None], float("-inf"))
    s -= s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = s.exp_()
    total = p.sum(-1, keepdim=True)
    p = p.view(batch, heads, n * group, -1)
    o = torch.matmul(p, v.transpose(1, 2)).view(batch, heads, n, group, D)
    o = (o / total.clamp(min=1e-30)).permute(0, 2, 1, 3, 4).reshape(batch, n, heads_q, D)
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    return o[b, t - cu[b]].to(q.dtype)


# ------------------------------------------------------- from the definition

def _two_to(e):
    """2^e in float64 for whole e in [-128, 128], from a table: exact on every device."""
    return torch.tensor([2.0 ** i for i in range(-128, 129)], dtype=torch.float64, device=e.device)[e.long() + 128]


def _e4m3_exact(y):
    """Nearest e4m3 value (ties to even) of float64 values within +-448."""
    _, e = torch.frexp(y)
    step = _two_to((e - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step


def _exact_rows(c, x, table_row, n):
    """Float64 values [n, heads, D] of a sequence's first n tokens; pages given back count as zeros."""
    pages = c[x + "_pages"]
    p = table_row[:-(-n // pages.shape[2])].long()
    r = pages.view(torch.uint8)[p.clamp(min=0)].view(pages.dtype).double() if c["k_exp"] is not None else pages[p.clamp(min=0)].double()
    if c["k_exp"] is not None:
        r = r * _two_to(c[x + "_exp"][p.clamp(min=0)].long() - 127)[..., None]
    r[p < 0] = 0
    return r.transpose(1, 2).reshape(-1, pages.shape[1], D)[:n]


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 2e12:
        return None
    state = prepare(case, seed)
    c = state["cache"]
    page = case["page"]
    if case["op"] == "append":
        out = {}
        ok = state["slots"] >= 0
        p, off = state["slots"][ok] // page, state["slots"][ok] % page
        for x in "kv":
            rows = state[x][ok].double()
            pages = c[x + "_pages"].double()
            if c["k_exp"] is not None:
                top = rows.abs().amax(-1)
                e = torch.ceil(torch.log2(top / 448)).clamp(-32, 64)
                e = torch.where(top > 448 * _two_to(e), e + 1, e)  # the logarithm's own rounding
                e = torch.where((top <= 448 * _two_to(e - 1)) & (e > -32), e - 1, e)
                e = torch.where(top == 0, torch.zeros_like(e), e)
                rows = _e4m3_exact(rows * _two_to(-e)[..., None])
                exps = c[x + "_exp"].clone()
                exps[p, :, off] = (e + 127).to(torch.uint8)
                out[x + "_exp"] = exps
            pages[p, :, off] = rows
            out[x] = pages
        return out
    lens, news = _lengths(case)
    if case["op"] == "gather":
        outs = []
        for x in "kv":
            o = torch.zeros((case["batch"], case["heads"], case["out_len"], D), dtype=torch.float64, device="cuda")
            for b, (n, s) in enumerate(zip(lens, _first(case, lens))):
                r = _exact_rows(c, x, state["table"][b], n)[s:s + case["out_len"]]
                o[b, :, :r.shape[0]] = r.transpose(0, 1)
            outs.append(o)
        return tuple(outs)
    out, t = [], 0
    group = case["heads_q"] // case["heads"]
    for b, (n, m) in enumerate(zip(lens, news)):
        k, v = _exact_rows(c, "k", state["table"][b], n), _exact_rows(c, "v", state["table"][b], n)
        j = torch.arange(n, device="cuda")
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        hide = j > pos
        if case["window"]:
            hide |= (j <= pos - case["window"]) & (j >= case["sinks"])
        o = torch.empty((m, case["heads_q"], D), dtype=torch.float64, device="cuda")
        for h in range(case["heads_q"]):
            s = state["q"][t:t + m, h].double() @ k[:, h // group].T * state["scale"]
            s[hide] = -math.inf
            o[:, h] = torch.softmax(s, -1) @ v[:, h // group]
        out.append(o)
        t += m
    return torch.cat(out)
