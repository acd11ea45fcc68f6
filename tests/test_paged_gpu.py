"""Paged-cache operators (append, gather, attend) on the GPU against the plain
64-bit implementation in tests/paged_ref.py.

Writing and reading back are compared bit for bit.  Attention: every output
within the bound that paged_ref.attend derives (rounding of the weights to the
16-bit operand type, 32-bit scores and sums) plus half a step of the output
type.  Places that no token sees are filled with NaN and infinities, page
tables with numbers of no page.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
D = 128
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def vq():
    from kv_cache_quantization_turboquantrvq_gb300 import api, build
    build.build()
    api.lib()
    return api


def _clean(vq, code=0):
    torch.cuda.synchronize()
    assert vq.vq_device_error() == code


def _poisoned(vq, NP, H, PS, dtype, gen):
    """A pool whose every place holds NaN, infinities or the largest codes."""
    c = vq.paged_cache(NP, H, PS, dtype, device="cpu")
    for x in "kv":
        if dtype == E4M3:
            bad = torch.tensor([0x7F, 0xFF, 0x7E, 0xFE], dtype=torch.uint8)
            c[x + "_pages"] = bad[torch.randint(0, 4, (NP, H, PS, D), generator=gen)].view(E4M3)
            c[x + "_exp"] = torch.tensor([255, 0, 254], dtype=torch.uint8)[torch.randint(0, 3, (NP, H, PS), generator=gen)]
        else:
            bad = torch.tensor([float("nan"), float("inf"), float("-inf"), torch.finfo(dtype).min], dtype=dtype)
            c[x + "_pages"] = bad[torch.randint(0, 4, (NP, H, PS, D), generator=gen)]
    return c


def _cuda(c):
    return {k: None if v is None else v.cuda() for k, v in c.items()}


def _case(vq, news, lens, Hkv, GQ, PS, dtype, cache, window=0, sinks=0, seed=0, scale=None, spread=1.0):
    """Tensors of an attention call on the CPU; the visible tokens' places hold
    data, everything else is poisoned and pages that nothing sees are not held."""
    gen = torch.Generator().manual_seed(seed)
    B, T, Hq = len(news), sum(news), Hkv * GQ
    width = max(1, max(-(-n // PS) for n in lens)) + 1
    used = [[False] * width for _ in range(B)]
    seen = []
    for b in range(B):
        s = set()
        for i in range(news[b]):
            p = lens[b] - news[b] + i
            lo = max(0, p - window + 1) if window else 0
            s.update(range(lo, p + 1))
            if window:
                s.update(range(0, min(sinks, p + 1)))
        s = np.array(sorted(s), dtype=np.int64)
        seen.append(s)
        for pg in set((s // PS).tolist()):
            used[b][pg] = True
    count = sum(map(sum, used))
    NP = count + 3
    perm = torch.randperm(NP, generator=gen)[:count].to(torch.int32)
    table = torch.tensor([-1, -7, NP, 2 ** 30], dtype=torch.int32)[torch.randint(0, 4, (B, width), generator=gen)]
    table[torch.tensor(used)] = perm
    c = _poisoned(vq, NP, Hkv, PS, cache, gen)
    for b in range(B):
        if len(seen[b]) == 0:
            continue
        j = torch.from_numpy(seen[b])
        pg, off = table[b][j // PS].long(), j % PS
        for x in "kv":
            d = torch.randn(len(j), Hkv, D, generator=gen) * spread
            d *= torch.exp2(torch.randint(-3, 4, (len(j), Hkv, 1), generator=gen).float())  # rows of different size
            if x == "k":
                d *= 0.5
            d = d.to(dtype)
            if cache == E4M3:
                code, e = ref.quantise(d)
                c[x + "_pages"].view(torch.uint8)[pg, :, off] = code
                c[x + "_exp"][pg, :, off] = e
            else:
                c[x + "_pages"][pg, :, off] = d
    q = torch.randn(T, Hq, D, generator=gen).to(dtype)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32)
    return dict(q=q, c=c, table=table, cu=cu, lens=torch.tensor(lens, dtype=torch.int32), window=window, sinks=sinks,
                scale=D ** -0.5 if scale is None else scale, max_q=max(1, max(news)))


def _run(vq, a, q=None, **kw):
    q = a["q"].cuda() if q is None else q
    return vq.vq_paged_attend(q, _cuda(a["c"]), a["table"].cuda(), a["cu"].cuda(), a["lens"].cuda(), a["scale"],
                              max_q=a["max_q"], window=a["window"], sinks=a["sinks"], **kw)


def _reference(a):
    dtype = a["q"].dtype
    c = a["c"]
    step = ref.U16[F16] if c["k_exp"] is not None else ref.U16[dtype]
    return ref.attend(a["q"], ref.values(c["k_pages"], c["k_exp"]), ref.values(c["v_pages"], c["v_exp"]), a["table"],
                      a["cu"], a["lens"], a["scale"], a["window"], a["sinks"], step)


def _check(vq, a, **kw):
    got = _run(vq, a, **kw)
    _clean(vq)
    o, bound = _reference(a)
    err = (got.cpu().double() - o).abs()
    tol = bound + ref.U16[a["q"].dtype] * (o.abs() + bound) + 2.0 ** -25
    assert torch.isfinite(got).all()
    assert bool((err <= tol).all()), "largest excess %g, error %g" % (float((err - tol).max()), float(err.max()))
    return got


TYPES = [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)]


# ---------------------------------------------------------------- the cache

@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("PS,H,T", [(16, 1, 1), (16, 3, 37), (64, 8, 130), (256, 2, 19)])
def test_append_writes_the_slots_and_nothing_else(vq, dtype, cache, PS, H, T):
    gen = torch.Generator().manual_seed(T + PS)
    NP = T // PS + 5
    c = vq.paged_cache(NP, H, PS, cache, device="cpu")
    for x in "kv":
        if cache == E4M3:
            c[x + "_pages"] = torch.randint(0, 256, (NP, H, PS, D), generator=gen, dtype=torch.uint8).view(E4M3)
            c[x + "_exp"] = torch.randint(0, 256, (NP, H, PS), generator=gen, dtype=torch.uint8)
        else:
            c[x + "_pages"] = torch.randn(NP, H, PS, D, generator=gen).to(dtype)
    # strided views: tokens of a fused projection, heads further apart than their width
    wide = torch.randn(T, H, 3 * D, generator=gen) * torch.exp2(torch.randint(-30, 8, (T, H, 1), generator=gen).float())
    wide[::7, 0] = 0.0                      # zero rows
    wide[1::5, -1, ::9] = 2.0 ** -24        # fp16's least
    wide = wide.to(dtype)
    slots = torch.randperm(NP * PS, generator=gen)[:T]
    slots[3::11] = -1
    if T > 8:
        slots[8] = -(2 ** 40)
    g = _cuda(c)
    w = wide.cuda()
    vq.vq_paged_append(w[:, :, :D], w[:, :, 2 * D:], g, slots.cuda())
    _clean(vq)
    for x, rows in (("k", wide[:, :, :D]), ("v", wide[:, :, 2 * D:])):
        want = c[x + "_pages"].view(torch.uint8 if cache == E4M3 else torch.int16).clone()
        we = None if cache != E4M3 else c[x + "_exp"].clone()
        if cache == E4M3:
            code, e = ref.quantise(rows)
        for t in range(T):
            s = int(slots[t])
            if s < 0:
                continue
            want[s // PS, :, s % PS] = code[t] if cache == E4M3 else rows[t].contiguous().view(torch.int16)
            if cache == E4M3:
                we[s // PS, :, s % PS] = e[t]
        assert torch.equal(g[x + "_pages"].cpu().view(want.dtype), want)
        if cache == E4M3:
            assert torch.equal(g[x + "_exp"].cpu(), we)


def test_append_e4m3_every_rounding(vq):
    """Every finite bf16 and fp16 magnitude class against the codes' definition:
    rows made of one large value that fixes the exponent and values over the
    whole range, ties among them; the largest values saturate."""
    for dtype in (F16, BF16):
        bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16)
        x = bits.view(dtype)
        x = x[torch.isfinite(x)]
        if dtype == BF16:
            x = x[x.abs() <= 2.0 ** 100]
        x = torch.cat([x, x[: -len(x) % 127]]) if len(x) % 127 else x
        rows = torch.cat([x.view(-1, 127), torch.zeros(len(x) // 127, 1, dtype=dtype)], 1)
        rows = torch.cat([rows, rows.flip(0).roll(1, 1)])
        rows[:, 127] = rows.float().abs().max(1).values.to(dtype)
        T = rows.shape[0]
        c = vq.paged_cache(T // 16 + 1, 1, 16, E4M3)
        r = rows.view(T, 1, D).cuda()
        vq.vq_paged_append(r, r, c, torch.arange(T).cuda())
        _clean(vq)
        code, e = ref.quantise(rows)
        got = c["k_pages"].cpu().view(torch.uint8).reshape(-1, D)[:T]
        assert torch.equal(c["k_exp"].cpu().reshape(-1)[:T], e)
        assert torch.equal(ref_values(got), ref_values(code))


def ref_values(code):
    return torch.from_numpy(ref.E4M3)[code.long()]


def test_append_slot_past_the_pool_is_reported(vq):
    c = vq.paged_cache(2, 1, 16, F16)
    x = torch.ones(3, 1, D, dtype=F16, device="cuda")
    vq.vq_paged_append(x, x, c, torch.tensor([5, 32, 2 ** 40], device="cuda"))
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
    assert int((c["k_pages"] != 0).sum()) == D
    _clean(vq)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("PS,H,S", [(16, 2, 1), (32, 3, 77), (128, 1, 200)])
def test_gather_reads_back(vq, dtype, cache, PS, H, S):
    lens = [0, 1, S, S + 40, 3 * PS, 5 * PS - 1]
    first = [0, 0, 0, 37, 2 * PS + 3, -2]
    gen = torch.Generator().manual_seed(PS + S)
    B, width = len(lens), -(-max(lens) // PS) + 1
    need = torch.tensor([[p * PS < n for p in range(width)] for n in lens])
    count = int(need.sum())
    c = _poisoned(vq, count + 2, H, PS, cache, gen)
    table = torch.full((B, width), 2 ** 30, dtype=torch.int32)
    table[need] = torch.randperm(count + 2, generator=gen)[:count].to(torch.int32)
    for b, n in enumerate(lens):
        j = torch.arange(n)
        if n == 0:
            continue
        pg, off = table[b][j // PS].long(), j % PS
        for x in "kv":
            d = (torch.randn(n, H, D, generator=gen) * 3).to(dtype)
            if cache == E4M3:
                code, e = ref.quantise(d)
                c[x + "_pages"].view(torch.uint8)[pg, :, off] = code
                c[x + "_exp"][pg, :, off] = e
            else:
                c[x + "_pages"][pg, :, off] = d
    k, v = vq.vq_paged_gather(_cuda(c), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), S,
                              first=torch.tensor(first, dtype=torch.int32).cuda(), dtype=dtype)
    only_v = vq.vq_paged_gather(_cuda(c), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), S,
                                dtype=dtype, want_k=False)
    _clean(vq)
    assert only_v[0] is None and only_v[1].shape == (B, H, S, D)
    for x, got in (("k", k), ("v", v)):
        val = ref.values(c[x + "_pages"], c[x + "_exp"])
        want = torch.zeros(B, H, S, D, dtype=torch.float64)
        for b in range(B):
            for i in range(S):
                t = first[b] + i
                if 0 <= t < lens[b]:
                    want[b, :, i] = val[table[b][t // PS].long(), :, t % PS]
        assert torch.equal(got.cpu(), want.to(dtype))


def test_gather_of_a_missing_page_is_reported(vq):
    c = vq.paged_cache(2, 1, 16, F16)
    c["k_pages"].fill_(1)
    t = torch.tensor([[1, -1, 5]], dtype=torch.int32, device="cuda")
    k, _ = vq.vq_paged_gather(c, t, torch.tensor([80], dtype=torch.int32, device="cuda"), 80)
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
    assert int((k != 0).sum()) == 16 * D


# ------------------------------------------------------------ the attention

@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("GQ,Hkv,PS", [(1, 2, 16), (4, 2, 16), (8, 1, 32), (3, 2, 64), (16, 1, 128), (5, 1, 256)])
def test_decode(vq, dtype, cache, GQ, Hkv, PS):
    """Single tokens: lengths from none to several tiles."""
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 300]
    _check(vq, _case(vq, [1] * len(lens), lens, Hkv, GQ, PS, dtype, cache, seed=GQ))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("GQ,PS", [(1, 16), (4, 32), (7, 16), (8, 128), (2, 256)])
def test_chunks_and_single_tokens_together(vq, dtype, cache, GQ, PS):
    """Chunks of any length, single tokens, sequences without a new token, and
    more new tokens than the cache holds (the first see nothing)."""
    news = [1, 40, 0, 3, 129, 1, 70, 5]
    lens = [77, 40, 9, 200, 300, 1, 20, 5]
    a = _case(vq, news, lens, 1, GQ, PS, dtype, cache, seed=10 + GQ)
    got = _check(vq, a)
    t = int(a["cu"][6])
    assert bool((got[t:t + 50] == 0).all())  # positions before the sequence's first token


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 130), (100, 3), (128, 0), (1000, 7)])
def test_window_and_first_tokens(vq, dtype, cache, window, sinks):
    news = [1, 1, 50, 150, 2, 1]
    lens = [1, 700, 613, 400, 131, 300]
    _check(vq, _case(vq, news, lens, 1, 4, 16, dtype, cache, window=window, sinks=sinks, seed=window + sinks))


def test_window_longer_than_anything(vq):
    """The largest window and number of first tokens there can be: as without."""
    a = _case(vq, [1, 40, 3], [200, 90, 1], 1, 4, 16, F16, F16, seed=37)
    plain = _run(vq, a)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1), (400, 0)):
        assert torch.equal(_run(vq, dict(a, window=window, sinks=sinks)), plain)
    _clean(vq)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_one_long_sequence_is_split_and_joined(vq, dtype, cache):
    """One sequence over every CTA, single token and chunk, with and without
    window (71, 80 and 119 parts to join)."""
    _check(vq, _case(vq, [1], [9001], 1, 4, 64, dtype, cache, seed=31))
    _check(vq, _case(vq, [3], [5003], 2, 5, 16, dtype, cache, seed=32))
    _check(vq, _case(vq, [1], [20000], 1, 8, 128, dtype, cache, window=15000, sinks=4, seed=33))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("GQ", [2, 12])
def test_many_tiles_for_every_block(vq, dtype, cache, GQ):
    """Single tokens with far more key tiles than blocks: the rings of copies
    come round many times, across items (8 and 16 row forms)."""
    news, lens = [1] * 40, [1500 + 61 * i for i in range(40)]
    _check(vq, _case(vq, news, lens, 8 if GQ == 2 else 4, GQ, 64, dtype, cache, seed=35))


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_many_chunk_tiles_for_every_block(vq, dtype, cache):
    """Chunks with several items and many tiles for every block, among them
    items of one query tile and of two."""
    news, lens = [33, 70, 1, 200, 130, 64], [2100, 3000, 900, 2500, 130, 1900]
    _check(vq, _case(vq, news, lens, 8, 4, 128, dtype, cache, seed=36))


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_scores_far_apart(vq, dtype, cache):
    """Large scores (one key takes nearly all weight, the maximum moves often), a
    negative scale, and scale 0 (plain means)."""
    for scale in (1.5, -0.7, 0.0):
        _check(vq, _case(vq, [1, 20, 140], [513, 300, 140], 1, 4, 16, dtype, cache, seed=41, scale=scale))


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
def test_strided_queries_and_given_buffers(vq, dtype, cache):
    a = _case(vq, [1, 9, 200], [50, 60, 300], 2, 3, 16, dtype, cache, seed=51)
    T, Hq, _ = a["q"].shape
    wide = torch.full((T, Hq + 4, 2 * D), float("nan"), dtype=dtype, device="cuda")
    wide[:, 2:Hq + 2, :D] = a["q"].cuda()
    out = torch.full((T, Hq, D), float("nan"), dtype=dtype, device="cuda")
    ws = torch.full((vq.vq_paged_attend_workspace(T, 3, Hq, 2, a["max_q"]),), 255, dtype=torch.uint8, device="cuda")
    got = _check(vq, a, q=wide[:, 2:Hq + 2, :D], out=out, workspace=ws)
    assert got.data_ptr() == out.data_ptr()
    plain = _run(vq, a)
    assert torch.equal(got, plain)


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
def test_output_at_any_16_bytes(vq, dtype, cache):
    """An output that starts 16 bytes past a multiple of 32, items whole and cut."""
    a = _case(vq, [1, 40, 200, 77], [50, 40, 3000, 77], 2, 4, 32, dtype, cache, seed=52)
    T, Hq, _ = a["q"].shape
    room = torch.full((T * Hq * D + 16,), float("nan"), dtype=dtype, device="cuda")
    out = room[8:8 + T * Hq * D].view(T, Hq, D)
    assert out.data_ptr() % 32 == 16
    got = _check(vq, a, out=out)
    assert torch.equal(got, _run(vq, a))
    assert bool(room[:8].isnan().all()) and bool(room[8 + T * Hq * D:].isnan().all())


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_query_rows_of_any_size_over_codes(vq, dtype):
    """Rows from 2^-60 (fp16: 2^-10) to 1, rows of zeros, and rows with entries far
    below their largest, for single tokens and chunks of several items."""
    a = _case(vq, [1, 50, 140, 1], [300, 50, 700, 129], 2, 4, 16, dtype, E4M3, seed=53)
    gen = torch.Generator().manual_seed(54)
    T, Hq, _ = a["q"].shape
    low = -60 if dtype == BF16 else -10
    size = torch.exp2(torch.randint(low, 1, (T, Hq, 1), generator=gen).float())
    size[torch.rand(T, Hq, 1, generator=gen) < 0.1] = 0.0
    inner = torch.exp2(torch.randint(-30, 1, (T, Hq, D), generator=gen).float())
    inner[: T // 2] = 1.0
    a["q"] = (a["q"].float() * size * inner).to(dtype)
    _check(vq, a)


def test_more_entries_than_the_plan_keeps_at_hand(vq):
    """More than a thousand chunks, of one query tile and of two, beside single
    tokens: the plan reads entries back from memory."""
    news = [17 + i % 5 if i % 9 else 150 for i in range(1100)]
    news[3::50] = [1] * len(news[3::50])
    lens = [n + i % 37 for i, n in enumerate(news)]
    _check(vq, _case(vq, news, lens, 1, 1, 16, F16, F16, seed=55))


def test_repeated_calls_agree_bit_for_bit(vq):
    a = _case(vq, [1, 130, 33], [4000, 700, 2000], 2, 4, 32, BF16, BF16, seed=61)
    first = _run(vq, a)
    for _ in range(5):
        assert torch.equal(_run(vq, a), first)
    _clean(vq)


def test_side_stream_and_graph(vq):
    """A call on another stream, and a captured one whose lengths and queries
    change between replays."""
    a = _case(vq, [1, 1, 1], [700, 90, 300], 2, 4, 16, F16, F16, seed=71)
    want = _run(vq, a)
    s = torch.cuda.Stream()
    dev = dict(q=a["q"].cuda(), c=_cuda(a["c"]), table=a["table"].cuda(), cu=a["cu"].cuda(), lens=a["lens"].cuda())
    torch.cuda.synchronize()
    got = vq.vq_paged_attend(dev["q"], dev["c"], dev["table"], dev["cu"], dev["lens"], a["scale"], max_q=1, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    ws = torch.empty(vq.vq_paged_attend_workspace(3, 3, 8, 2, 1), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vq.vq_paged_attend(dev["q"], dev["c"], dev["table"], dev["cu"], dev["lens"], a["scale"], max_q=1, out=out,
                           workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    short = dict(a, lens=torch.tensor([650, 90, 17], dtype=torch.int32))
    dev["lens"].copy_(short["lens"])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _run(vq, short))
    _clean(vq)


def test_a_missing_visible_page_and_too_many_tokens_are_reported(vq):
    a = _case(vq, [1, 1], [100, 40], 1, 4, 16, F16, F16, seed=81)
    keep = a["table"].clone()
    a["table"][0, 2] = -1
    got = _run(vq, a)
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
    a["table"] = keep
    ok = _run(vq, a)
    _clean(vq)
    assert torch.equal(got[1], ok[1])
    b = _case(vq, [5, 1], [100, 40], 1, 4, 16, F16, F16, seed=82)
    b["max_q"] = 2
    _run(vq, b)
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
    # numbers of tokens that make no sense stay inside the buffers
    b["cu"] = torch.tensor([0, 1000, -5], dtype=torch.int32)
    b["max_q"] = 6
    _run(vq, b)
    torch.cuda.synchronize()
    vq.vq_device_error()


def test_fp16_over_long_context_keeps_its_precision(vq):
    """Equal scores over many keys: every weight counts, none may vanish."""
    a = _case(vq, [1], [30000], 1, 1, 128, F16, F16, seed=91, scale=0.0)
    _check(vq, a)


# ------------------------------------------------------------- used together

@pytest.mark.parametrize("cache,window,limit", [("float16", 0, 0.01), ("float16", 100, 0.01), ("e4m3", 0, 0.06), ("e4m3", 100, 0.06)])
def test_the_example_serves_and_compresses(vq, cache, window, limit):
    """examples/serve_paged.py: prompts in chunks and decodes in one batch, pages
    given back behind a window, blocks read back for the codecs.  Against plain
    attention over the uncompressed fp16 keys and values: the fp16 cache adds the
    weights' and outputs' rounding (2^-11 each; 0.01 leaves room for the plain
    side's 32-bit sums), e4m3 entries are off by 2^-4 at most and 2^-4 / sqrt(3)
    in the mean, of keys (which move a weight by their score's error, about
    2^-4 / sqrt(3) / sqrt(3) of a unit score) and values, averaged over the keys
    that carry the weight: below the 0.06 of a single entry."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import serve_paged
    got, want, pages, done = serve_paged.serve(prompts=(300, 177, 512, 130), steps=8, cache=cache, window=window, seed=3)
    off = float((got - want).norm() / want.norm())
    assert off < limit, off
    if window:
        held = sum(p >= 0 for r in pages.table for p in r)
        assert held <= 4 * (1 + 100 // 16 + 2)
    else:
        kivi, rvq, tokens = serve_paged.compress(pages, done)
        assert tokens == 128
        k, v = vq.vq_kivi_unpack_dequant(kivi, 4, 8, 128, 2, 32)
        c1, _, c2, _ = vq.vq_rvq_codebook(D, 2)
        kr = vq.vq_rvq_unpack_dequant(*rvq, 2, c1, c2)
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        k0, v0 = vq.vq_paged_gather(pages.cache, pages.device_table(), lens, 128, dtype=F16)
        for a, b in ((k, k0), (v, v0), (kr, k0)):
            assert float((a.float() - b.float()).norm() / b.float().norm()) < 0.6  # 2-bit codes
    _clean(vq)
