"""Attention of trees of drafted tokens over a paged cache, on the GPU against the
64-bit implementation in paged_tree_ref: every output within the derived bound
plus half a step of the output type.  Places that no token sees hold NaN and
infinities, pages that none sees numbers of no page."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_ref as ref  # noqa: E402
import paged_tree_ref as tref  # noqa: E402
import test_paged_exponents_gpu as exponents  # noqa: E402
from test_paged_gpu import TYPES, _clean, _cuda, _poisoned, vq  # noqa: E402,F401

pytestmark = pytest.mark.gpu
D = 128
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


def _tree(kind, n, gen):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "roots":
        return [-1] * n
    if kind == "two":  # two chains side by side
        return [-1 if i < 2 else i - 2 for i in range(n)]
    if kind == "comb":  # a chain with a leaf at every token
        return [-1 if i == 0 else i - 2 if i % 2 == 0 else i - 1 for i in range(n)]
    r = torch.rand(n, generator=gen)
    return [int((i + 1) * float(r[i]) ** 0.5) - 1 for i in range(n)]


def _case(vq, news, lens, Hkv, GQ, PS, dtype, cache, window=0, sinks=0, seed=0, scale=None, kind="any", spread=1.0):  # noqa: F811
    gen = torch.Generator().manual_seed(seed)
    B, T, Hq = len(news), sum(news), Hkv * GQ
    parents, keys = [], []
    for b in range(B):
        up = _tree(kind, news[b], gen)
        parents += up
        keys += tref.tree_keys(up, lens[b] - news[b], news[b], window, sinks)
    cu = np.concatenate([[0], np.cumsum(news)])
    width = max(1, max(-(-n // PS) for n in lens)) + 1
    seen = [torch.cat(keys[cu[b]:cu[b + 1]]).unique() if news[b] else torch.zeros(0, dtype=torch.long) for b in range(B)]
    used = torch.zeros(B, width, dtype=torch.bool)
    for b in range(B):
        used[b, seen[b] // PS] = True
    NP = int(used.sum()) + 3
    table = torch.tensor([-1, -7, NP, 2 ** 30], dtype=torch.int32)[torch.randint(0, 4, (B, width), generator=gen)]
    table[used] = torch.randperm(NP, generator=gen)[:NP - 3].to(torch.int32)
    c = _poisoned(vq, NP, Hkv, PS, cache, gen)
    for b in range(B):
        j = seen[b]
        if len(j) == 0:
            continue
        pg, off = table[b][j // PS].long(), j % PS
        for x in "kv":
            d = torch.randn(len(j), Hkv, D, generator=gen) * spread
            d *= torch.exp2(torch.randint(-3, 4, (len(j), Hkv, 1), generator=gen).float())
            d = (d * (0.5 if x == "k" else 1.0)).to(dtype)
            if cache == E4M3:
                code, e = ref.quantise(d)
                c[x + "_pages"].view(torch.uint8)[pg, :, off] = code
                c[x + "_exp"][pg, :, off] = e
            else:
                c[x + "_pages"][pg, :, off] = d
    i32 = torch.int32
    return dict(q=torch.randn(T, Hq, D, generator=gen).to(dtype), c=c, table=table, cu=torch.tensor(cu, dtype=i32),
                lens=torch.tensor(lens, dtype=i32), parents=torch.tensor(parents, dtype=i32), keys=keys, window=window, sinks=sinks,
                scale=D ** -0.5 if scale is None else scale, max_q=max(1, max(news)))


def _run(vq, a, q=None, **kw):  # noqa: F811
    return vq.vq_paged_attend_tree(a["q"].cuda() if q is None else q, _cuda(a["c"]), a["table"].cuda(), a["cu"].cuda(),
                                   a["lens"].cuda(), a["parents"].cuda(), a["scale"], max_q=a["max_q"], window=a["window"],
                                   sinks=a["sinks"], **kw)


def _check(vq, a, **kw):  # noqa: F811
    got = _run(vq, a, **kw)
    _clean(vq)
    c, dtype = a["c"], a["q"].dtype
    o, bound, _ = tref.attend(a["q"], ref.values(c["k_pages"], c["k_exp"]), ref.values(c["v_pages"], c["v_exp"]), a["table"],
                              a["cu"], a["keys"], a["scale"], ref.U16[F16] if c["k_exp"] is not None else ref.U16[dtype])
    err = (got.cpu().double() - o).abs()
    tol = bound + ref.U16[dtype] * (o.abs() + bound) + 2.0 ** -25
    assert torch.isfinite(got).all()
    assert bool((err <= tol).all()), "largest excess %g, error %g" % (float((err - tol).max()), float(err.max()))
    return got


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("GQ,Hkv,PS", [(1, 2, 16), (4, 2, 16), (8, 1, 32), (3, 2, 64), (16, 1, 128), (2, 1, 256)])
def test_small_trees(vq, dtype, cache, GQ, Hkv, PS):  # noqa: F811
    """At most 16 query rows to a kv head, over caches of nothing but the tree, and of several tiles."""
    n = 16 // GQ
    news = [n, 1, max(1, n - 1), n, n, 0, max(1, n // 2), n, n]
    lens = [n, 1, 77, 128, 129, 9, 300, 127 + n, 2 * n + 1]
    _check(vq, _case(vq, news, lens, Hkv, GQ, PS, dtype, cache, seed=GQ))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("GQ,PS", [(1, 16), (4, 32), (7, 16), (8, 128), (16, 64)])
def test_trees_of_all_sizes_together(vq, dtype, cache, GQ, PS):  # noqa: F811
    news = [40, 1, 0, 3, 129, 64, 5, 33, 2, 250]
    lens = [77, 40, 9, 200, 300, 64, 205, 161, 2, 384]
    _check(vq, _case(vq, news, lens, 1, GQ, PS, dtype, cache, seed=10 + GQ))


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
@pytest.mark.parametrize("kind", ["chain", "roots", "two", "comb"])
@pytest.mark.parametrize("GQ", [1, 5])
def test_kinds_of_trees(vq, dtype, cache, kind, GQ):  # noqa: F811
    news, lens = [16 // GQ, 200, 40, 256, 31], [50, 333, 40, 400, 1000]
    _check(vq, _case(vq, news, lens, 2, GQ, 16, dtype, cache, seed=20 + GQ, kind=kind))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 130), (100, 3), (128, 0), (1000, 7), (3, 2 ** 31 - 1)])
@pytest.mark.parametrize("kind", ["any", "chain"])
def test_window_and_first_tokens(vq, dtype, cache, window, sinks, kind):  # noqa: F811
    """Windows shorter than a path, first tokens that reach into the tree."""
    news, lens = [4, 3, 50, 150, 1, 30, 12], [4, 700, 613, 400, 300, 131, 15]
    _check(vq, _case(vq, news, lens, 1, 4, 16, dtype, cache, window=window, sinks=sinks, seed=window, kind=kind))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("news", [[1, 1, 1], [3, 1, 4], [64, 1, 256]])
def test_chains_are_plain_attention(vq, dtype, cache, news):  # noqa: F811
    """A tree without branches gives what the same tokens give in order, bit for bit."""
    a = _case(vq, news, [2500, 700, 1300], 2, 4, 32, dtype, cache, seed=31, kind="chain")
    got = _run(vq, a)
    want = vq.vq_paged_attend(a["q"].cuda(), _cuda(a["c"]), a["table"].cuda(), a["cu"].cuda(), a["lens"].cuda(), a["scale"],
                              max_q=a["max_q"])
    _clean(vq)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_many_tiles_for_every_block(vq, dtype, cache):  # noqa: F811
    news, lens = [16, 70, 1, 200, 64, 33], [2100, 3300, 900, 2500, 130, 1900]
    _check(vq, _case(vq, news, lens, 8, 4, 128, dtype, cache, seed=36))
    _check(vq, _case(vq, [2] * 40, [1500 + 61 * i for i in range(40)], 8, 4, 64, dtype, cache, seed=37))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("GQ,n", [(4, 5), (4, 32), (4, 33), (16, 8), (1, 128), (7, 18)])
def test_one_query_tile(vq, dtype, cache, GQ, n):  # noqa: F811
    """Rows that fill one query tile, or just not; runs of one key tile, of an even and
    of an odd number, cut ones among them."""
    news = [n, n, max(1, n - 1), n, n, n]
    lens = [n, 128, 129 + n, 300 + n, 2000 + n, 6000 + n]
    _check(vq, _case(vq, news, lens, 2, GQ, 32, dtype, cache, seed=38 + n))
    _check(vq, _case(vq, news, lens, 1, GQ, 16, dtype, cache, seed=39 + n, window=200, sinks=7))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("news", [[20, 7, 32], [50, 64, 20], [3, 4, 1]])
@pytest.mark.parametrize("zeros", [False, True])
def test_rows_of_very_different_sizes_over_codes(vq, dtype, news, zeros):  # noqa: F811
    """Tiles whose exponents lie far apart, zero value rows among them (bounds: as in
    test_paged_exponents_gpu; a chain sees what the same tokens see in order)."""
    def rows(b, gen):
        n = 900 - 100 * b
        k, v = (torch.randn(n, 2, D, generator=gen).double() * torch.exp2(torch.randint(lo, 3, (n, 2, 1), generator=gen)) for lo in (-4, -14))
        k[:, :, 0] *= 0.05
        if zeros:
            v[torch.rand(n, generator=gen) < 0.2] = 0.0
        return k, v
    a = exponents._case(rows, news, 4, 2, 16, dtype, seed=sum(news))
    a["parents"] = torch.tensor([i - 1 for m in news for i in range(m)], dtype=torch.int32)
    c = {k: v.cuda() for k, v in a["c"].items()}
    for x in "kv":
        c[x + "_pages"] = c[x + "_pages"].view(E4M3)
    got = _run(vq, dict(a, c=c))
    _clean(vq)
    o, bound = exponents._reference(a, 2.0 ** -24)
    err = (got.cpu().double() - o).abs()
    tol = bound + ref.U16[dtype] * (o.abs() + bound) + (2.0 ** -25 if dtype == F16 else 0.0)
    assert bool((err <= tol).all()), "error %.2f times the bound" % float((err / tol).nan_to_num(0.0).max())


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_scores_far_apart(vq, dtype, cache):  # noqa: F811
    for scale in (1.5, -0.7, 0.0):
        _check(vq, _case(vq, [4, 20, 140], [513, 300, 140], 1, 4, 16, dtype, cache, seed=41, scale=scale))


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
def test_strided_queries_and_given_buffers(vq, dtype, cache):  # noqa: F811
    a = _case(vq, [1, 9, 200], [50, 60, 300], 2, 3, 16, dtype, cache, seed=51)
    T, Hq, _ = a["q"].shape
    wide = torch.full((T, Hq + 4, 2 * D), float("nan"), dtype=dtype, device="cuda")
    wide[:, 2:Hq + 2, :D] = a["q"].cuda()
    out = torch.full((T, Hq, D), float("nan"), dtype=dtype, device="cuda")
    ws = torch.full((vq.vq_paged_attend_tree_workspace(T, 3, Hq, 2, a["max_q"]),), 255, dtype=torch.uint8, device="cuda")
    got = _check(vq, a, q=wide[:, 2:Hq + 2, :D], out=out, workspace=ws)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, _run(vq, a))


@pytest.mark.parametrize("news", [[4, 3], [40, 64]])
def test_parents_and_lengths_that_make_no_sense_are_reported(vq, news):  # noqa: F811
    """A parent that is not before its token counts as -1; other sequences are as they were."""
    a = _case(vq, news, [100, 130], 1, 4, 16, F16, F16, seed=81, kind="two")
    good = _run(vq, a)
    _clean(vq)
    for bad in (2, 5, -2, 2 ** 31 - 1, -2 ** 31, 256):
        b = dict(a, parents=a["parents"].clone())
        b["parents"][2] = bad
        got = _run(vq, b)
        _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
        assert torch.equal(got[news[0]:], good[news[0]:])
        b["parents"][2] = -1
        assert torch.equal(got, _run(vq, b))
        _clean(vq)
    b = dict(a, lens=torch.tensor([news[0] - 1, 130], dtype=torch.int32))  # a tree longer than its sequence
    got = _run(vq, b)
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
    assert torch.equal(got[news[0]:], good[news[0]:])


def test_more_drafts_than_a_tree_holds(vq):  # noqa: F811
    a = _case(vq, [256], [300], 1, 1, 16, F16, F16, seed=82)
    _check(vq, a)
    with pytest.raises(vq.VQError):
        _run(vq, dict(a, max_q=257))
    b = dict(a, max_q=100)  # fewer than the sequence has: the others are left out
    _run(vq, b)
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)


@pytest.mark.parametrize("news", [[4, 1, 3], [64, 1, 20]])
def test_a_captured_call_follows_its_trees(vq, news):  # noqa: F811
    """Replayed over other trees and lengths, and on another stream."""
    lens = [700, 90, 300]
    a = _case(vq, news, lens, 2, 4, 16, BF16, BF16, seed=91)
    T = sum(news)
    dev = {k: a[k].cuda() for k in ("q", "table", "cu", "lens", "parents")}
    c = _cuda(a["c"])
    out = torch.empty_like(dev["q"])
    ws = torch.empty(vq.vq_paged_attend_tree_workspace(T, 3, 8, 2, a["max_q"]), dtype=torch.uint8, device="cuda")

    def call(**kw):
        return vq.vq_paged_attend_tree(dev["q"], c, dev["table"], dev["cu"], dev["lens"], dev["parents"], a["scale"],
                                       max_q=a["max_q"], **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=out, workspace=ws)
    for i, kind in enumerate(["chain", "roots", "any", "comb"]):
        b = _case(vq, news, [n - 17 * i for n in lens], 2, 4, 16, BF16, BF16, seed=91 + i, kind=kind)
        want = _check(vq, b)
        pad = dict(b["c"])
        for k in ("k_pages", "v_pages"):
            c[k].zero_()
            c[k][:pad[k].shape[0]].copy_(pad[k])
        dev["table"].fill_(-1)
        dev["table"][:, :b["table"].shape[1]].copy_(b["table"])
        for k in ("q", "lens", "parents"):
            dev[k].copy_(b[k])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=s)
    s.synchronize()
    assert torch.equal(got, out)
    _clean(vq)


def test_verify_a_tree_and_keep_the_accepted_path(vq):  # noqa: F811
    """The loop of speculative decoding: drafts appended, attended as a tree, the
    accepted path moved together; a next token then sees what it would see had the
    path been written in order."""
    gen = torch.Generator("cuda").manual_seed(5)
    H, GQ, PS, n, base = 2, 4, 16, 12, [50, 131, 16]
    pages = 16
    up = [-1, 0, 0, 1, 1, 2, 3, 4, 6, 6, 8, 8]
    paths = [[0, 1, 3, 6, 8, 10], [0, 2, 5], []]
    B = len(base)
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(6)).view(B, pages).to(torch.int32).cuda()

    def slots(b, j):
        j = torch.tensor(j, dtype=torch.long, device="cuda")
        return table[b].long()[j // PS] * PS + j % PS

    for cache in (F16, E4M3):
        c = vq.paged_cache(B * pages, H, PS, cache)
        total = sum(base)
        kv = torch.randn(2, total, H, D, generator=gen, device="cuda").half()
        vq.vq_paged_append(kv[0], kv[1], c, torch.cat([slots(b, list(range(m))) for b, m in enumerate(base)]))
        draft = torch.randn(2, B * n, H, D, generator=gen, device="cuda").half()
        ordered = {k: None if x is None else x.clone() for k, x in c.items()}
        vq.vq_paged_append(draft[0], draft[1], c, torch.cat([slots(b, list(range(m, m + n))) for b, m in enumerate(base)]))
        i32 = dict(dtype=torch.int32, device="cuda")
        lens = torch.tensor([m + n for m in base], **i32)
        cu = torch.tensor([n * b for b in range(B + 1)], **i32)
        q = torch.randn(B * n, H * GQ, D, generator=gen, device="cuda").half()
        out = vq.vq_paged_attend_tree(q, c, table, cu, lens, torch.tensor(up * B, **i32), D ** -0.5, max_q=n)
        keep = torch.full((B, 1, n), -1, **i32)
        for b, path in enumerate(paths):
            keep[b, 0, :len(path)] = torch.tensor([base[b] + a for a in path], **i32)
        counts = torch.tensor([len(x) for x in paths], **i32)
        first = torch.tensor(base, **i32)
        vq.vq_paged_compact(c, table, keep, counts, first=first)
        # the same tokens written one after another
        at = torch.cat([slots(b, list(range(base[b], base[b] + len(x)))) for b, x in enumerate(paths)])
        pick = torch.tensor([b * n + a for b, x in enumerate(paths) for a in x], device="cuda")
        vq.vq_paged_append(draft[0][pick], draft[1][pick], ordered, at)
        lens = first + counts
        path_q = torch.cat([q[pick], torch.zeros(0, H * GQ, D, device="cuda").half()])
        cu = torch.tensor(np.cumsum([0] + [len(x) for x in paths]), **i32)
        for cc in (c, ordered):
            got = vq.vq_paged_attend(path_q, cc, table, cu, lens, D ** -0.5, max_q=6)
            # in the tree and in order: the same keys, in sums of another order.  Weights
            # are rounded to fp16 (2^-11) on either side, outputs once more.
            scale = out[pick].float().abs().amax(-1, keepdim=True)
            assert bool(((got.float() - out[pick].float()).abs() <= 4 * 2.0 ** -11 * scale + 2.0 ** -10).all())
        k, v = vq.vq_paged_gather(c, table, lens, 160)
        k2, v2 = vq.vq_paged_gather(ordered, table, lens, 160)
        assert torch.equal(k, k2) and torch.equal(v, v2)
    _clean(vq)


def test_more_trees_than_a_block_has_threads(vq):  # noqa: F811
    news = [17 + i % 5 if i % 9 else 40 for i in range(1100)]
    news[3::50] = [1] * len(news[3::50])
    _check(vq, _case(vq, news, [n + i % 37 for i, n in enumerate(news)], 1, 1, 16, F16, F16, seed=56))
    _check(vq, _case(vq, [1 + i % 4 for i in range(1300)], [5 + i % 60 for i in range(1300)], 1, 4, 16, F16, F16, seed=57))
