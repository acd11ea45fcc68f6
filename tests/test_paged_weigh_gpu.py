"""Attention over a paged cache that adds up the softmax weight of every cached
token, on the GPU against 64-bit sums: the outputs are those of the plain call,
bit for bit; the weights lie within a bound that is derived below; the places of
tokens that nothing sees keep their bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_ref as ref  # noqa: E402
import paged_tree_ref as tref  # noqa: E402
from test_paged_gpu import TYPES, _case, _clean, _cuda, vq  # noqa: E402,F401

pytestmark = pytest.mark.gpu
D = 128
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


def _keys(lens, news, window, sinks):
    out = []
    for n, m in zip(lens, news):
        for i in range(m):
            p = n - m + i
            j = torch.arange(max(p + 1, 0))
            out.append(j[(j > p - window) | (j < sinks)] if window else j)
    return out


def _reference(a, w, observe, decay):
    """(weights, bound, which places are updated) in 64 bits.

    A weight 2^(s - lse) is off by what its score and the row's lse are off: the
    score's sum of 128 products and its scaling by d = 140 * 2^-24 * scale * sum |q k|
    (in units of 1, as paged_ref.attend counts it; the rounding of s and of
    s - lse is less), lse by the mean of that, by n keys' sums (n^0.5 2^-22 there) and
    by one rounding of log2; the exponential adds 2^-20.  The sum over rows rounds
    by 2^-24 a row, the update twice."""
    c = a["c"]
    k, v = ref.values(c["k_pages"], c["k_exp"]), ref.values(c["v_pages"], c["v_exp"])
    PS, H = k.shape[2], k.shape[1]
    cu, lens, table = a["cu"].tolist(), a["lens"].tolist(), a["table"].long()
    news = [y - x for x, y in zip(cu, cu[1:])]
    keys = _keys(lens, news, a["window"], a["sinks"])
    _, _, soft = tref.attend(a["q"], k, v, a["table"], a["cu"], keys, a["scale"], 0.0)
    out, bound, hit = w.double().clone(), torch.zeros(w.shape, dtype=torch.float64), torch.zeros(w.shape, dtype=torch.bool)
    for b, (n, m) in enumerate(zip(lens, news)):
        if m == 0:
            continue
        add, off = torch.zeros(max(n, 1), H, dtype=torch.float64), torch.zeros(max(n, 1), H, dtype=torch.float64)
        seen = torch.zeros(max(n, 1), dtype=torch.bool)
        rows = 0
        for i in range(m):
            t = cu[b] + i
            j = keys[t]
            seen[j] = True
            if (observe and i < m - observe) or len(j) == 0:
                continue
            pg = table[b][j // PS]
            kh = k[pg, :, j % PS].transpose(0, 1)
            qt = a["q"][t].double().view(H, -1, D).transpose(1, 2)
            d = 2.0 ** -24 * 140 * (kh.abs() @ qt.abs()).amax(1) * abs(a["scale"])  # [H, G]
            rel = 2 * torch.expm1(d) + len(j) ** 0.5 * 2.0 ** -22 + 2.0 ** -19
            add[j] += soft[t].sum(1).T
            off[j] += (soft[t] * rel[..., None]).sum(1).T
            rows += soft[t].shape[1]
        j = seen.nonzero()[:, 0]
        at = (table[b][j // PS], slice(None), j % PS)
        old = torch.where((j >= n - m)[:, None] | torch.tensor(decay == 0.0), torch.zeros(len(j), H, dtype=torch.float64), decay * w.double()[at])
        out[at] = old + add[j]
        bound[at] = off[j] + add[j] * rows * 2.0 ** -24 + 2.0 ** -23 * (old.abs() + add[j]) + 1e-30
        hit[at] = True
    return out, bound, hit


def _weights(a, seed, decay):
    """Numbers everywhere; NaN and infinities where they must not be asked for."""
    gen = torch.Generator().manual_seed(seed)
    c = a["c"]["k_pages"]
    w = torch.rand(c.shape[:3], generator=gen) * 3
    PS = c.shape[2]
    cu, lens = a["cu"].tolist(), a["lens"].tolist()
    bad = torch.tensor([float("nan"), float("inf"), -1.0])
    for b, n in enumerate(lens):
        m = cu[b + 1] - cu[b]
        j = torch.arange(0 if decay == 0.0 else max(n - m, 0), n)
        pg = a["table"][b].long()[j // PS]
        ok = (pg >= 0) & (pg < c.shape[0])
        w[pg[ok], :, (j % PS)[ok]] = bad[torch.randint(0, 3, (int(ok.sum()), c.shape[1]), generator=gen)]
    return w


def _run(vq, a, w, observe, decay, q=None, **kw):  # noqa: F811
    return vq.vq_paged_attend_weigh(a["q"].cuda() if q is None else q, _cuda(a["c"]), w, a["table"].cuda(), a["cu"].cuda(),
                                    a["lens"].cuda(), a["scale"], max_q=a["max_q"], window=a["window"], sinks=a["sinks"],
                                    observe=observe, decay=decay, **kw)


def _check(vq, a, observe=0, decay=1.0, seed=0, **kw):  # noqa: F811
    w = _weights(a, seed, decay)
    g = w.cuda()
    out = _run(vq, a, g, observe, decay, **kw)
    plain = vq.vq_paged_attend(a["q"].cuda(), _cuda(a["c"]), a["table"].cuda(), a["cu"].cuda(), a["lens"].cuda(), a["scale"],
                               max_q=a["max_q"], window=a["window"], sinks=a["sinks"])
    _clean(vq)
    assert torch.equal(out, plain)
    want, bound, hit = _reference(a, w, observe, decay)
    got = g.cpu()
    assert torch.equal(got.view(torch.int32)[~hit], w.view(torch.int32)[~hit])
    err = (got.double() - want).abs()[hit]
    assert torch.isfinite(got[hit]).all()
    assert bool((err <= bound[hit]).all()), "largest excess %g, error %g" % (float((err - bound[hit]).max()), float(err.max()))
    return got


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("GQ,Hkv,PS", [(1, 2, 16), (4, 2, 16), (8, 1, 32), (3, 2, 64), (16, 1, 128), (5, 1, 256)])
def test_decode(vq, dtype, cache, GQ, Hkv, PS):  # noqa: F811
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 300, 1500]
    _check(vq, _case(vq, [1] * len(lens), lens, Hkv, GQ, PS, dtype, cache, seed=GQ), decay=0.97)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("GQ,PS", [(1, 16), (4, 32), (7, 16), (8, 128), (2, 256), (15, 64)])
@pytest.mark.parametrize("observe,decay", [(0, 1.0), (32, 0.5), (1, 0.0)])
def test_chunks_and_single_tokens_together(vq, dtype, cache, GQ, PS, observe, decay):  # noqa: F811
    """Chunks of any length, single tokens, sequences without a new token, and more
    new tokens than the cache holds."""
    news = [1, 40, 0, 3, 129, 1, 70, 5]
    lens = [77, 40, 9, 200, 300, 1, 20, 5]
    _check(vq, _case(vq, news, lens, 1, GQ, PS, dtype, cache, seed=10 + GQ), observe, decay)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 130), (100, 3), (128, 0), (1000, 7), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("observe", [0, 20])
def test_window_and_first_tokens(vq, dtype, cache, window, sinks, observe):  # noqa: F811
    news = [1, 1, 50, 150, 2, 1]
    lens = [1, 700, 613, 400, 131, 300]
    _check(vq, _case(vq, news, lens, 1, 4, 16, dtype, cache, window=window, sinks=sinks, seed=window % 1000 + sinks % 1000), observe,
           decay=0.9)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_long_sequences_and_many_units(vq, dtype, cache):  # noqa: F811
    """Sequences over every block, single token and chunk; more units than blocks,
    chunks cut into several parts."""
    _check(vq, _case(vq, [1], [9001], 1, 4, 64, dtype, cache, seed=31))
    _check(vq, _case(vq, [3], [5003], 2, 5, 16, dtype, cache, seed=32), decay=0.5)
    _check(vq, _case(vq, [1] * 40, [1500 + 61 * i for i in range(40)], 4, 2, 64, dtype, cache, seed=33))
    _check(vq, _case(vq, [600, 1, 350], [1600, 900, 351], 4, 4, 128, dtype, cache, seed=34))
    _check(vq, _case(vq, [1200], [1200], 1, 4, 32, dtype, cache, seed=35), observe=700)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_scores_far_apart(vq, dtype, cache):  # noqa: F811
    for scale in (1.5, -0.7, 0.0):
        _check(vq, _case(vq, [1, 20, 140], [513, 300, 140], 1, 4, 16, dtype, cache, seed=41, scale=scale))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_value_exponents_do_not_count(vq, dtype):  # noqa: F811
    """Over codes: values of very different sizes, zero rows among them, leave the
    weights of their tokens as they are."""
    a = _case(vq, [1, 50, 140], [300, 50, 700], 2, 4, 16, dtype, E4M3, seed=43)
    gen = torch.Generator().manual_seed(44)
    e = a["c"]["v_exp"]
    ok = (e > 100) & (e < 140)
    e[ok] = torch.randint(97, 150, (int(ok.sum()),), generator=gen, dtype=torch.uint8)
    _check(vq, a)


def test_strided_queries_padding_rows_and_given_buffers(vq):  # noqa: F811
    """Query rows of no sequence hold NaN; buffers are given, with NaN in them."""
    for dtype, cache in [(F16, F16), (BF16, E4M3)]:
        a = _case(vq, [1, 9, 200], [50, 60, 300], 2, 3, 16, dtype, cache, seed=51)
        T, Hq, _ = a["q"].shape
        wide = torch.full((T + 70, Hq + 4, 2 * D), float("nan"), dtype=dtype, device="cuda")
        wide[:T, 2:Hq + 2, :D] = a["q"].cuda()
        w = _weights(a, 1, 1.0)
        g, g2 = w.cuda(), w.cuda()
        ws = torch.full((vq.vq_paged_attend_weigh_workspace(T + 70, 3, Hq, 2, a["max_q"], a["table"].shape[1], 16),), 255,
                        dtype=torch.uint8, device="cuda")
        out = torch.full((T + 70, Hq, D), 7.0, dtype=dtype, device="cuda")
        got = _run(vq, a, g, 0, 1.0, q=wide[:, 2:Hq + 2, :D], out=out, workspace=ws)
        plain = _run(vq, a, g2, 0, 1.0)
        _clean(vq)
        assert got.data_ptr() == out.data_ptr() and torch.equal(got[:T], plain) and bool((got[T:] == 7.0).all())
        assert torch.equal(g.view(torch.int32), g2.view(torch.int32))


def test_repeated_calls_agree_bit_for_bit(vq):  # noqa: F811
    a = _case(vq, [1, 330, 33], [4000, 700, 2000], 2, 4, 32, BF16, BF16, seed=61)
    w = _weights(a, 2, 1.0)
    first = w.cuda()
    _run(vq, a, first, 0, 1.0)
    for _ in range(5):
        g = w.cuda()
        _run(vq, a, g, 0, 1.0)
        assert torch.equal(g.view(torch.int32), first.view(torch.int32))
    _clean(vq)


@pytest.mark.parametrize("news", [[1, 1, 1], [1, 200, 40]])
def test_side_stream_and_graph(vq, news):  # noqa: F811
    """Captured; replayed over other lengths and queries, weights adding up from replay to replay."""
    a = _case(vq, news, [700, 390, 300], 2, 4, 16, F16, F16, seed=71)
    T = sum(news)
    dev = dict(q=a["q"].cuda(), c=_cuda(a["c"]), table=a["table"].cuda(), cu=a["cu"].cuda(), lens=a["lens"].cuda())
    w = torch.zeros(a["c"]["k_pages"].shape[:3], device="cuda")
    out = torch.empty_like(dev["q"])
    ws = torch.empty(vq.vq_paged_attend_weigh_workspace(T, 3, 8, 2, a["max_q"], a["table"].shape[1], 16), dtype=torch.uint8, device="cuda")

    def call(to, **kw):
        return vq.vq_paged_attend_weigh(dev["q"], dev["c"], to, dev["table"], dev["cu"], dev["lens"], a["scale"], max_q=a["max_q"], **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(w, out=out, workspace=ws)
    want = torch.zeros_like(w)
    gen = torch.Generator().manual_seed(72)
    for lens in ([700, 390, 300], [650, 390, 217], [1 + news[0], 201, 299]):
        dev["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        dev["q"].copy_(torch.randn(a["q"].shape, generator=gen).half())
        torch.cuda.synchronize()
        g.replay()
        got = call(want)
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(w, want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(w, stream=s)
    call(want, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(w, want)
    _clean(vq)


def test_numbers_that_make_no_sense_are_reported(vq):  # noqa: F811
    a = _case(vq, [5, 60], [100, 140], 1, 4, 16, F16, F16, seed=82)
    w = _weights(a, 3, 1.0).cuda()
    for bad in (dict(cu=torch.tensor([0, 1000, -5], dtype=torch.int32)), dict(max_q=2), dict(lens=torch.tensor([100, 10 ** 6], dtype=torch.int32)),
                dict(lens=torch.tensor([-1, 140], dtype=torch.int32))):
        _run(vq, dict(a, **bad), w.clone(), 0, 1.0)
        torch.cuda.synchronize()
        assert vq.vq_device_error() == vq.VQ_DEVERR_BAD_OFFSET
    _check(vq, a)


@pytest.mark.parametrize("cache", [F16, E4M3])
def test_a_bounded_cache(vq, cache):  # noqa: F811
    """The loop of eviction by accumulated weight: a prompt in chunks, then tokens one
    by one; when a sequence has outgrown its budget, the tokens of largest weight stay
    and move together.  At every step the outputs are those of plain attention
    over the tokens that each head kept, and the weights are those tokens' sums."""
    gen = torch.Generator("cuda").manual_seed(3)
    H, GQ, PS, B, budget, room = 2, 4, 16, 3, 96, 160
    pages = room // PS
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(4)).view(B, pages).to(torch.int32).cuda()
    c = vq.paged_cache(B * pages, H, PS, cache)
    w = torch.zeros(B * pages, H, PS, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    kept = [[[] for _ in range(H)] for _ in range(B)]  # (key, value, weight) of each head's tokens, 64 bits
    length = [0] * B
    scale = D ** -0.5
    for step in range(60):
        news = [40, 7, 23] if step < 3 else [1, 1, 1]
        T = sum(news)
        q = torch.randn(T, H * GQ, D, generator=gen, device="cuda").half()
        kv = torch.randn(2, T, H, D, generator=gen, device="cuda").half()
        b_of = torch.repeat_interleave(torch.arange(B), torch.tensor(news))
        cu = np.cumsum([0] + news)
        j = torch.tensor([length[b] + t - cu[b] for t, b in enumerate(b_of.tolist())], device="cuda")
        vq.vq_paged_append(kv[0], kv[1], c, table[b_of.cuda(), j // PS].long() * PS + j % PS)
        lens = torch.tensor([x + n for x, n in zip(length, news)], **i32)
        out = vq.vq_paged_attend_weigh(q, c, w, table, torch.tensor(cu, **i32), lens, scale, max_q=max(news), decay=0.99)
        if cache == E4M3:
            kq = [ref.values(*ref.quantise(kv[i].cpu())) for i in range(2)]
        else:
            kq = [kv[i].cpu().double() for i in range(2)]
        for b in range(B):
            for h in range(H):
                rows = kept[b][h]
                for r in rows:
                    r[2] *= 0.99
                for t in range(cu[b], cu[b + 1]):
                    rows.append([kq[0][t, h], kq[1][t, h], 0.0])
                K, V = torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])
                for t in range(cu[b], cu[b + 1]):
                    n = length[b] + (t - cu[b]) + 1
                    s = torch.softmax(K[:n] @ q[t, h * GQ:(h + 1) * GQ].cpu().double().T * scale, 0)
                    o = s.T @ V[:n]
                    got = out[t, h * GQ:(h + 1) * GQ].cpu().double()
                    # weights and outputs rounded to fp16, 2^-11 each
                    assert bool(((got - o).abs() <= 2.0 ** -11 * (s.T @ V[:n].abs()) + 2.0 ** -11 * o.abs() + 2.0 ** -16).all())
                    for i, x in enumerate(s.sum(1).tolist()):
                        rows[i][2] += x
        length = [x + n for x, n in zip(length, news)]
        have = w[table.long()].permute(0, 2, 1, 3).reshape(B, H, -1).cpu().double()
        for b in range(B):
            for h in range(H):
                want = torch.tensor([r[2] for r in kept[b][h]], dtype=torch.float64)
                # 60 steps' sums in 32 bits, scores' rounding (2^-24 * 140 * sum |q k| below 2^-15)
                assert torch.allclose(have[b, h, :length[b]], want, rtol=2.0 ** -12, atol=2.0 ** -20)
        if max(length) > room - 45:
            keep, counts = vq.vq_paged_select(w, table, lens, budget, recent=16, sinks=4)
            vq.vq_paged_compact(c, table, keep, counts, weights=w)
            for b in range(B):
                for h in range(H):
                    kept[b][h] = [kept[b][h][i] for i in keep[b, h].tolist() if i >= 0]
            length = counts.tolist()
            assert all(len(kept[b][h]) == length[b] for b in range(B) for h in range(H))
    _clean(vq)


def test_more_sequences_than_a_block_has_threads(vq):  # noqa: F811
    """Over a thousand chunks and single tokens: units of weighing are found among
    sequences that the plan goes through in several steps."""
    news = [17 + i % 5 if i % 9 else 40 for i in range(1100)]
    news[3::50] = [1] * len(news[3::50])
    lens = [n + i % 37 for i, n in enumerate(news)]
    _check(vq, _case(vq, news, lens, 1, 1, 16, F16, F16, seed=55), observe=9, decay=0.5)
