"""Choosing the tokens of a paged cache that stay, and moving them together, on
the GPU against plain host code.  Both are exact: every index and every byte of
the pools is compared, what must not change included."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
D = 128
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def vq():
    from kv_cache_quantization_turboquantrvq_gb300 import api, build
    build.build()
    api.lib()
    return api


def _cuda(c):
    return {k: None if x is None else x.cuda() for k, x in c.items()}


def _clean(vq, code=0):
    torch.cuda.synchronize()
    assert vq.vq_device_error() == code


def _table(gen, lens, PS, extra=1):
    """Shuffled pages of all sequences, numbers of no page behind them; pages in the pool."""
    width = max(1, max(-(-n // PS) for n in lens)) + extra
    need = torch.tensor([[p * PS < n for p in range(width)] for n in lens])
    NP = int(need.sum()) + 3
    table = torch.tensor([-1, -7, NP, 2 ** 30], dtype=torch.int32)[torch.randint(0, 4, need.shape, generator=gen)]
    table[need] = torch.randperm(NP, generator=gen)[:int(need.sum())].to(torch.int32)
    return table, NP


# ---------------------------------------------------------------- the choice

def _select_ref(w, table, lens, budget, recent, sinks):
    PS, H = w.shape[2], w.shape[1]
    keep = np.full((len(lens), H, budget), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for h in range(H):
            if n <= budget:
                keep[b, h, :n] = np.arange(n)
                continue
            j = np.arange(sinks, n - recent)
            x = w[table[b].numpy()[j // PS], h, j % PS].numpy().astype(np.float64)
            x = np.where(np.isnan(x), np.inf, x)
            nan = np.isnan(w[table[b].numpy()[j // PS], h, j % PS].numpy())
            order = np.lexsort((j, -x, ~nan))  # NaN first, then by weight, then by index
            best = j[order[:budget - sinks - recent]]
            keep[b, h] = np.concatenate([np.arange(sinks), np.sort(best), np.arange(n - recent, n)])
    return keep


def _weights(gen, NP, H, PS, kind):
    x = torch.randn(NP, H, PS, generator=gen)
    if kind == "softmax":
        return torch.exp(2 * x) / 1000 * (torch.rand(NP, H, PS, generator=gen) > 0.05)
    if kind == "ties":
        return torch.randint(0, 4, (NP, H, PS), generator=gen).float() / 8
    if kind == "equal":
        return torch.full((NP, H, PS), 0.25)
    if kind == "close":  # differ in the last bits alone
        return (torch.randint(0, 64, (NP, H, PS), generator=gen, dtype=torch.int32) + 0x3F800000).view(torch.float32)
    if kind == "any":
        w = x * torch.exp2(torch.randint(-140, 120, (NP, H, PS), generator=gen).float())
        special = torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan"), 1e-45, -1e-45])
        pick = torch.rand(NP, H, PS, generator=gen) < 0.2
        w[pick] = special[torch.randint(0, 7, (int(pick.sum()),), generator=gen)]
        return w
    raise ValueError(kind)


def _select(vq, w, table, lens, budget, recent, sinks, **kw):
    return vq.vq_paged_select(w.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), budget, recent=recent,
                              sinks=sinks, **kw)


@pytest.mark.parametrize("kind", ["softmax", "ties", "equal", "close", "any"])
@pytest.mark.parametrize("PS,H,lens,budget,recent,sinks", [
    (16, 2, [0, 1, 16, 17, 40, 100, 333], 16, 0, 0),
    (16, 1, [0, 1, 99, 100, 101, 102, 700], 100, 30, 4),
    (32, 3, [5000, 64, 4100, 1], 1, 0, 0),
    (64, 2, [300, 77, 2500], 64, 32, 32),              # nothing left to choose
    (128, 8, [9001, 12000], 2049, 256, 4),             # clusters
    (256, 1, [70001], 3001, 100, 130)])
def test_select(vq, kind, PS, H, lens, budget, recent, sinks):
    gen = torch.Generator().manual_seed(budget + PS)
    table, NP = _table(gen, lens, PS)
    w = _weights(gen, NP, H, PS, kind)
    keep, counts = _select(vq, w, table, lens, budget, recent, sinks)
    _clean(vq)
    assert counts.tolist() == [min(n, budget) for n in lens]
    assert np.array_equal(keep.cpu().numpy(), _select_ref(w, table, lens, budget, recent, sinks))


@pytest.mark.parametrize("B,H,n", [(1, 1, 400000), (40, 8, 3000), (200, 1, 45000)])
def test_select_of_few_long_and_many_short_rows(vq, B, H, n):
    """More weights than one block, or a whole cluster, keeps at hand; more rows than blocks at a time."""
    gen = torch.Generator().manual_seed(n)
    lens = [n - 13 * i for i in range(B)]
    table, NP = _table(gen, lens, 256)
    w = _weights(gen, NP, H, 256, "softmax")
    keep, counts = _select(vq, w, table, lens, 1000, 50, 4)
    _clean(vq)
    rows = list(range(B)) if B < 50 else [0, 1, B // 2, B - 1]
    want = _select_ref(w, table[rows], [lens[b] for b in rows], 1000, 50, 4)
    assert np.array_equal(keep.cpu().numpy()[rows], want)
    assert counts.tolist() == [1000] * B


def test_select_a_table_far_wider_than_the_lengths(vq):
    gen = torch.Generator().manual_seed(5)
    lens = [500, 30, 7]
    table, NP = _table(gen, lens, 16, extra=60000)
    w = _weights(gen, NP, 2, 16, "softmax")
    keep, _ = _select(vq, w, table, lens, 20, 5, 1)
    _clean(vq)
    assert np.array_equal(keep.cpu().numpy(), _select_ref(w, table, lens, 20, 5, 1))


def test_select_reports_lengths_and_pages(vq):
    gen = torch.Generator().manual_seed(6)
    table, NP = _table(gen, [64, 64, 64], 16, extra=0)
    w = _weights(gen, NP, 1, 16, "softmax")
    good = _select(vq, w, table, [64, 64, 64], 20, 4, 4)[0]
    _clean(vq)
    keep, counts = _select(vq, w, table, [-3, 64, 1000], 20, 4, 4)
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
    assert counts.tolist() == [0, 20, 20] and bool((keep[0] == -1).all())
    assert torch.equal(keep[1], good[1]) and torch.equal(keep[2], good[2])
    hole = table.clone()
    hole[1, 1] = NP
    keep, _ = _select(vq, w, hole, [64, 64, 64], 20, 4, 4)
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
    assert torch.equal(keep[0], good[0]) and torch.equal(keep[2], good[2])
    assert not bool(((keep[1] >= 16) & (keep[1] < 32)).any())
    # pages of the tokens that stay anyway are not read
    edge = table.clone()
    edge[:, 3] = -1
    keep, _ = _select(vq, w, edge, [64, 64, 64], 20, 16, 0)
    _clean(vq)


# --------------------------------------------------------------- moving rows

def _pool(vq, NP, H, PS, dtype, gen):
    """Pools of random bytes (any code, any exponent, NaN among them)."""
    c = vq.paged_cache(NP, H, PS, dtype, device="cpu")
    for x in "kv":
        if dtype == E4M3:
            c[x + "_pages"] = torch.randint(0, 256, (NP, H, PS, D), generator=gen, dtype=torch.uint8).view(E4M3)
            c[x + "_exp"] = torch.randint(0, 256, (NP, H, PS), generator=gen, dtype=torch.uint8)
        else:
            c[x + "_pages"] = torch.randint(-2 ** 15, 2 ** 15, (NP, H, PS, D), generator=gen).to(torch.int16).view(dtype)
    return c


def _bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)


def _compact_ref(c, w, table, keep, counts, first):
    parts = {k: _bits(x) for k, x in c.items() if x is not None}
    if w is not None:
        parts["w"] = _bits(w)
    out = {k: x.clone() for k, x in parts.items()}
    PS = c["k_pages"].shape[2]
    for b, n in enumerate(counts):
        d = torch.arange(n) + (0 if first is None else first[b])
        for h in range(c["k_pages"].shape[1]):
            s = keep[b, h if keep.shape[1] > 1 else 0, :n].long()
            for k in parts:
                out[k][table[b][d // PS].long(), h, d % PS] = parts[k][table[b][s // PS].long(), h, s % PS]
    return out


def _lists(gen, H, lens, counts, first, K):
    keep = torch.full((len(lens), H, K), -1, dtype=torch.int32)
    for b, (n, m) in enumerate(zip(lens, counts)):
        f = 0 if first is None else first[b]
        for h in range(H):
            keep[b, h, :m] = f + torch.randperm(n - f, generator=gen)[:m].sort().values
    return keep


def _check_move(vq, c, w, table, keep, counts, first, code=0, **kw):
    want = _compact_ref(c, w, table, keep, counts, first)
    g = {k: None if x is None else x.cuda() for k, x in c.items()}
    gw = None if w is None else w.cuda()
    i32 = torch.int32
    got = vq.vq_paged_compact(g, table.cuda(), keep.cuda(), torch.tensor(counts, dtype=i32).cuda(),
                              first=None if first is None else torch.tensor(first, dtype=i32).cuda(), weights=gw, **kw)
    _clean(vq, code)
    assert got is g
    for k in want:
        assert torch.equal(_bits(gw if k == "w" else g[k]).cpu(), want[k]), k


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
@pytest.mark.parametrize("PS,H,shared,with_first,with_w", [
    (16, 2, False, False, True), (32, 3, True, True, False), (64, 1, False, True, True), (256, 2, False, False, False),
    (128, 4, True, False, True)])
def test_compact(vq, dtype, PS, H, shared, with_first, with_w):
    """Lists of no token, of one, of all (nothing moves), of rounds that are cut."""
    gen = torch.Generator().manual_seed(PS + H)
    lens = [40, 1, 17, 700, 2500, 300, 5]
    first = [3, 0, 16, 130, 7, 299, 5] if with_first else None
    counts = [0, 1, 1, 129, 1600, 1, 0] if with_first else [0, 1, 17, 129, 1600, 299, 5]
    table, NP = _table(gen, lens, PS)
    c = _pool(vq, NP, H, PS, dtype, gen)
    w = torch.randn(NP, H, PS, generator=gen) if with_w else None
    keep = _lists(gen, 1 if shared else H, lens, counts, first, 1603)
    _check_move(vq, c, w, table, keep, counts, first)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,H,n,m", [(1, 1, 60000, 50001), (12, 8, 5000, 4097), (70, 2, 400, 128)])
def test_compact_long_lists(vq, dtype, B, H, n, m):
    """Many rounds, most sources only just behind their places and all of them far behind."""
    gen = torch.Generator().manual_seed(n)
    lens = [n + i for i in range(B)]
    counts = [m - 7 * i if i % 3 else m for i in range(B)]
    counts = [max(1, x) for x in counts]
    table, NP = _table(gen, lens, 64)
    c = _pool(vq, NP, H, 64, dtype, gen)
    keep = _lists(gen, H, lens, counts, None, m)
    keep[0, 0, :counts[0]] = torch.arange(counts[0]) + (n - counts[0])  # a shift of the whole row
    _check_move(vq, c, torch.randn(NP, H, 64, generator=gen), table, keep, counts, None)


def test_compact_strided_lists(vq):
    """Lists cut out of a wider tensor; one list expanded to all heads."""
    gen = torch.Generator().manual_seed(8)
    lens, counts = [300, 500], [100, 77]
    table, NP = _table(gen, lens, 16)
    c = _pool(vq, NP, 4, 16, F16, gen)
    keep = _lists(gen, 4, lens, counts, None, 100)
    wide = torch.full((2, 6, 150), -5, dtype=torch.int32)
    wide[:, 1:5, 20:120] = keep
    g = {k: None if x is None else x.cuda() for k, x in c.items()}
    cnt = torch.tensor(counts, dtype=torch.int32).cuda()
    vq.vq_paged_compact(g, table.cuda(), wide.cuda()[:, 1:5, 20:120], cnt)
    want = _compact_ref(c, None, table, keep, counts, None)
    _clean(vq)
    assert torch.equal(_bits(g["k_pages"]).cpu(), want["k_pages"]) and torch.equal(_bits(g["v_pages"]).cpu(), want["v_pages"])
    one = keep[:, :1]
    g = {k: None if x is None else x.cuda() for k, x in c.items()}
    vq.vq_paged_compact(g, table.cuda(), one.cuda().expand(-1, 4, -1), cnt)
    want = _compact_ref(c, None, table, one, counts, None)
    _clean(vq)
    assert torch.equal(_bits(g["k_pages"]).cpu(), want["k_pages"]) and torch.equal(_bits(g["v_pages"]).cpu(), want["v_pages"])


def test_compact_leaves_out_and_reports_what_makes_no_sense(vq):
    gen = torch.Generator().manual_seed(9)
    lens = [64] * 7
    table, NP = _table(gen, lens, 16, extra=0)
    c = _pool(vq, NP, 1, 16, F16, gen)
    keep = torch.full((7, 1, 4), -1, dtype=torch.int32)
    keep[:, 0] = torch.tensor([5, 9, 20, 63])
    keep[0, 0, 3] = 64                   # past the block table
    keep[1, 0, 0] = -9                   # before the sequence
    keep[2, 0, 2] = 1                    # before its place
    table[3, 3] = NP + 5                 # no such page: token 63
    first = [0, 0, 0, 0, -1, 65, 2 ** 31 - 1]
    counts = [4] * 7
    g = {k: None if x is None else x.cuda() for k, x in c.items()}
    i32 = torch.int32
    vq.vq_paged_compact(g, table.cuda(), keep.cuda(), torch.tensor(counts, dtype=i32).cuda(), first=torch.tensor(first, dtype=i32).cuda())
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
    want = {x: _bits(c[x + "_pages"]).clone() for x in "kv"}
    for b, moved in enumerate([[0, 1, 2], [1, 2, 3], [0, 1, 3], [0, 1, 2], [], [], []]):
        for i in moved:
            s = int(keep[b, 0, i])
            for x in "kv":
                want[x][table[b, 0], 0, i] = _bits(c[x + "_pages"])[table[b, s // 16], 0, s % 16]
    assert all(torch.equal(_bits(g[x + "_pages"]).cpu(), want[x]) for x in "kv")
    # counts past the list are cut to it, negative ones move nothing
    g = {k: None if x is None else x.cuda() for k, x in c.items()}
    keep = torch.tensor([5, 9, 20, 40], dtype=i32).repeat(7, 1, 1).reshape(7, 1, 4)
    vq.vq_paged_compact(g, table.cuda(), keep.cuda(), torch.tensor([9, -1, 2, 0, 2 ** 31 - 1, -2 ** 31, 4], dtype=i32).cuda())
    _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
    want = _compact_ref(c, None, table, keep, [4, 0, 2, 0, 4, 0, 4], None)
    assert torch.equal(_bits(g["k_pages"]).cpu(), want["k_pages"])


def test_compact_reports_a_list_that_goes_back_to_a_token_in_its_place(vq):
    """The order is asked of every token of a list, those that stay where they are among
    them; a sequence beside it moves as it should.  Pages of tokens that stay are not
    asked for."""
    gen = torch.Generator().manual_seed(13)
    table, NP = _table(gen, [64, 64], 16, extra=0)
    c = _pool(vq, NP, 2, 16, F16, gen)
    i32 = torch.int32
    good = [5, 9, 20, 63]
    for back, first in (([0, 5, 2, 40], 0), ([0, 1, 9, 3], 0), ([16, 30, 18, 19], 16), ([0, 0, 2, 3], 0)):
        keep = torch.tensor([back, good], dtype=i32)[:, None]
        g = _cuda(c)
        vq.vq_paged_compact(g, table.cuda(), keep.cuda(), torch.tensor([4, 4], dtype=i32).cuda(),
                            first=torch.tensor([first, 0], dtype=i32).cuda())
        _clean(vq, vq.VQ_DEVERR_BAD_OFFSET)
        want = _compact_ref(c, None, table, keep, [0, 4], [0, 0])
        mine = table[1].long()
        for x in ("k_pages", "v_pages"):
            assert torch.equal(_bits(g[x]).cpu()[mine], want[x][mine])
    # the first two pages were given back; their tokens and the next ones stay, then others move
    hole = table.clone()
    hole[:, :2] = torch.tensor([-1, NP + 3], dtype=i32)
    keep = torch.tensor(list(range(40)) + [44, 50], dtype=i32).repeat(2, 1)[:, None]
    g = _cuda(c)
    vq.vq_paged_compact(g, hole.cuda(), keep.cuda(), torch.tensor([42, 40], dtype=i32).cuda())
    _clean(vq)
    want = _compact_ref(c, None, table, keep, [42, 40], None)
    assert all(torch.equal(_bits(g[x]).cpu(), want[x]) for x in ("k_pages", "v_pages"))


def test_select_and_compact_on_a_stream_and_in_a_graph(vq):
    """Captured once, replayed over other weights and lengths, as a serving loop
    does; then what is left is read back."""
    gen = torch.Generator().manual_seed(10)
    lens, PS, H, budget = [900, 300, 1200], 32, 2, 256
    table, NP = _table(gen, lens, PS)
    c = _pool(vq, NP, H, PS, BF16, gen)
    w = _weights(gen, NP, H, PS, "softmax")
    g = {k: None if x is None else x.cuda() for k, x in c.items()}
    gw, gt, gl = w.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    keep = torch.empty((3, H, budget), dtype=torch.int32, device="cuda")
    counts = torch.empty(3, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vq.vq_paged_select(gw, gt, gl, budget, recent=16, sinks=4, keep=keep, counts=counts)
        vq.vq_paged_compact(g, gt, keep, counts, weights=gw)
    for i in range(4):
        ln = [n - 100 * i for n in lens]
        w = _weights(gen, NP, H, PS, "softmax")
        c = _pool(vq, NP, H, PS, BF16, gen)
        for k in c:
            if c[k] is not None:
                g[k].copy_(c[k])
        gw.copy_(w)
        gl.copy_(torch.tensor(ln, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref = torch.from_numpy(_select_ref(w, table, ln, budget, 16, 4))
        assert torch.equal(keep.cpu(), ref)
        want = _compact_ref(c, w, table, ref, [min(n, budget) for n in ln], None)
        assert torch.equal(_bits(g["v_pages"]).cpu(), want["v_pages"]) and torch.equal(_bits(gw).cpu(), want["w"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    k2, c2 = vq.vq_paged_select(gw, gt, gl, budget, recent=16, sinks=4, stream=s)
    vq.vq_paged_compact(g, gt, k2, c2, weights=gw, stream=s.cuda_stream)
    s.synchronize()
    _clean(vq)
    assert torch.equal(k2.cpu(), torch.from_numpy(_select_ref(want["w"].view(torch.float32), table, ln, budget, 16, 4)))
