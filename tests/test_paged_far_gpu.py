"""Tree attention, weighing, selection and compaction at the far end of a large
pool, in calls that run at the same time, and in two graphs that share a
workspace: each gives the bits of a plain call."""
import pytest

torch = pytest.importorskip("torch")
from test_paged_gpu import _clean, vq  # noqa: E402,F401

pytestmark = pytest.mark.gpu
D = 128
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
I32 = torch.int32


def _state(vq, lens, news, H=2, GQ=4, PS=16, dtype=F16, cache=F16, seed=0, far=0):  # noqa: F811
    """Tensors of a call; `far` pages lie in the pool before those of the sequences."""
    gen = torch.Generator("cuda").manual_seed(seed)
    per = [-(-n // PS) for n in lens]
    NP = far + sum(per)
    if far:
        shape = (NP, H, PS, D)
        c = {x + "_pages": torch.empty(shape, dtype=torch.uint8 if cache == E4M3 else cache, device="cuda").view(cache) for x in "kv"}
        c.update({x + "_exp": torch.empty(shape[:3], dtype=torch.uint8, device="cuda") if cache == E4M3 else None for x in "kv"})
    else:
        c = vq.paged_cache(NP, H, PS, cache)
    table = torch.full((len(lens), max(per)), -1, dtype=I32)
    at = far
    for b, m in enumerate(per):
        table[b, :m] = torch.arange(at, at + m).flip(0)
        at += m
    total = sum(per) * PS
    kv = torch.randn(2, total, H, D, generator=gen, device="cuda").to(dtype)
    vq.vq_paged_append(kv[0], kv[1], c, torch.arange(far * PS, far * PS + total, device="cuda"))
    w = torch.empty((NP, H, PS), device="cuda")
    w[far:] = torch.rand((NP - far, H, PS), generator=gen, device="cuda")
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    g = torch.Generator().manual_seed(seed)
    up = [int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for n in news for i in range(n)]
    return dict(q=torch.randn(cu[-1], H * GQ, D, generator=gen, device="cuda").to(dtype), c=c, w=w, table=table.cuda(),
                cu=torch.tensor(cu, dtype=I32, device="cuda"), lens=torch.tensor(lens, dtype=I32, device="cuda"),
                up=torch.tensor(up, dtype=I32, device="cuda"), max_q=max(news), far=far)


def _all(vq, a, budget=100, **kw):  # noqa: F811
    """Every operator once; weights and cache are changed."""
    tree = vq.vq_paged_attend_tree(a["q"], a["c"], a["table"], a["cu"], a["lens"], a["up"], D ** -0.5, max_q=a["max_q"], **kw)
    out = vq.vq_paged_attend_weigh(a["q"], a["c"], a["w"], a["table"], a["cu"], a["lens"], D ** -0.5, max_q=a["max_q"], decay=0.5, **kw)
    keep, counts = vq.vq_paged_select(a["w"], a["table"], a["lens"], budget, recent=8, sinks=4, **kw)
    vq.vq_paged_compact(a["c"], a["table"], keep, counts, weights=a["w"], **kw)
    return [tree, out, keep, counts]


def _bits(a):
    f = a["far"]
    parts = [a["c"]["k_pages"][f:], a["c"]["v_pages"][f:], a["w"][f:]] + ([a["c"]["k_exp"][f:], a["c"]["v_exp"][f:]] if a["c"]["k_exp"] is not None else [])
    return [x.contiguous().view(torch.uint8) for x in parts]


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
@pytest.mark.parametrize("news", [[1, 1], [4, 200]])
def test_the_far_end_of_a_large_pool(vq, dtype, cache, news):  # noqa: F811
    """More than 2^32 entries lie before the sequences' pages (17 GB of a 16-bit cache)."""
    PS, H = 256, 2
    far = 2 ** 32 // (PS * H * D) + 7
    kw = dict(lens=[700, 900], news=news, H=H, PS=PS, dtype=dtype, cache=cache, seed=1)
    near, away = _state(vq, **kw), _state(vq, far=far, **kw)
    for x, y in zip(_all(vq, near), _all(vq, away)):
        assert torch.equal(x, y)
    _clean(vq)
    for x, y in zip(_bits(near), _bits(away)):
        assert torch.equal(x, y)
    del near, away
    torch.cuda.empty_cache()


@pytest.mark.parametrize("cache", [F16, E4M3])
def test_calls_at_the_same_time(vq, cache):  # noqa: F811
    """Different sequences on different streams, chunks and single tokens, over and over."""
    jobs = [dict(lens=[900, 1300, 400], news=[1, 130, 40]), dict(lens=[5000], news=[1]), dict(lens=[700] * 20, news=[4] * 20),
            dict(lens=[2100, 300], news=[64, 256])]
    plain = [_state(vq, cache=cache, seed=i, **j) for i, j in enumerate(jobs)]
    want = [_all(vq, a) for a in plain]
    torch.cuda.synchronize()
    for _ in range(3):
        states = [_state(vq, cache=cache, seed=i, **j) for i, j in enumerate(jobs)]
        streams = [torch.cuda.Stream() for _ in jobs]
        torch.cuda.synchronize()
        got = [None] * len(jobs)
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _all(vq, states[i])
        torch.cuda.synchronize()
        for i in range(len(jobs)):
            assert all(torch.equal(x, y) for x, y in zip(got[i], want[i]))
            assert all(torch.equal(x, y) for x, y in zip(_bits(states[i]), _bits(plain[i])))
    _clean(vq)


def test_two_graphs_share_a_workspace(vq):  # noqa: F811
    """Captured tree and weighing calls with one workspace, replayed one after another."""
    a = _state(vq, [900, 1300, 400], [1, 130, 40], seed=7)
    b = _state(vq, [800, 700], [64, 2], seed=8)
    need = max(vq.vq_paged_attend_tree_workspace(171, 3, 8, 2, 130), vq.vq_paged_attend_weigh_workspace(66, 2, 8, 2, 64, b["table"].shape[1], 16))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    o1, o2 = torch.empty_like(a["q"]), torch.empty_like(b["q"])

    def first(out=None, workspace=None):
        return vq.vq_paged_attend_tree(a["q"], a["c"], a["table"], a["cu"], a["lens"], a["up"], D ** -0.5, max_q=130, out=out, workspace=workspace)

    def second(w, out=None, workspace=None):
        return vq.vq_paged_attend_weigh(b["q"], b["c"], w, b["table"], b["cu"], b["lens"], D ** -0.5, max_q=64, observe=5, out=out, workspace=workspace)
    w1, w2 = b["w"].clone(), b["w"].clone()
    want1 = first()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        first(o1, ws)
    with torch.cuda.graph(g2):
        second(w1, o2, ws)
    for _ in range(4):
        o1.zero_()
        o2.zero_()
        g1.replay()
        g2.replay()
        want2 = second(w2)
        torch.cuda.synchronize()
        assert torch.equal(o1, want1) and torch.equal(o2, want2) and torch.equal(w1, w2)
    _clean(vq)


def test_given_buffers_are_all_that_is_used(vq):  # noqa: F811
    """With outputs and workspace given nothing is allocated."""
    a = _state(vq, [900, 1300, 400], [1, 130, 40], seed=9)
    out = torch.empty_like(a["q"])
    wt = torch.empty(vq.vq_paged_attend_tree_workspace(171, 3, 8, 2, 130), dtype=torch.uint8, device="cuda")
    ww = torch.empty(vq.vq_paged_attend_weigh_workspace(171, 3, 8, 2, 130, a["table"].shape[1], 16), dtype=torch.uint8, device="cuda")
    keep, counts = torch.empty((3, 2, 100), dtype=I32, device="cuda"), torch.empty(3, dtype=I32, device="cuda")

    def run():
        vq.vq_paged_attend_tree(a["q"], a["c"], a["table"], a["cu"], a["lens"], a["up"], D ** -0.5, max_q=130, out=out, workspace=wt)
        vq.vq_paged_attend_weigh(a["q"], a["c"], a["w"], a["table"], a["cu"], a["lens"], D ** -0.5, max_q=130, out=out, workspace=ww)
        vq.vq_paged_select(a["w"], a["table"], a["lens"], 100, keep=keep, counts=counts)
        vq.vq_paged_compact(a["c"], a["table"], keep, counts, weights=a["w"])
    run()
    torch.cuda.synchronize()
    before, free = torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]
    for _ in range(5):
        run()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before and torch.cuda.mem_get_info()[0] == free
    _clean(vq)
