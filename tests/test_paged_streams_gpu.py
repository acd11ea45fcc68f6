"""Streams of the paged-cache calls: whose memory the buffers made by a call are,
calls given a stream's handle, a captured call of chunks and single tokens."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def vq():
    from kv_cache_quantization_turboquantrvq_gb300 import api, build
    build.build()
    api.lib()
    return api


def _call(vq, news, lens, GQ=4, Hkv=2, PS=16, dtype=torch.float16, cache=torch.float16, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    NP = sum(-(-n // PS) for n in lens)
    c = vq.paged_cache(NP, Hkv, PS, cache)
    width = max(-(-n // PS) for n in lens)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // PS)
        table[b, :m] = torch.arange(at, at + m)
        at += m
    kv = torch.randn(2, NP * PS, Hkv, D, generator=gen, device="cuda").to(dtype)
    vq.vq_paged_append(kv[0], kv[1], c, torch.arange(NP * PS, device="cuda"))
    q = torch.randn(sum(news), Hkv * GQ, D, generator=gen, device="cuda").to(dtype)
    cu = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    return dict(q=q, cache=c, block_table=table.cuda(), cu_q=cu,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=D ** -0.5, max_q=max(news))


class _NoLaunch:
    """The library with attend and gather taken out: their arguments are kept."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        return getattr(self.real, name)

    def vq_paged_attend(self, *a):
        self.args = a
        return 0

    def vq_paged_gather(self, *a):
        self.args = a
        return 0


@pytest.mark.parametrize("form", ["stream", "handle"])
def test_buffers_made_by_a_call_belong_to_its_stream(vq, monkeypatch, form):
    """A block that the current stream gave back must not become an output that
    another stream writes, nor a workspace that one still uses the current
    stream's next block.  Nothing is launched."""
    a = _call(vq, [700, 1], [700, 300])
    s = torch.cuda.Stream()
    st = s if form == "stream" else s.cuda_stream
    lib = _NoLaunch(vq.lib())
    monkeypatch.setattr(vq, "_lib", lib)
    out_bytes = a["q"].numel() * 2
    ws_bytes = vq.vq_paged_attend_workspace(701, 2, 8, 2, 700)
    torch.cuda.empty_cache()
    x, w = torch.empty(out_bytes, dtype=torch.uint8, device="cuda"), torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    mine = {x.data_ptr(), w.data_ptr()}
    del x, w
    out = vq.vq_paged_attend(stream=st, **a)
    (ws,) = [p for p, n in zip(lib.args[-3:], lib.args[-2:]) if n == ws_bytes]
    assert out.data_ptr() not in mine and ws not in mine
    y, z = torch.empty(out_bytes, dtype=torch.uint8, device="cuda"), torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    assert ws not in (y.data_ptr(), z.data_ptr())
    del y, z
    k, v = vq.vq_paged_gather(a["cache"], a["block_table"], a["lens"], 700, stream=st)
    x = torch.empty_like(k)
    mine = x.data_ptr()
    del x
    k2, v2 = vq.vq_paged_gather(a["cache"], a["block_table"], a["lens"], 700, stream=st)
    assert mine not in (k2.data_ptr(), v2.data_ptr())


@pytest.mark.parametrize("cache", [torch.float16, torch.float8_e4m3fn])
@pytest.mark.parametrize("news", [[1, 1], [300, 1]])
def test_handles_and_streams_give_the_same(vq, cache, news):
    a = _call(vq, news, [700, 300], cache=cache, seed=1)
    want = vq.vq_paged_attend(**a)
    kw, vw = vq.vq_paged_gather(a["cache"], a["block_table"], a["lens"], 300)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for st in (s, s.cuda_stream, 0, torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream):
        got = vq.vq_paged_attend(stream=st, **a)
        k, v = vq.vq_paged_gather(a["cache"], a["block_table"], a["lens"], 300, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(k, kw) and torch.equal(v, vw)
    assert vq.vq_device_error() == 0


@pytest.mark.parametrize("cache", [torch.float16, torch.float8_e4m3fn])
def test_a_captured_mixed_call_follows_its_inputs(vq, cache):
    """Plan, chunks, single tokens and merge overlap on the GPU; replayed with other
    lengths, other numbers of new tokens and other queries, back to back, each
    replay gives what a call of its own gives."""
    a = _call(vq, [300, 1, 1, 40], [2700, 900, 1500, 1300], cache=cache, seed=2)
    T = a["q"].shape[0]
    out = torch.empty_like(a["q"])
    ws = torch.full((vq.vq_paged_attend_workspace(T, 4, 8, 2, 300),), 255, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vq.vq_paged_attend(out=out, workspace=ws, **a)
    gen = torch.Generator().manual_seed(3)
    seen, want = [], []
    for i in range(12):
        cut = sorted(torch.randint(0, 301, (3,), generator=gen).tolist())
        cu = [0, cut[0], cut[1], cut[2], min(T, cut[2] + 300)] if i % 2 else [0, 300, 301, 302, 342]
        lens = [int(torch.randint(m // 4, m + 1, (1,), generator=gen)) for m in (2700, 900, 1500, 1300)]
        q = torch.randn(a["q"].shape, generator=gen).to(a["q"].dtype).cuda()
        cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, lens))
        w = torch.zeros_like(out)
        vq.vq_paged_attend(**dict(a, q=q, cu_q=cu, lens=lens, out=w))
        seen.append((q, cu, lens))
        want.append(w)
    torch.cuda.synchronize()
    got = [torch.zeros_like(out) for _ in want]
    for (q, cu, lens), o in zip(seen, got):  # (no wait between the replays)
        a["q"].copy_(q)
        a["cu_q"].copy_(cu)
        a["lens"].copy_(lens)
        out.zero_()
        g.replay()
        o.copy_(out)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert vq.vq_device_error() == 0
