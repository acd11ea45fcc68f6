"""Refusals of tree attention and of the calls that keep a part of a paged cache (host arithmetic, no
GPU: fake addresses that never reach a device)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from test_paged_binding import Fake, _cache, api as binding  # noqa: E402,F401
from test_paged_host import A, M, P, api  # noqa: E402,F401

I32, F32 = torch.int32, torch.float32


def _select(api, w=A, NP=4, H=2, PS=16, table=A + M, mp=3, lens=A + 2 * M, B=2, budget=20, recent=4, sinks=2, keep=A + 3 * M,
            counts=A + 4 * M):
    return api.lib().vq_paged_select(P(w), NP, H, PS, P(table), mp, P(lens), B, budget, recent, sinks, P(keep), P(counts), None)


def test_select_refusals(api):  # noqa: F811
    assert _select(api, PS=24) == api.VQ_ERR_UNSUPPORTED
    assert _select(api, mp=(1 << 26) + 1) == api.VQ_ERR_UNSUPPORTED
    assert _select(api, B=1 << 24) == api.VQ_ERR_UNSUPPORTED
    assert _select(api, budget=(1 << 30) + 1) == api.VQ_ERR_UNSUPPORTED
    assert _select(api, H=0) == api.VQ_ERR_INVALID_ARG
    assert _select(api, B=-1) == api.VQ_ERR_INVALID_ARG
    assert _select(api, budget=-1, recent=0, sinks=0) == api.VQ_ERR_INVALID_ARG
    assert _select(api, recent=-1) == api.VQ_ERR_INVALID_ARG
    assert _select(api, sinks=-1) == api.VQ_ERR_INVALID_ARG
    assert _select(api, recent=19) == api.VQ_ERR_INVALID_ARG          # 19 + 2 of 20
    assert _select(api, recent=2 ** 31 - 1, sinks=2 ** 31 - 1) == api.VQ_ERR_INVALID_ARG
    assert _select(api, w=0) == api.VQ_ERR_INVALID_ARG
    assert _select(api, lens=0) == api.VQ_ERR_INVALID_ARG
    assert _select(api, keep=0) == api.VQ_ERR_INVALID_ARG
    assert _select(api, counts=0) == api.VQ_ERR_INVALID_ARG
    assert _select(api, table=0) == api.VQ_ERR_INVALID_ARG
    assert _select(api, w=A + 2) == api.VQ_ERR_MISALIGNED
    assert _select(api, keep=A + 3 * M + 1) == api.VQ_ERR_MISALIGNED
    assert _select(api, keep=A + 16) == api.VQ_ERR_ALIASING           # over the weights
    assert _select(api, counts=A + 3 * M + 4) == api.VQ_ERR_ALIASING  # over the list
    assert _select(api, keep=A + M) == api.VQ_ERR_ALIASING            # over the block table
    assert _select(api, B=0, w=0, keep=0) == api.VQ_OK


def _compact(api, kp=A, vp=A + M, ke=0, ve=0, ct=0, NP=4, H=2, PS=16, D=128, table=A + 2 * M, mp=3, keep=A + 3 * M, sb=40, sh=20,
             K=20, counts=A + 4 * M, first=0, B=2, w=0):
    return api.lib().vq_paged_compact(P(kp), P(vp), P(ke), P(ve), ct, NP, H, PS, D, P(table), mp, P(keep), sb, sh, K, P(counts),
                                      P(first), B, P(w), None)


def test_compact_refusals(api):  # noqa: F811
    assert _compact(api, D=64) == api.VQ_ERR_UNSUPPORTED
    assert _compact(api, PS=8) == api.VQ_ERR_UNSUPPORTED
    assert _compact(api, mp=(1 << 26) + 1) == api.VQ_ERR_UNSUPPORTED
    assert _compact(api, B=1 << 24) == api.VQ_ERR_UNSUPPORTED
    assert _compact(api, K=(1 << 30) + 1) == api.VQ_ERR_UNSUPPORTED
    assert _compact(api, sb=1 << 38) == api.VQ_ERR_UNSUPPORTED
    assert _compact(api, B=-1) == api.VQ_ERR_INVALID_ARG
    assert _compact(api, K=-1) == api.VQ_ERR_INVALID_ARG
    assert _compact(api, sh=-1) == api.VQ_ERR_INVALID_ARG
    assert _compact(api, ct=3) == api.VQ_ERR_INVALID_ARG
    assert _compact(api, ct=2) == api.VQ_ERR_INVALID_ARG              # codes without exponents
    assert _compact(api, kp=0) == api.VQ_ERR_INVALID_ARG
    assert _compact(api, keep=0) == api.VQ_ERR_INVALID_ARG
    assert _compact(api, counts=0) == api.VQ_ERR_INVALID_ARG
    assert _compact(api, table=0) == api.VQ_ERR_INVALID_ARG
    assert _compact(api, NP=0) == api.VQ_ERR_INVALID_ARG
    assert _compact(api, kp=A + 8) == api.VQ_ERR_MISALIGNED
    assert _compact(api, keep=A + 3 * M + 2) == api.VQ_ERR_MISALIGNED
    assert _compact(api, first=A + 5 * M + 2) == api.VQ_ERR_MISALIGNED
    assert _compact(api, w=A + 5 * M + 1) == api.VQ_ERR_MISALIGNED
    assert _compact(api, vp=A + 512) == api.VQ_ERR_ALIASING
    assert _compact(api, keep=A + 512) == api.VQ_ERR_ALIASING
    assert _compact(api, w=A + M) == api.VQ_ERR_ALIASING
    assert _compact(api, w=A + 4 * M) == api.VQ_ERR_ALIASING          # over the counts
    assert _compact(api, K=0, keep=0) == api.VQ_OK
    assert _compact(api, B=0, kp=0, vp=0) == api.VQ_OK


# ---------------------------------------------------------------- the binding

def _bind_select(b, device=0, **kw):
    a = dict(weights=Fake((4, 2, 16), F32, device), block_table=Fake((2, 3), I32, device), lens=Fake((2,), I32, device),
             budget=20, recent=4, sinks=2, keep=Fake((2, 2, 20), I32, device), counts=Fake((2,), I32, device), stream=64)
    a.update(kw)
    return b.vq_paged_select(**a)


def _bind_compact(b, device=0, **kw):
    a = dict(cache=_cache(device), block_table=Fake((2, 3), I32, device), keep=Fake((2, 2, 20), I32, device),
             counts=Fake((2,), I32, device), first=Fake((2,), I32, device), weights=Fake((4, 2, 16), F32, device), stream=64)
    a.update(kw)
    return b.vq_paged_compact(**a)


def test_bound_calls_reach_the_library_on_their_gpu(binding):  # noqa: F811
    _bind_select(binding, device=1)
    _bind_compact(binding, device=1)
    assert [(n, d) for n, d, _ in binding.log] == [("vq_paged_select", 1), ("vq_paged_compact", 1)]


def test_one_list_for_all_heads_has_no_head_stride(binding):  # noqa: F811
    _bind_compact(binding, keep=Fake((2, 1, 20), I32))
    _bind_compact(binding)
    assert [a[12:15] for _, _, a in binding.log] == [(20, 0, 20), (40, 20, 20)]


@pytest.mark.parametrize("call,name,bad", [
    (_bind_select, "weights", Fake((4, 2, 16), F32, 1)), (_bind_select, "weights", Fake((4, 2, 16), torch.float16)),
    (_bind_select, "lens", Fake((3,), I32)), (_bind_select, "lens", Fake((2,), torch.int64)),
    (_bind_select, "keep", Fake((2, 2, 19), I32)), (_bind_select, "counts", Fake((2,), I32, 1)),
    (_bind_select, "block_table", Fake((2, 3), I32, contiguous=False)), (_bind_select, "block_table", Fake((2, 3), I32, -1)),
    (_bind_compact, "keep", Fake((2, 3, 20), I32)), (_bind_compact, "keep", Fake((2, 2, 20), torch.int64)),
    (_bind_compact, "keep", Fake((3, 2, 20), I32)), (_bind_compact, "keep", Fake((2, 2, 20), I32, 1)),
    (_bind_compact, "counts", Fake((2,), torch.int64)), (_bind_compact, "first", Fake((3,), I32)),
    (_bind_compact, "weights", Fake((4, 2, 32), F32)), (_bind_compact, "weights", Fake((4, 2, 16), torch.float16)),
    (_bind_compact, "cache", _cache(1))])
def test_bound_refusals(binding, call, name, bad):  # noqa: F811
    with pytest.raises(ValueError):
        call(binding, **{name: bad})
    assert not binding.log


@pytest.mark.parametrize("name", ["budget", "recent", "sinks"])
@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 4])
def test_numbers_past_32_bits_are_refused(binding, name, value):  # noqa: F811
    with pytest.raises(ValueError):
        _bind_select(binding, **{name: value})
    assert not binding.log


# ------------------------------------------------- trees and weights: refusals

def _tree(api, parents=A + 8 * M, max_q=4, wb=1 << 30, q=A, qst=1024, T=8, Hq=8, out=A + 6 * M, ws=A + 7 * M, window=0, scale=0.1):
    return api.lib().vq_paged_attend_tree(P(q), qst, 128, 0, P(A + M), P(A + 2 * M), P(0), P(0), 0, 4, 2, 16, 128, P(A + 3 * M), 3,
                                          P(A + 4 * M), P(A + 5 * M), P(parents), T, 2, Hq, max_q, window, 0,
                                          ctypes.c_float(scale), P(out), P(ws), wb, None)


def test_tree_refusals(api):  # noqa: F811
    assert _tree(api, max_q=257) == api.VQ_ERR_UNSUPPORTED
    assert _tree(api, Hq=34) == api.VQ_ERR_UNSUPPORTED
    assert _tree(api, max_q=0) == api.VQ_ERR_INVALID_ARG
    assert _tree(api, parents=0) == api.VQ_ERR_INVALID_ARG
    assert _tree(api, window=-1) == api.VQ_ERR_INVALID_ARG
    assert _tree(api, scale=float("inf")) == api.VQ_ERR_INVALID_ARG
    assert _tree(api, wb=1000) == api.VQ_ERR_INVALID_ARG
    assert _tree(api, parents=A + 8 * M + 2) == api.VQ_ERR_MISALIGNED
    assert _tree(api, qst=1028) == api.VQ_ERR_MISALIGNED
    assert _tree(api, parents=A + 6 * M) == api.VQ_ERR_ALIASING        # over the output
    assert _tree(api, parents=A + 7 * M + 64) == api.VQ_ERR_ALIASING   # in the workspace
    assert _tree(api, T=0, parents=0) == api.VQ_OK
    n = ctypes.c_size_t(0)
    f = api.lib().vq_paged_attend_tree_workspace
    assert f(8, 2, 8, 2, 4, None) == api.VQ_ERR_INVALID_ARG
    assert f(8, 2, 8, 2, 257, ctypes.byref(n)) == api.VQ_ERR_UNSUPPORTED
    assert f(8, 2, 7, 2, 4, ctypes.byref(n)) == api.VQ_ERR_INVALID_ARG
    assert f(800, 2, 8, 2, 256, ctypes.byref(n)) == api.VQ_OK and n.value >= 800 * 36


def _weigh(api, w=A + 8 * M, observe=0, decay=1.0, max_q=4, wb=1 << 29, q=A, T=8, Hq=8, out=A + 6 * M, ws=A + 7 * M, mp=3, PS=16):
    return api.lib().vq_paged_attend_weigh(P(q), 1024, 128, 0, P(A + M), P(A + 2 * M), P(0), P(0), 0, 4, 2, PS, 128, P(A + 3 * M), mp,
                                           P(A + 4 * M), P(A + 5 * M), T, 2, Hq, max_q, 0, 0, ctypes.c_float(0.1), P(w), observe,
                                           ctypes.c_float(decay), P(out), P(ws), wb, None)


def test_weigh_refusals(api):  # noqa: F811
    assert _weigh(api, observe=-1) == api.VQ_ERR_INVALID_ARG
    for decay in (-0.1, 1.1, float("nan"), float("inf")):
        assert _weigh(api, decay=decay) == api.VQ_ERR_INVALID_ARG
    assert _weigh(api, w=0) == api.VQ_ERR_INVALID_ARG
    assert _weigh(api, wb=1000) == api.VQ_ERR_INVALID_ARG
    assert _weigh(api, w=A + 8 * M + 8) == api.VQ_ERR_MISALIGNED
    assert _weigh(api, w=A + 6 * M) == api.VQ_ERR_ALIASING             # over the output
    assert _weigh(api, w=A + 7 * M + 64) == api.VQ_ERR_ALIASING        # in the workspace
    assert _weigh(api, w=A + M) == api.VQ_ERR_ALIASING                 # over the keys
    assert _weigh(api, w=A + 5 * M) == api.VQ_ERR_ALIASING             # over the lengths
    assert _weigh(api, T=0, w=0) == api.VQ_OK
    n = ctypes.c_size_t(0)
    f = api.lib().vq_paged_attend_weigh_workspace
    assert f(8, 2, 8, 2, 4, 3, 16, None) == api.VQ_ERR_INVALID_ARG
    assert f(8, 2, 8, 2, 4, -1, 16, ctypes.byref(n)) == api.VQ_ERR_INVALID_ARG
    assert f(8, 2, 8, 2, 4, 3, 24, ctypes.byref(n)) == api.VQ_ERR_UNSUPPORTED
    assert f(8, 2, 8, 2, 4, (1 << 26) + 1, 16, ctypes.byref(n)) == api.VQ_ERR_UNSUPPORTED
    assert f(1 << 20, 1 << 20, 64, 64, 1, 1 << 22, 256, ctypes.byref(n)) == api.VQ_ERR_UNSUPPORTED  # a petabyte
    assert f(64, 64, 32, 8, 1, 1024, 16, ctypes.byref(n)) == api.VQ_OK and n.value >= 64 * 8 * 4 * 16384 * 4


def _bind_tree(b, device=0, **kw):
    a = dict(q=Fake((5, 8, 128), torch.float16, device), cache=_cache(device), block_table=Fake((2, 3), I32, device),
             cu_q=Fake((3,), I32, device), lens=Fake((2,), I32, device), parents=Fake((5,), I32, device), scale=0.1, max_q=4,
             out=Fake((5, 8, 128), torch.float16, device), workspace=Fake((1 << 20,), torch.uint8, device), stream=64)
    a.update(kw)
    return b.vq_paged_attend_tree(**a)


def _bind_weigh(b, device=0, **kw):
    a = dict(q=Fake((5, 8, 128), torch.float16, device), cache=_cache(device), block_table=Fake((2, 3), I32, device),
             cu_q=Fake((3,), I32, device), lens=Fake((2,), I32, device), weights=Fake((4, 2, 16), F32, device), scale=0.1, max_q=4,
             out=Fake((5, 8, 128), torch.float16, device), workspace=Fake((1 << 20,), torch.uint8, device), stream=64)
    a.update(kw)
    return b.vq_paged_attend_weigh(**a)


def test_bound_attention_reaches_the_library_on_its_gpu(binding, monkeypatch):  # noqa: F811
    _bind_tree(binding, device=1)
    _bind_weigh(binding, device=1)
    monkeypatch.setattr(binding, "_empty", lambda shape, dtype, device, stream, returned=True: Fake((shape,), dtype, 1))
    _bind_tree(binding, device=1, workspace=None)
    _bind_weigh(binding, device=1, workspace=None)
    _bind_weigh(binding, device=1, workspace=None, block_table=Fake((2, 5), I32, 1))
    assert [(n, d) for n, d, _ in binding.log] == [(x, 1) for x in (
        "vq_paged_attend_tree", "vq_paged_attend_weigh", "vq_paged_attend_tree_workspace", "vq_paged_attend_tree",
        "vq_paged_attend_weigh_workspace", "vq_paged_attend_weigh", "vq_paged_attend_weigh_workspace", "vq_paged_attend_weigh")]


@pytest.mark.parametrize("call,name,bad", [
    (_bind_tree, "parents", Fake((4,), I32)), (_bind_tree, "parents", Fake((5,), torch.int64)), (_bind_tree, "parents", Fake((5,), I32, 1)),
    (_bind_tree, "parents", Fake((5,), I32, contiguous=False)), (_bind_tree, "lens", Fake((2,), I32, 1)),
    (_bind_weigh, "weights", Fake((4, 2, 16), F32, 1)), (_bind_weigh, "weights", Fake((4, 2, 32), F32)),
    (_bind_weigh, "weights", Fake((4, 2, 16), torch.float16)), (_bind_weigh, "weights", Fake((4, 2, 16), F32, contiguous=False)),
    (_bind_weigh, "cache", _cache(1)), (_bind_weigh, "observe", 1 << 31), (_bind_weigh, "max_q", 1 << 32), (_bind_tree, "window", 1 << 40)])
def test_bound_attention_refusals(binding, call, name, bad):  # noqa: F811
    with pytest.raises(ValueError):
        call(binding, **{name: bad})
    assert not binding.log


@pytest.mark.parametrize("max_q", [1 << 27, 1 << 28, (1 << 28) + 1, (1 << 31) - 1])
def test_weigh_workspace_of_any_max_q(api, max_q):  # noqa: F811
    """max_q times the query heads passes 32 bits: as much room as for chunks of 100 tokens."""
    f = api.lib().vq_paged_attend_weigh_workspace
    sizes = []
    for m in (100, max_q):
        n = ctypes.c_size_t(0)
        assert f(150, 2, 16, 1, m, 4, 16, ctypes.byref(n)) == api.VQ_OK
        sizes.append(n.value)
    assert sizes[0] == sizes[1]
