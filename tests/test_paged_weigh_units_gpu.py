"""Accumulated weights where a block of the weighing kernel takes many units, of one and
of two key tiles in turn, and where a chunk's sums are shared out in several parts.
That a call does so is asserted from the same arithmetic as the kernel's.  Outputs are
those of the plain call, weights lie within the bound of test_paged_weigh_gpu, and
repeats give the same bits."""
import random

import pytest

torch = pytest.importorskip("torch")
import paged_ref as ref  # noqa: E402
from test_paged_gpu import TYPES, _case, _clean, _cuda, vq  # noqa: E402,F401
from test_paged_weigh_gpu import _run, _weights  # noqa: E402

pytestmark = pytest.mark.gpu
D = 128


def _units(a, Hkv, GQ, observe):
    """For each unit in the kernel's order: (key tiles, query tiles, parts)."""
    cu, lens = a["cu"].tolist(), a["lens"].tolist()
    news = [y - x for x, y in zip(cu, cu[1:])]
    small = len(news) * a["max_q"] > sum(news)
    rows = (8 if GQ <= 8 else 16) if small else 0
    tqt, out = 128 // GQ, []
    for n, m in zip(lens, news):
        if m * GQ <= rows:
            continue
        i0 = max(0, m - observe) if observe else 0
        parts = min(max(-(-(m - i0) // tqt) // 16, 1), 8)
        tiles = max(1, -(-n // 128))
        for t in range(0, tiles, 2):
            first = (max(i0, t * 128 - (n - m)) - i0) // tqt  # tokens before the key see nothing of it
            cnt = max(0, -(-(m - i0) // tqt) - first)
            for _ in range(Hkv):
                out += [(min(2, tiles - t), cnt * (p + 1) // parts - cnt * p // parts, parts) for p in range(parts)]
    return out


def _blocks(units):
    """The units with something to multiply of each block."""
    n = torch.cuda.get_device_properties(0).multi_processor_count
    return [[u for u in units[i::n] if u[1] > 0] for i in range(min(n, len(units)))]


def _reference(a, w, observe, decay):
    """(weights, bound, places updated) as in test_paged_weigh_gpu, a sequence at a time (64 bits, on the GPU)."""
    c = a["c"]
    k = ref.values(c["k_pages"], c["k_exp"])
    PS, H = k.shape[2], k.shape[1]
    cu, lens, table = a["cu"].tolist(), a["lens"].tolist(), a["table"].long()
    out, bound, hit = w.double().clone(), torch.zeros(w.shape, dtype=torch.float64), torch.zeros(w.shape, dtype=torch.bool)
    for b, n in enumerate(lens):
        m = cu[b + 1] - cu[b]
        if m == 0:
            continue
        j = torch.arange(n)
        p = torch.arange(n - m, n)[:, None]
        see = (j <= p) & ((j > p - a["window"]) | (j < a["sinks"]) if a["window"] else torch.tensor(True))
        j = see.any(0).nonzero()[:, 0]
        see = see[:, j].cuda()
        at = (table[b][j // PS], slice(None), j % PS)
        kh = k[at].cuda().transpose(0, 1)                                                   # [H, keys, D]
        i0 = max(0, m - observe) if observe else 0
        q = a["q"][cu[b] + i0:cu[b + 1]].cuda().double().view(m - i0, H, -1, D).transpose(0, 1)  # [H, tokens, G, D]
        G = q.shape[2]
        s = (q.reshape(H, -1, D) @ kh.transpose(1, 2)).view(H, m - i0, G, -1) * a["scale"]
        hide = ~see[None, i0:, None]
        soft = torch.softmax(s.masked_fill(hide, -torch.inf), -1)
        d = (q.abs().reshape(H, -1, D) @ kh.abs().transpose(1, 2)).view(H, m - i0, G, -1).masked_fill(hide, 0.0).amax(-1)
        d = 2.0 ** -24 * 140 * d * abs(a["scale"])
        rel = 2 * torch.expm1(d) + see[i0:].sum(1).double()[None, :, None] ** 0.5 * 2.0 ** -22 + 2.0 ** -19
        add, off = soft.sum((1, 2)).T.cpu(), (soft * rel[..., None]).sum((1, 2)).T.cpu()
        old = torch.where((j >= n - m)[:, None] | torch.tensor(decay == 0.0), torch.zeros(len(j), H, dtype=torch.float64), decay * w.double()[at])
        out[at] = old + add
        bound[at] = off + add * (m - i0) * G * 2.0 ** -24 + 2.0 ** -23 * (old.abs() + add) + 1e-30
        hit[at] = True
    return out, bound, hit


def _check(vq, a, observe=0, decay=1.0, seed=0):  # noqa: F811
    w = _weights(a, seed, decay)
    first = w.cuda()
    out = _run(vq, a, first, observe, decay)
    plain = vq.vq_paged_attend(a["q"].cuda(), _cuda(a["c"]), a["table"].cuda(), a["cu"].cuda(), a["lens"].cuda(), a["scale"],
                               max_q=a["max_q"], window=a["window"], sinks=a["sinks"])
    _clean(vq)
    assert torch.equal(out, plain)
    want, bound, hit = _reference(a, w, observe, decay)
    got = first.cpu()
    assert torch.equal(got.view(torch.int32)[~hit], w.view(torch.int32)[~hit])
    assert torch.isfinite(got[hit]).all()
    err = (got.double() - want).abs()[hit]
    assert bool((err <= bound[hit]).all()), "largest excess %g, error %g" % (float((err - bound[hit]).max()), float(err.max()))
    for _ in range(3):
        g = w.cuda()
        assert torch.equal(_run(vq, a, g, observe, decay), out)
        assert torch.equal(g.view(torch.int32), first.view(torch.int32))
    _clean(vq)


def _turns(units):
    """Blocks that take units of one and of two key tiles, three at least."""
    return sum(len(b) > 2 and len({u[0] for u in b}) == 2 for b in _blocks(units))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("B,Hkv,PS,observe,decay", [(400, 1, 16, 0, 1.0), (300, 2, 64, 1, 0.0), (64, 7, 32, 16, 0.9), (64, 8, 128, 32, 1.0),
                                                    (80, 8, 16, 0, 0.5)])
def test_prompts_of_a_batch(vq, dtype, cache, B, Hkv, PS, observe, decay):  # noqa: F811
    """Prompts of 1 to 400 tokens, four query heads to a kv head."""
    lens = [random.Random(B + i).randint(1, 400) for i in range(B)]
    a = _case(vq, lens, lens, Hkv, 4, PS, dtype, cache, seed=B + Hkv)
    units = _units(a, Hkv, 4, observe)
    assert len(units) > 2 * torch.cuda.get_device_properties(0).multi_processor_count and _turns(units) > 10
    _check(vq, a, observe, decay)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_short_chunks_and_single_tokens(vq, dtype, cache):  # noqa: F811
    """Chunks of 8 tokens over 100 to 1000, single tokens among them."""
    r = random.Random(3)
    lens = [r.randint(100, 1000) for _ in range(140)]
    news = [1 if i % 5 == 2 else 8 for i in range(140)]
    a = _case(vq, news, lens, 4, 4, 16, dtype, cache, seed=4)
    units = _units(a, 4, 4, 0)
    assert _turns(units) > 10
    _check(vq, a, 0, 0.97)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_windows_and_first_tokens_of_a_batch(vq, dtype, cache):  # noqa: F811
    r = random.Random(5)
    lens = [r.randint(1, 700) for _ in range(60)]
    news = [min(n, r.choice([1, 9, 40, 300])) for n in lens]
    for window, sinks in ((130, 4), (300, 0)):
        _check(vq, _case(vq, news, lens, 8, 4, 32, dtype, cache, window=window, sinks=sinks, seed=window), 25, 0.9)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("GQ,Hkv,news,lens,observe,parts", [
    (16, 1, [256, 3], [300, 20], 0, {1, 2}),
    (16, 2, [1024], [1024], 0, {8}),
    (16, 1, [300, 1000, 40], [300, 1100, 700], 0, {2, 7, 1}),
    (16, 3, [1100, 1, 500], [1300, 50, 900], 530, {4, 3}),
    (5, 8, [900, 130, 2], [901, 260, 2], 0, {2, 1})])
def test_sums_in_several_parts(vq, dtype, cache, GQ, Hkv, news, lens, observe, parts):  # noqa: F811
    """Query tiles that the parts divide, and that they do not; parts with nothing to add."""
    a = _case(vq, news, lens, Hkv, GQ, 64, dtype, cache, seed=sum(news))
    assert {u[2] for u in _units(a, Hkv, GQ, observe)} == parts
    _check(vq, a, observe, 0.5)
