"""Attention over an 8-bit paged cache whose rows have exponents far apart, and
zero rows among them, against a plain 64-bit implementation.

The bound on an output of one query row, with weights p_j (sum 1), values
v_j = 2^b_j V_j (|V_j| <= 448) and scores s_j:

  * a weight enters the value product in fp16 as p_j 2^b_j times a power of two
    that brings the largest of the row to 2^7 or more (2^-1 or more in a chunk,
    whose tiles share an exponent where theirs lie within 2^8): it is off by
    2^-11 of itself, or, below 2^-14, by 2^-25.  So
      sum_j 2^-11 p_j |v_j|  +  2^-32 (2^-24) max_i(p_i 2^b_i) sum_j |V_j|;
  * a score, a sum of 128 exact products in 32 bits, is off by
    d_j = 140 * 2^-24 scale |q| . |k_j|, and score and exponential together by
    2^-20 more: sum_j p_j e_j |v_j| in the numerator, sum_j p_j e_j of the output
    in the denominator, with e_j = exp(d_j + 2^-20) - 1;
  * the sums over n keys and the division: sqrt(n) 2^-22 of both;
  * the output's own rounding.

A zero row counts in the denominator alone, whatever exponent it is stored with.
"""
import math

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


def _case(rows, news, GQ, Hkv, PS, dtype, window=0, sinks=0, seed=0):
    """A call on the CPU; rows(b, gen) gives the keys and values of sequence b, float64
    [n, Hkv, 128].  Queries lie along the first coordinate, about 8 of it."""
    gen = torch.Generator().manual_seed(seed)
    B = len(news)
    kv = [rows(b, gen) for b in range(B)]
    lens = [k.shape[0] for k, _ in kv]
    width = max(-(-n // PS) for n in lens)
    count = sum(-(-n // PS) for n in lens)
    table = torch.full((B, width), -1, dtype=torch.int32)
    perm = torch.randperm(count, generator=gen).to(torch.int32)
    c = {}
    for x in "kv":
        c[x + "_pages"] = torch.full((count, Hkv, PS, D), 0x7F, dtype=torch.uint8)
        c[x + "_exp"] = torch.full((count, Hkv, PS), 255, dtype=torch.uint8)
    at = 0
    for b in range(B):
        n = -(-lens[b] // PS)
        table[b, :n] = perm[at:at + n]
        at += n
        j = torch.arange(lens[b])
        pg, off = table[b][j // PS].long(), j % PS
        for x, d in zip("kv", kv[b]):
            code, e = ref.quantise(d)
            c[x + "_pages"][pg, :, off] = code
            c[x + "_exp"][pg, :, off] = e
    T, Hq = sum(news), Hkv * GQ
    q = torch.randn(T, Hq, D, generator=gen)
    q[:, :, 0] = 8.0 + 0.25 * q[:, :, 0]
    return dict(q=q.to(dtype), c=c, table=table, cu=torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32),
                lens=torch.tensor(lens, dtype=torch.int32), window=window, sinks=sinks, scale=D ** -0.5, max_q=max(news),
                PS=PS, Hkv=Hkv)


def _reference(a, floor):
    """(out, bound before the output's rounding); floor: 2^-32 or 2^-24, see above."""
    q = a["q"].double()
    T, Hq, _ = q.shape
    Hkv, PS = a["Hkv"], a["PS"]
    G = Hq // Hkv
    codes = {x: torch.from_numpy(ref.E4M3)[a["c"][x + "_pages"].long()] for x in "kv"}
    exps = {x: a["c"][x + "_exp"].double() - 127 for x in "kv"}
    out, bound = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    for b in range(len(a["lens"])):
        n = int(a["cu"][b + 1] - a["cu"][b])
        for i in range(n):
            p = int(a["lens"][b]) - n + i
            j = torch.arange(p + 1)
            if a["window"]:
                j = j[(j > p - a["window"]) | (j < a["sinks"])]
            pg, off = a["table"][b][j // PS].long(), j % PS
            t = int(a["cu"][b]) + i
            for h in range(Hkv):
                K = codes["k"][pg, h, off] * torch.exp2(exps["k"][pg, h, off])[:, None]
                V, e = codes["v"][pg, h, off], exps["v"][pg, h, off].clone()
                e[(V == 0).all(1)] = -32
                v = V * torch.exp2(e)[:, None]
                x = q[t, h * G:(h + 1) * G]
                w = torch.softmax(x @ K.T * a["scale"], 1)
                o = w @ v
                d = torch.expm1(140 * 2.0 ** -24 * a["scale"] * (x.abs() @ K.abs().T) + 2.0 ** -20)
                s = len(j) ** 0.5 * 2.0 ** -22
                top = (w * torch.exp2(e)).amax(1, keepdim=True)
                err = (w * (2.0 ** -11 + d + s)) @ v.abs() + floor * top * V.abs().sum(0)
                err = err + ((w * d).sum(1, keepdim=True) + s) * o.abs()
                out[t, h * G:(h + 1) * G], bound[t, h * G:(h + 1) * G] = o, err
    return out, bound


def _check(vq, a, floor):
    c = {k: v.cuda() for k, v in a["c"].items()}
    for x in "kv":
        c[x + "_pages"] = c[x + "_pages"].view(E4M3)
    got = vq.vq_paged_attend(a["q"].cuda(), c, a["table"].cuda(), a["cu"].cuda(), a["lens"].cuda(), a["scale"],
                             max_q=a["max_q"], window=a["window"], sinks=a["sinks"])
    torch.cuda.synchronize()
    assert vq.vq_device_error() == 0
    o, bound = _reference(a, floor)
    g = got.cpu().double()
    least = 2.0 ** -25 if a["q"].dtype == F16 else 0.0  # half of the output type's least step
    tol = bound + ref.U16[a["q"].dtype] * (o.abs() + bound) + least
    assert torch.isfinite(g).all()
    err = (g - o).abs()
    assert bool((err <= tol).all()), "error %.2f times the bound" % float((err / tol).nan_to_num(0.0).max())


def _first_zero(n, Hkv, size, score):
    """Keys of unit size and values of `size`; token 0 has a zero value row and a
    key with `score` above the others (in units of the softmax's exponent)."""
    def rows(b, gen):
        k = torch.randn(n, Hkv, D, generator=gen).double() * 0.5
        v = torch.randn(n, Hkv, D, generator=gen).double() * size
        k[:, :, 0] = 0.0
        k[0] = 0.0
        k[0, :, 0] = score / 8 / D ** -0.5
        v[0] = 0.0
        return k, v
    return rows


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size,score", [(1.0, 8.0), (1e-2, 11.0), (1e-3, 9.0), (1e-4, 9.0)])
@pytest.mark.parametrize("GQ", [1, 4, 12])
def test_a_zero_value_row_that_takes_attention_single_tokens(vq, dtype, size, score, GQ):
    _check(vq, _case(_first_zero(1100, 2, size, score), [1, 1], GQ, 2, 16, dtype, seed=1), 2.0 ** -32)
    _check(vq, _case(_first_zero(900, 1, size, score), [1], GQ, 1, 64, dtype, window=300, sinks=1, seed=2), 2.0 ** -32)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size,score", [(1.0, 8.0), (1e-2, 11.0), (1e-3, 9.0), (1e-4, 9.0)])
@pytest.mark.parametrize("PS", [16, 128, 256])
def test_a_zero_value_row_that_takes_attention_chunks(vq, dtype, size, score, PS):
    _check(vq, _case(_first_zero(700, 1, size, score), [40], 4, 1, PS, dtype, seed=3), 2.0 ** -24)
    _check(vq, _case(_first_zero(900, 1, size, score), [70, 33], 2, 1, PS, dtype, window=200, sinks=1, seed=4),
           2.0 ** -24)


def _many_zero(n, Hkv, size):
    """A third of the value rows, and whole stretches of them, are zero."""
    def rows(b, gen):
        k = torch.randn(n, Hkv, D, generator=gen).double()
        v = torch.randn(n, Hkv, D, generator=gen).double() * size
        v[torch.rand(n, Hkv, generator=gen) < 0.33] = 0.0
        v[128:256] = 0.0
        v[300:310] = -0.0
        return k, v
    return rows


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [0.3, 1e-4, 0.0])
def test_zero_value_rows_everywhere_single_tokens(vq, dtype, size):
    _check(vq, _case(_many_zero(700, 2, size), [1, 1], 4, 2, 32, dtype, seed=5), 2.0 ** -32)
    _check(vq, _case(_many_zero(300, 1, size), [1], 4, 1, 16, dtype, seed=7), 2.0 ** -32)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [0.3, 1e-4, 0.0])
def test_zero_value_rows_everywhere_chunks(vq, dtype, size):
    _check(vq, _case(_many_zero(600, 2, size), [50, 130], 3, 2, 32, dtype, seed=6), 2.0 ** -24)
    _check(vq, _case(_many_zero(300, 1, size), [60], 4, 1, 16, dtype, seed=7), 2.0 ** -24)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size,score", [(1e-2, 11.0), (1e-4, 9.0)])
def test_a_zero_value_row_in_the_middle_of_a_share(vq, dtype, size, score):
    """Several items and many tiles for every block, so that blocks meet the zero
    row at an item's start, after others that they finished: items of two query
    tiles and of one, whole ones and cut ones."""
    _check(vq, _case(_first_zero(2100, 8, size, score), [150, 20, 70, 40], 4, 8, 64, dtype, seed=14), 2.0 ** -24)


def _spread(n, Hkv, lo, hi, keys=0):
    """Value rows of sizes 2^lo to 2^hi whose weights fall as their sizes grow, so
    that a row of any size carries some of the output; with `keys`, key rows down
    to 2^-keys and zero ones too."""
    def rows(b, gen):
        r = torch.randint(lo, hi + 1, (n, Hkv), generator=gen).double()
        v = torch.randn(n, Hkv, D, generator=gen).double() * torch.exp2(r)[..., None]
        k = torch.randn(n, Hkv, D, generator=gen).double() * 0.1
        k[:, :, 0] = -r * math.log(2) / 8 / D ** -0.5
        if keys:
            small = torch.rand(n, Hkv, generator=gen) < 0.3
            k[small] *= torch.exp2(-torch.randint(0, keys + 1, (n, Hkv), generator=gen).double())[small][:, None]
            k[torch.rand(n, Hkv, generator=gen) < 0.05] = 0.0
        return k, v
    return rows


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lo,hi", [(-3, 3), (-8, 1), (-16, 0), (-20, 6), (-30, 4)])
@pytest.mark.parametrize("keys", [0, 28])
def test_rows_of_any_size_single_tokens(vq, dtype, lo, hi, keys):
    if dtype == F16 and hi - lo > 24:
        lo = hi - 24  # (smaller outputs are below fp16's)
    _check(vq, _case(_spread(600, 2, lo, hi, keys), [1, 1], 4, 2, 16, dtype, seed=8), 2.0 ** -32)
    _check(vq, _case(_spread(600, 1, lo, hi, keys), [1], 16, 1, 128, dtype, seed=9), 2.0 ** -32)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lo,hi", [(-3, 3), (-8, 1), (-16, 0), (-20, 6), (-30, 4)])
@pytest.mark.parametrize("keys", [0, 28])
def test_rows_of_any_size_chunks(vq, dtype, lo, hi, keys):
    if dtype == F16 and hi - lo > 24:
        lo = hi - 24
    _check(vq, _case(_spread(500, 1, lo, hi, keys), [45, 300], 4, 1, 16, dtype, seed=10), 2.0 ** -24)
    _check(vq, _case(_spread(700, 2, lo, hi, keys), [130], 2, 2, 128, dtype, window=150, sinks=20, seed=11), 2.0 ** -24)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("news", [[1], [40]])
def test_a_small_row_carries_the_weight(vq, dtype, news):
    """One value row, from 2^-20 of its neighbour's size down to 2^-30, has nearly all weight."""
    for down in (20, 24, 25, 26, 30):
        def rows(b, gen):
            k = torch.randn(200, 1, D, generator=gen).double() * 0.1
            v = torch.randn(200, 1, D, generator=gen).double() * 2.0 ** (10 - down)
            k[:, :, 0] = -40 / 8 / D ** -0.5
            k[37, :, 0] = 40 / 8 / D ** -0.5
            v[38] *= 2.0 ** down
            return k, v
        _check(vq, _case(rows, news, 4, 1, 32, dtype, seed=12), 2.0 ** -32 if news == [1] else 2.0 ** -24)


@pytest.mark.parametrize("news", [[1, 1], [33, 1]])
def test_small_scales_over_codes(vq, news):
    """Scales so small that their product with a key's exponent has no 32-bit
    number: plain means, as scale 0."""
    def rows(b, gen):
        return torch.randn(150, 1, D, generator=gen).double() * 1e-9, torch.randn(150, 1, D, generator=gen).double()
    a = _case(rows, news, 4, 1, 16, F16, seed=13)
    for scale in (0.0, 1e-30, 1e-36, 1e-45):
        _check(vq, dict(a, scale=scale), 2.0 ** -24)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_repeated_calls_agree_where_blocks_change_over(vq, dtype):
    """Blocks that meet a tile to be taken key by key go on from the item that is
    furthest behind, which depends on their warps' timing; the outputs do not.  A
    zero row in the middle, at an item's start, and sizes far apart in a few tiles."""
    def rows(b, gen):
        k, v = _first_zero(2300, 8, 0.01, 9.0)(b, gen)
        if b % 2:
            v[0] = v[1]
            v[1500, ::3] = 0.0
            v[700:720] *= 2.0 ** 14
        return k, v
    a = _case(rows, [150, 90, 40, 200], 4, 8, 32, dtype, seed=15)
    c = {k: v.cuda() for k, v in a["c"].items()}
    for x in "kv":
        c[x + "_pages"] = c[x + "_pages"].view(E4M3)
    args = (a["q"].cuda(), c, a["table"].cuda(), a["cu"].cuda(), a["lens"].cuda(), a["scale"])
    first = vq.vq_paged_attend(*args, max_q=a["max_q"])
    noise = torch.randn(4096, 4096, device="cuda")
    for i in range(20):
        if i % 2:
            noise @ noise  # (other clocks and cache contents)
        assert torch.equal(vq.vq_paged_attend(*args, max_q=a["max_q"]), first)
    assert vq.vq_device_error() == 0
