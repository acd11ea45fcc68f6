"""Plain 64-bit implementation of the paged-cache operators (test infrastructure).

Written from the definitions, on the CPU, for tests/test_paged_gpu.py and
tests/test_paged_host.py: e4m3 codes by searching the 256 values, attention one
query row at a time over the keys that the row sees (so what a masked place
holds cannot reach it).
"""
import math

import numpy as np
import torch

D = 128
U16 = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def _e4m3_value(code):
    s, e, m = code >> 7, (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -x if s else x


E4M3 = np.array([_e4m3_value(c) for c in range(256)])


def quantise(x):
    """(codes uint8, exponent + 127 uint8) of rows x [..., 128]."""
    x = x.double().numpy()
    top = np.abs(x).max(-1)
    e = np.minimum(np.searchsorted(448 * 2.0 ** np.arange(-32, 65), top), 96) - 32  # the least that holds top
    e[top == 0] = 0
    y = np.clip(x / (2.0 ** e)[..., None], -448, 448)
    pos = E4M3[:127]  # ascending non-negative values
    a = np.abs(y)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == pos[hi], hi, code)
    code = code + 128 * np.signbit(y)
    return torch.from_numpy(code.astype(np.uint8)), torch.from_numpy((e + 127).astype(np.uint8))


def values(pages, exps):
    """Float64 values of a cache's pages (uint8 codes with exponents, or 16-bit)."""
    if exps is None:
        return pages.double()
    v = torch.from_numpy(E4M3)[pages.view(torch.uint8).long()]
    return v * torch.from_numpy(2.0 ** (exps.numpy().astype(np.float64) - 127))[..., None]


def attend(q, k, v, table, cu, lens, scale, window, sinks, w_step):
    """(out, bound) float64 [T, Hq, 128] for pages' values k, v [NP, Hkv, PS, 128].

    bound: what the outputs may be off before their own rounding.  The weights
    are rounded to w_step relative (and to multiples of 2^-24 below 2^-14, where
    the largest is at least 2^7); a score's sum of 128 products, its scaling
    and the exponential are off by at most d, which moves weight and sum by
    e^d - 1 each; the sums over n keys, the merge and the division by a few 2^-24 more.
    """
    T, Hq, _ = q.shape
    Hkv, PS = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    bound = torch.zeros(T, Hq, D, dtype=torch.float64)
    q = q.double()
    for b in range(len(lens)):
        n = int(cu[b + 1]) - int(cu[b])
        L = int(lens[b])
        for i in range(n):
            p = L - n + i
            j = torch.arange(0, max(p + 1, 0))
            if window:
                j = j[(j > p - window) | (j < sinks)]
            if len(j) == 0:
                continue
            pg = table[b].long()[j // PS]
            kk, vv = k[pg, :, j % PS], v[pg, :, j % PS]  # [n, Hkv, D]
            t = int(cu[b]) + i
            kh, vh = kk.transpose(0, 1), vv.transpose(0, 1)  # [Hkv, n, D]
            qt = q[t].view(Hkv, G, D).transpose(1, 2)        # [Hkv, D, G]
            w = torch.softmax(kh @ qt * scale, 1).transpose(1, 2)
            out[t] = (w @ vh).reshape(Hq, D)
            d = 2.0 ** -24 * 140 * (kh.abs() @ qt.abs()).amax(1) * abs(scale) + 2.0 ** -20  # [Hkv, G]
            small = len(j) * 2.0 ** -32 * vh.abs().amax(1, keepdim=True)
            u = w_step + 2 * torch.expm1(d) + len(j) ** 0.5 * 2.0 ** -22
            bound[t] = (u[..., None] * (w @ vh.abs()) + small).reshape(Hq, D)
    return out, bound
