"""Serving with a paged cache in front of the codecs.

One attention layer (random weights, grouped-query heads) serves a few prompts:
each step takes a chunk of every prompt that is not finished and one token of
every sequence that decodes, all in one batch.

  1. the new tokens' keys and values go into pages          vq_paged_append
  2. the new tokens attend over the pages                   vq_paged_attend
     (causal; with a window, pages that fall behind it are given back)
  3. at the end the oldest whole blocks of 128 tokens come   vq_paged_gather
     out of the pages and are compressed                     vq_kivi_quant_pack,
                                                             vq_rvq_encode_pack

Run: python examples/serve_paged.py [--cache e4m3|float16|bfloat16] [--window N]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kv_cache_quantization_turboquantrvq_gb300 import api, build  # noqa: E402

D = 128


class Pages:
    """Pages of one layer: the pool, the free ones, and which page holds which tokens."""

    def __init__(self, pages, heads, page_size, dtype, sequences):
        self.cache = api.paged_cache(pages, heads, page_size, dtype)
        self.size = page_size
        self.free = list(range(pages))[::-1]
        self.table = [[] for _ in range(sequences)]

    def slots(self, b, first, count):
        """Places for tokens first .. first + count - 1 of sequence b (pages taken as needed)."""
        while len(self.table[b]) * self.size < first + count:
            self.table[b].append(self.free.pop())
        return [self.table[b][t // self.size] * self.size + t % self.size for t in range(first, first + count)]

    def release(self, b, below, keep):
        """Give back the pages of sequence b whose tokens all lie in [keep, below)."""
        for p, page in enumerate(self.table[b]):
            if page >= 0 and p * self.size >= keep and (p + 1) * self.size <= below:
                self.free.append(page)
                self.table[b][p] = -1

    def device_table(self):
        width = max(1, max(map(len, self.table)))
        return torch.tensor([r + [-1] * (width - len(r)) for r in self.table], dtype=torch.int32, device="cuda")


def serve(prompts=(300, 77, 512, 1), steps=20, chunk=128, heads=8, group=4, cache="e4m3", window=0, sinks=4, page_size=16,
          seed=0):
    """Runs the loop; returns (outputs of the last step, the same from plain
    attention over all keys and values, number of free pages)."""
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = torch.bfloat16 if cache == "bfloat16" else torch.float16
    width = heads * group * D
    hidden = 256
    w = torch.randn(hidden, (heads * group + 2 * heads) * D, generator=gen, device="cuda", dtype=dt) / math.sqrt(hidden)
    wo = torch.randn(width, hidden, generator=gen, device="cuda", dtype=dt) / math.sqrt(width)
    total = sum(p + steps for p in prompts)
    pages = Pages(total // page_size + 2 * len(prompts), heads, page_size,
                  torch.float8_e4m3fn if cache == "e4m3" else dt, len(prompts))
    done = [0] * len(prompts)  # tokens in the cache
    x = [torch.randn(p, hidden, generator=gen, device="cuda", dtype=dt) for p in prompts]  # tokens to come
    kept = [[] for _ in prompts]  # all keys and values, for the comparison
    while min(d - p for d, p in zip(done, prompts)) < steps:
        # this step's tokens: a chunk of a prompt, or the one that the last step gave
        new = [min(chunk, x[b].shape[0]) if done[b] < prompts[b] + steps else 0 for b in range(len(prompts))]
        batch = torch.cat([x[b][:n] for b, n in enumerate(new)])
        T = batch.shape[0]
        qkv = batch @ w
        q = qkv[:, :width].view(T, heads * group, D)
        k = qkv[:, width:width + heads * D].view(T, heads, D)
        v = qkv[:, width + heads * D:].view(T, heads, D)
        slots = sum((pages.slots(b, done[b], n) for b, n in enumerate(new)), [])
        api.vq_paged_append(k, v, pages.cache, torch.tensor(slots, device="cuda"))
        cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        lens = torch.tensor([d + n for d, n in zip(done, new)], dtype=torch.int32, device="cuda")
        out = api.vq_paged_attend(q, pages.cache, pages.device_table(), cu, lens, 1 / math.sqrt(D), max_q=max(new),
                                  window=window, sinks=sinks)
        y = out.view(T, width) @ wo
        last = []
        for b, n in enumerate(new):
            t = int(cu[b])
            kept[b].append((k[t:t + n], v[t:t + n]))
            x[b] = x[b][n:]
            done[b] += n
            if n and x[b].shape[0] == 0:
                x[b] = y[t + n - 1:t + n]  # decoding: the next token is this one's output
            if window:
                pages.release(b, done[b] - window + 1, -(-sinks // page_size) * page_size)
            if n:
                last.append((b, q[t + n - 1], out[t + n - 1]))
    # plain attention of the last step's tokens over everything that was ever cached
    got, want = [], []
    for b, qb, ob in last:
        kb, vb = (torch.cat([c[i] for c in kept[b]]).float().transpose(0, 1) for i in (0, 1))  # [heads, n, D]
        s = torch.einsum("hgd,hnd->hgn", qb.float().view(heads, group, D), kb) / math.sqrt(D)
        n = kb.shape[1]
        j = torch.arange(n, device="cuda")
        if window:
            s = s.masked_fill((j <= n - 1 - window) & (j >= sinks), float("-inf"))
        want.append(torch.einsum("hgn,hnd->hgd", s.softmax(-1), vb).reshape(heads * group, D))
        got.append(ob.float())
    return torch.stack(got), torch.stack(want), pages, done


def compress(pages, done, block=128):
    """The whole blocks of every sequence out of the pages and through both codecs:
    (KIVI storage, RVQ storage of the keys, tokens compressed of each sequence)."""
    tokens = min(done) // block * block
    if tokens == 0:
        return None, None, 0
    lens = torch.tensor(done, dtype=torch.int32, device="cuda")
    k, v = api.vq_paged_gather(pages.cache, pages.device_table(), lens, tokens, dtype=torch.float16)
    kivi = api.vq_kivi_quant_pack(k, v, bits=2, group=32, residual_length=0)
    c1, b1, c2, b2 = api.vq_rvq_codebook(D, 2)
    return kivi, api.vq_rvq_encode_pack(k, 2, c1, b1, c2, b2), tokens


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--cache", default="e4m3", choices=["e4m3", "float16", "bfloat16"])
    ap.add_argument("--window", type=int, default=0)
    a = ap.parse_args()
    build.build()
    got, want, pages, done = serve(prompts=(300, 177, 512, 130), cache=a.cache, window=a.window)
    off = float((got - want).norm() / want.norm())
    print("tokens cached %s, pages free %d" % (done, len(pages.free)))
    print("last step against plain attention over uncompressed keys and values: relative difference %.4f" % off)
    if not a.window:
        kivi, rvq, tokens = compress(pages, done)
        print("compressed the first %d tokens of each sequence: KIVI %d bytes, RVQ keys %d bytes" % (
            tokens, sum(t.numel() * t.element_size() for t in kivi.values()),
            sum(t.numel() * t.element_size() for t in rvq)))
    assert api.vq_device_error() == 0


if __name__ == "__main__":
    main()
