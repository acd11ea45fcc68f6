"""A bf16 paged cache read back as fp16, the type of the codecs."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
D = 128
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def vq():
    from kv_cache_quantization_turboquantrvq_gb300 import api, build
    build.build()
    api.lib()
    return api


@pytest.mark.parametrize("PS,H,S", [(16, 2, 1), (32, 3, 77), (256, 1, 130)])
def test_every_value_rounded_once(vq, PS, H, S):
    """Bit for bit against the values rounded to nearest even: all finite bf16
    numbers, those past fp16's range (infinite) and below its least among them."""
    B, width = 3, -(-200 // PS)
    bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16).view(BF16)
    gen = torch.Generator().manual_seed(PS)
    pages = bits[torch.randint(0, 65536, (B * width, 2, H, PS, D), generator=gen)]
    pages = torch.where(torch.isnan(pages), torch.zeros_like(pages), pages)
    c = vq.paged_cache(B * width, H, PS, BF16)
    c["k_pages"].copy_(pages[:, 0])
    c["v_pages"].copy_(pages[:, 1])
    table = torch.randperm(B * width, generator=gen).to(torch.int32).view(B, width)
    lens, first = [200, S, 0], [3, 0, 0]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k, v = vq.vq_paged_gather(c, table.cuda(), i32(lens), S, first=i32(first), dtype=F16)
    assert vq.vq_device_error() == 0
    for got, x in ((k, 0), (v, 1)):
        want = torch.zeros(B, H, S, D, dtype=F16)
        for b in range(B):
            for i in range(S):
                t = first[b] + i
                if t < lens[b]:
                    want[b, :, i] = pages[int(table[b][t // PS]), x, :, t % PS].to(F16)
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))


def test_a_bf16_cache_reaches_both_codecs(vq):
    """Values that fp16 holds exactly: the codecs' storage is that of an fp16 cache."""
    gen = torch.Generator("cuda").manual_seed(1)
    kv = torch.randn(2, 256, 2, D, generator=gen, device="cuda").to(BF16)
    slots = torch.arange(256, device="cuda")
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(1, 16)
    lens = torch.tensor([256], dtype=torch.int32, device="cuda")
    stored = []
    for t in (BF16, F16):
        c = vq.paged_cache(16, 2, 16, t)
        vq.vq_paged_append(kv[0].to(t), kv[1].to(t), c, slots)
        k, v = vq.vq_paged_gather(c, table, lens, 256, dtype=F16)
        c1, b1, c2, b2 = vq.vq_rvq_codebook(D, 2)
        stored.append(list(vq.vq_kivi_quant_pack(k, v, 2, 32, 0).values()) + list(vq.vq_rvq_encode_pack(k, 2, c1, b1, c2, b2)))
    assert vq.vq_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(*stored))


@pytest.mark.parametrize("window", [0, 100])
def test_the_example_serves_from_a_bf16_cache(vq, window):
    """examples/serve_paged.py with bf16 tensors: weights, outputs and the plain side's
    inputs are rounded to 2^-8 of each; 0.02 leaves room for both products."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import serve_paged
    got, want, pages, done = serve_paged.serve(prompts=(300, 177, 512, 130), steps=8, cache="bfloat16", window=window, seed=3)
    assert float((got - want).norm() / want.norm()) < 0.02
    if not window:
        kivi, rvq, tokens = serve_paged.compress(pages, done)
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        k0, v0 = vq.vq_paged_gather(pages.cache, pages.device_table(), lens, tokens, dtype=F16)
        k, v = vq.vq_kivi_unpack_dequant(kivi, 4, 8, tokens, 2, 32)
        for a, b in ((k, k0), (v, v0)):
            assert float((a.float() - b.float()).norm() / b.float().norm()) < 0.6  # 2-bit codes
    assert vq.vq_device_error() == 0
