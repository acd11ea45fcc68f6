"""Lengths and token offsets on the device that make no sense: attention reports
them, stays inside its buffers and computes the sequences that make sense."""
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


def _run(vq, T, cu, lens, max_q, pages=8, PS=16, GQ=4):
    """One kv head, sequences of `pages` pages each, all of one pool."""
    B = len(lens)
    gen = torch.Generator("cuda").manual_seed(T)
    c = vq.paged_cache(pages * B, 1, PS, torch.float16)
    kv = torch.randn(2, pages * B * PS, 1, D, generator=gen, device="cuda").half()
    vq.vq_paged_append(kv[0], kv[1], c, torch.arange(pages * B * PS, device="cuda"))
    table = torch.arange(pages * B, dtype=torch.int32, device="cuda").view(B, pages)
    q = torch.randn(T, GQ, D, generator=gen, device="cuda").half()
    room = torch.full((T + 64, GQ, D), 7.0, dtype=torch.float16, device="cuda")
    out = room[32:T + 32]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    vq.vq_paged_attend(q, c, table, i32(cu), i32(lens), D ** -0.5, max_q, out=out)
    code = vq.vq_device_error()
    assert bool((room[:32] == 7).all()) and bool((room[T + 32:] == 7).all())
    return out, code


@pytest.mark.parametrize("T,cu,max_q", [(3, [0, 1, 2, 3], 1), (82, [0, 1, 41, 82], 41)])
def test_a_length_past_the_table_is_reported(vq, T, cu, max_q):
    want, code = _run(vq, T, cu, [100, 128, 60], max_q)
    assert code == 0
    for bad in (129, 10 ** 6, 2 ** 31 - 1, -1):
        got, code = _run(vq, T, cu, [100, bad, 60], max_q)
        assert code == vq.VQ_DEVERR_BAD_OFFSET
        assert torch.equal(got[:cu[1]], want[:cu[1]]) and torch.equal(got[cu[2]:], want[cu[2]:])


def test_a_length_past_the_table_of_a_sequence_without_new_tokens_is_not(vq):
    for T, cu, max_q in ((2, [0, 1, 1, 2], 1), (80, [0, 40, 40, 80], 41)):
        assert _run(vq, T, cu, [100, 10 ** 6, 60], max_q)[1] == 0


@pytest.mark.parametrize("cu", [[0, 3, 1, 4], [0, 4, 0, 4], [-2, 1, 2, 4], [0, 1, 2, 5], [2, 1, 0, -1]])
def test_offsets_of_single_tokens_that_make_no_sense(vq, cu):
    assert _run(vq, 4, cu, [100, 90, 60], 4)[1] == vq.VQ_DEVERR_BAD_OFFSET


@pytest.mark.parametrize("cu", [[0, 120, 0, 120], [0, 60, 30, 120], [-5, 60, 90, 120], [0, 60, 90, 121],
                                [0, 120, 2 ** 31 - 1, 120], [120, 0, 120, 0]])
def test_offsets_of_chunks_that_make_no_sense(vq, cu):
    assert _run(vq, 120, cu, [128, 128, 128], 120)[1] == vq.VQ_DEVERR_BAD_OFFSET


def test_many_sequences_over_the_same_tokens(vq):
    """Offsets that go back and forth name far more chunks than there is room for."""
    B, T = 3000, 200
    out, code = _run(vq, T, [0 if b % 2 == 0 else T for b in range(B + 1)], [128] * B, T)
    assert code == vq.VQ_DEVERR_BAD_OFFSET


def test_offsets_that_end_before_the_tokens_do(vq):
    """Padding tokens behind the last sequence are allowed, and not written."""
    out, code = _run(vq, 90, [0, 40, 41, 70], [100, 90, 60], 41)
    assert code == 0 and bool((out[70:] == 7).all()) and not bool((out[:70] == 7).any())
