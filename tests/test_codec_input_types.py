"""The codecs read fp16: inputs of other floating types are refused before they
reach the library (no GPU: a library that fails when it is called)."""
import pytest

torch = pytest.importorskip("torch")


class NoLibrary:
    def __getattr__(self, name):
        raise AssertionError("%s was called" % name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float8_e4m3fn])
def test_other_types_than_fp16_are_refused(monkeypatch, dtype):
    from kv_cache_quantization_turboquantrvq_gb300 import api
    books = api.vq_rvq_codebook(128, 2)
    monkeypatch.setattr(api, "_lib", NoLibrary())
    x, h = torch.zeros(1, 2, 64, 128).to(dtype), torch.zeros(1, 2, 64, 128).half()
    for call in (lambda: api.vq_rvq_encode_pack(x, 2, *books),
                 lambda: api.vq_kivi_quant_pack(x, None, 2, 32, 0), lambda: api.vq_kivi_quant_pack(h, x, 2, 32, 0),
                 lambda: api.vq_flush_decode(x, h, 0, kivi=dict(bits=2, group=32)),
                 lambda: api.vq_flush_decode(h, x, 0, kivi=dict(bits=2, group=32))):
        with pytest.raises(ValueError):
            call()
