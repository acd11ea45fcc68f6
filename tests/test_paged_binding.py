"""What the binding of the paged-cache calls passes on and refuses (no GPU:
stand-ins for CUDA tensors, and a library that keeps its arguments)."""
import pytest

torch = pytest.importorskip("torch")

D = 128
F16, I32, U8 = torch.float16, torch.int32, torch.uint8


class Fake:
    """As much of a CUDA tensor as the binding looks at."""
    next_address = 1 << 40

    def __init__(self, shape, dtype, device=0, contiguous=True):
        self.shape, self.dtype, self._device, self._contiguous = torch.Size(shape), dtype, device, contiguous
        self.is_cuda = device >= 0
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")
        Fake.next_address += 1 << 32
        self._address = Fake.next_address

    def get_device(self):
        return self._device

    def stride(self):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st)

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return self._address

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()


class Library:
    """Keeps what it is called with, and the device that was current."""

    def __init__(self, log, current):
        self.log, self.current = log, current

    def __getattr__(self, name):
        def call(*a):
            self.log.append((name, self.current[-1], a))
            return 0
        return call


@pytest.fixture
def api(monkeypatch):
    from kv_cache_quantization_turboquantrvq_gb300 import api
    log, current = [], [0]
    monkeypatch.setattr(api, "_lib", Library(log, current))

    class On:
        def __init__(self, device):
            self.device = torch.device(device).index if not isinstance(device, int) else device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *a):
            current.pop()

    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(api, "_gpus", 2)
    api._workspace_bytes.clear()
    api.log = log
    yield api
    api._workspace_bytes.clear()
    del api.log


def _cache(device=0, dtype=F16, **other):
    c = {"k_pages": Fake((4, 2, 16, D), dtype, device), "v_pages": Fake((4, 2, 16, D), dtype, device), "k_exp": None, "v_exp": None}
    c.update(other)
    return c


def _attend(api, device=0, **kw):
    a = dict(q=Fake((5, 8, D), F16, device), cache=_cache(device), block_table=Fake((2, 3), I32, device),
             cu_q=Fake((3,), I32, device), lens=Fake((2,), I32, device), scale=0.1, max_q=4, out=Fake((5, 8, D), F16, device),
             workspace=Fake((1 << 20,), U8, device), stream=64)
    a.update(kw)
    return api.vq_paged_attend(**a)


def _append(api, device=0, **kw):
    a = dict(k=Fake((5, 2, D), F16, device), v=Fake((5, 2, D), F16, device), cache=_cache(device),
             slots=Fake((5,), torch.int64, device), stream=64)
    a.update(kw)
    return api.vq_paged_append(**a)


def _gather(api, device=0, **kw):
    a = dict(cache=_cache(device), block_table=Fake((2, 3), I32, device), lens=Fake((2,), I32, device), S_out=7,
             first=Fake((2,), I32, device), k_out=Fake((2, 2, 7, D), F16, device), v_out=Fake((2, 2, 7, D), F16, device), stream=64)
    a.update(kw)
    return api.vq_paged_gather(**a)


def test_calls_that_are_right_reach_the_library(api):
    _append(api)
    _gather(api)
    _attend(api)
    assert [n for n, _, _ in api.log] == ["vq_paged_append", "vq_paged_gather", "vq_paged_attend"]
    assert all(d == 0 for _, d, _ in api.log)


@pytest.mark.parametrize("workspace", [Fake((1 << 20,), U8, -1), Fake((1 << 20,), U8, 0, contiguous=False)])
def test_a_workspace_has_to_be_whole_memory_of_the_gpu(api, workspace):
    with pytest.raises(ValueError):
        _attend(api, workspace=workspace)
    assert not api.log


@pytest.mark.parametrize("call,name,bad", [
    (_append, "k", Fake((5, 2, D), F16, 1)), (_append, "v", Fake((5, 2, D), F16, 1)),
    (_append, "slots", Fake((5,), torch.int64, 1)), (_append, "cache", _cache(0, v_pages=Fake((4, 2, 16, D), F16, 1))),
    (_gather, "block_table", Fake((2, 3), I32, 1)), (_gather, "lens", Fake((2,), I32, 1)),
    (_gather, "first", Fake((2,), I32, 1)), (_gather, "k_out", Fake((2, 2, 7, D), F16, 1)), (_gather, "cache", _cache(1)),
    (_attend, "q", Fake((5, 8, D), F16, 1)), (_attend, "cache", _cache(1)), (_attend, "block_table", Fake((2, 3), I32, 1)),
    (_attend, "cu_q", Fake((3,), I32, 1)), (_attend, "lens", Fake((2,), I32, 1)), (_attend, "out", Fake((5, 8, D), F16, 1)),
    (_attend, "workspace", Fake((1 << 20,), U8, 1))])
def test_tensors_of_two_gpus_are_refused(api, call, name, bad):
    with pytest.raises(ValueError):
        call(api, **{name: bad})
    assert not api.log


@pytest.mark.parametrize("call", [_append, _gather, _attend])
def test_the_tensors_gpu_is_made_current(api, call):
    call(api, device=1)
    assert [d for _, d, _ in api.log] == [1]


def test_the_workspace_is_sized_for_the_tensors_gpu(api, monkeypatch):
    monkeypatch.setattr(api, "_empty", lambda shape, dtype, device, stream, returned=True: Fake((shape,), dtype, 1))
    _attend(api, device=1, workspace=None)
    assert [(n, d) for n, d, _ in api.log] == [("vq_paged_attend_workspace", 1), ("vq_paged_attend", 1)]


@pytest.mark.parametrize("call,name", [(_attend, "max_q"), (_attend, "window"), (_attend, "sinks"), (_gather, "S_out")])
@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 4, 1 << 40])
def test_numbers_past_32_bits_are_refused(api, call, name, value):
    kw = {name: value}
    if name == "S_out":
        kw.update(k_out=Fake((2, 2, value, D), F16), v_out=Fake((2, 2, value, D), F16))
    with pytest.raises(ValueError):
        call(api, **kw)
    assert not api.log
