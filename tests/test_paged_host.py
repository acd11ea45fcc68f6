"""Refusals of the paged-cache operators (host arithmetic, no GPU: fake
addresses that never reach a device) and the plain reference's own checks."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_ref as ref  # noqa: E402

A = 1 << 40
M = 1 << 30
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def api():
    from kv_cache_quantization_turboquantrvq_gb300 import api as a, build
    build.build()
    a.lib()
    return a


def _append(api, k=A, kst=256, ksh=128, v=A + M, vst=256, vsh=128, it=0, T=8, slots=A + 2 * M, kp=A + 3 * M, vp=A + 4 * M,
            ke=0, ve=0, ct=0, NP=4, H=2, PS=16, D=128):
    return api.lib().vq_paged_append(P(k), kst, ksh, P(v), vst, vsh, it, T, P(slots), P(kp), P(vp), P(ke), P(ve), ct, NP,
                                     H, PS, D, None)


def test_append_refusals(api):
    e = dict(ct=2, ke=A + 5 * M, ve=A + 6 * M)
    assert _append(api, D=64) == api.VQ_ERR_UNSUPPORTED
    assert _append(api, PS=24) == api.VQ_ERR_UNSUPPORTED
    assert _append(api, PS=8) == api.VQ_ERR_UNSUPPORTED
    assert _append(api, NP=1 << 28) == api.VQ_ERR_UNSUPPORTED        # 2^31 rows and more
    assert _append(api, PS=0) == api.VQ_ERR_INVALID_ARG
    assert _append(api, H=0) == api.VQ_ERR_INVALID_ARG
    assert _append(api, T=-1) == api.VQ_ERR_INVALID_ARG
    assert _append(api, it=2) == api.VQ_ERR_INVALID_ARG              # input in 8 bits
    assert _append(api, it=0, ct=1) == api.VQ_ERR_INVALID_ARG        # fp16 into a bf16 cache
    assert _append(api, ct=3) == api.VQ_ERR_INVALID_ARG
    assert _append(api, k=0) == api.VQ_ERR_INVALID_ARG
    assert _append(api, slots=0) == api.VQ_ERR_INVALID_ARG
    assert _append(api, vp=0) == api.VQ_ERR_INVALID_ARG
    assert _append(api, ct=2) == api.VQ_ERR_INVALID_ARG              # codes without exponents
    assert _append(api, kst=64) == api.VQ_ERR_INVALID_ARG            # tokens overlap
    assert _append(api, vsh=-128) == api.VQ_ERR_INVALID_ARG
    assert _append(api, kst=260) == api.VQ_ERR_MISALIGNED
    assert _append(api, k=A + 8) == api.VQ_ERR_MISALIGNED
    assert _append(api, kp=A + 3 * M + 8) == api.VQ_ERR_MISALIGNED
    assert _append(api, slots=A + 2 * M + 4) == api.VQ_ERR_MISALIGNED
    assert _append(api, kp=A + 64) == api.VQ_ERR_ALIASING            # pages over the keys
    assert _append(api, vp=A + 3 * M + 16) == api.VQ_ERR_ALIASING    # the pools overlap
    assert _append(api, **dict(e, ve=A + 5 * M)) == api.VQ_ERR_ALIASING
    assert _append(api, T=0, k=0, v=0, slots=0, kp=0, vp=0) == api.VQ_OK


def _gather(api, kp=A, vp=A + M, ke=0, ve=0, ct=0, NP=4, H=2, PS=16, D=128, table=A + 2 * M, mp=3, lens=A + 3 * M, first=0,
            B=2, S=8, ot=0, ko=A + 4 * M, vo=A + 5 * M):
    return api.lib().vq_paged_gather(P(kp), P(vp), P(ke), P(ve), ct, NP, H, PS, D, P(table), mp, P(lens), P(first), B, S,
                                     ot, P(ko), P(vo), None)


def test_gather_refusals(api):
    assert _gather(api, D=256) == api.VQ_ERR_UNSUPPORTED
    assert _gather(api, PS=512) == api.VQ_ERR_UNSUPPORTED
    assert _gather(api, S=1 << 30) == api.VQ_ERR_UNSUPPORTED
    assert _gather(api, B=-1) == api.VQ_ERR_INVALID_ARG
    assert _gather(api, ot=1) == api.VQ_ERR_INVALID_ARG              # bf16 out of an fp16 cache
    assert _gather(api, ot=2) == api.VQ_ERR_INVALID_ARG
    assert _gather(api, ko=0, vo=0) == api.VQ_ERR_INVALID_ARG
    assert _gather(api, kp=0) == api.VQ_ERR_INVALID_ARG
    assert _gather(api, lens=0) == api.VQ_ERR_INVALID_ARG
    assert _gather(api, table=0) == api.VQ_ERR_INVALID_ARG
    assert _gather(api, ct=2) == api.VQ_ERR_INVALID_ARG
    assert _gather(api, ko=A + 4 * M + 2) == api.VQ_ERR_MISALIGNED
    assert _gather(api, lens=A + 3 * M + 2) == api.VQ_ERR_MISALIGNED
    assert _gather(api, ko=A + 256) == api.VQ_ERR_ALIASING
    assert _gather(api, vo=A + 4 * M + 256) == api.VQ_ERR_ALIASING
    assert _gather(api, ko=A + 3 * M) == api.VQ_ERR_ALIASING         # over the lengths
    assert _gather(api, S=0, ko=A, vo=A) == api.VQ_OK


def _attend(api, q=A, qst=1024, qsh=128, qt=0, kp=A + M, vp=A + 2 * M, ke=0, ve=0, ct=0, NP=4, H=2, PS=16, D=128,
            table=A + 3 * M, mp=3, cu=A + 4 * M, lens=A + 5 * M, T=8, B=2, Hq=8, max_q=4, window=0, sinks=0, scale=0.1,
            out=A + 6 * M, ws=A + 7 * M, wb=None):
    if wb is None:
        n = ctypes.c_size_t(0)
        st = api.lib().vq_paged_attend_workspace(T, B, Hq, H, max_q, ctypes.byref(n))
        wb = n.value if st == 0 else 1 << 30
    return api.lib().vq_paged_attend(P(q), qst, qsh, qt, P(kp), P(vp), P(ke), P(ve), ct, NP, H, PS, D, P(table), mp, P(cu),
                                     P(lens), T, B, Hq, max_q, window, sinks, ctypes.c_float(scale), P(out), P(ws), wb,
                                     None)


def test_attend_refusals(api):
    assert _attend(api, D=64) == api.VQ_ERR_UNSUPPORTED
    assert _attend(api, Hq=34) == api.VQ_ERR_UNSUPPORTED             # 17 query heads to a kv head
    assert _attend(api, mp=(1 << 26) + 1) == api.VQ_ERR_UNSUPPORTED  # positions past 2^30
    assert _attend(api, Hq=7) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, max_q=0) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, window=-1) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, sinks=-1) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, scale=float("nan")) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, qt=2) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, qt=1) == api.VQ_ERR_INVALID_ARG              # bf16 queries over an fp16 cache
    assert _attend(api, ct=2) == api.VQ_ERR_INVALID_ARG              # codes without exponents
    assert _attend(api, NP=0) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, q=0) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, table=0) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, cu=0) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, out=0) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, ws=0) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, wb=100) == api.VQ_ERR_INVALID_ARG            # workspace too small
    assert _attend(api, qst=100) == api.VQ_ERR_INVALID_ARG
    assert _attend(api, qst=1028) == api.VQ_ERR_MISALIGNED
    assert _attend(api, q=A + 4) == api.VQ_ERR_MISALIGNED
    assert _attend(api, ws=A + 7 * M + 16) == api.VQ_ERR_MISALIGNED
    assert _attend(api, vp=A + 2 * M + 8) == api.VQ_ERR_MISALIGNED
    assert _attend(api, out=A + 512) == api.VQ_ERR_ALIASING          # over the queries
    assert _attend(api, ws=A + 6 * M + 256) == api.VQ_ERR_ALIASING   # workspace over the output
    assert _attend(api, ws=A + M) == api.VQ_ERR_ALIASING             # workspace over the cache
    assert _attend(api, T=0, q=0, out=0, ws=0) == api.VQ_OK
    assert _attend(api, B=0) == api.VQ_OK
    n = ctypes.c_size_t(0)
    f = api.lib().vq_paged_attend_workspace
    assert f(8, 2, 8, 2, 4, None) == api.VQ_ERR_INVALID_ARG
    assert f(-1, 2, 8, 2, 4, ctypes.byref(n)) == api.VQ_ERR_INVALID_ARG
    assert f(8, 2, 8, 2, 4, ctypes.byref(n)) == api.VQ_OK and n.value > 0


def test_binding_refuses_what_it_would_have_to_copy(api):
    c = api.paged_cache(4, 2, 16, torch.float16, device="cpu")
    with pytest.raises(ValueError):  # not a CUDA tensor
        api.vq_paged_append(torch.zeros(3, 2, 128).half(), torch.zeros(3, 2, 128).half(), c, torch.zeros(3).long())
    with pytest.raises(ValueError):
        api.paged_cache(4, 2, 16, torch.float32, device="cpu")
    with pytest.raises(ValueError):
        api._typed(torch.zeros(3), torch.float32, (3,), "x")


def test_reference_quantiser():
    """The reference's codes by hand: exponents at the borders, ties to even, saturation."""
    x = torch.zeros(6, 128)
    x[0, 0] = 448.0          # e = 0, the largest code
    x[1, 0] = 449.0          # one more needs e = 1
    x[2, 0], x[2, 1], x[2, 2], x[2, 3] = 256.0, 17.0, 19.0, 2.0 ** -10  # ties: 16 and 20; half of the least code: 0
    x[3, 0] = 2.0 ** 100     # saturates at 448 * 2^64
    x[4, 0] = 2.0 ** -45     # below the least exponent: 2^-13 of a code's unit
    code, e = ref.quantise(x)
    assert (e.int() - 127).tolist() == [0, 1, 0, 64, -32, 0]
    v = ref.E4M3[code.numpy()]
    assert v[0, 0] == 448 and v[1, 0] == 224 and v[2, 1] == 16 and v[2, 2] == 20 and v[2, 3] == 0
    assert v[3, 0] == 448 and v[4, 0] == 0 and np.all(v[5] == 0)
    t = torch.tensor(ref.E4M3).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    ok = ~np.isnan(ref.E4M3)
    assert np.array_equal(t[ok], np.arange(256)[ok])
