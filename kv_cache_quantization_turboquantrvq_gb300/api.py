"""Python binding of the C ABI in include/vq.h (ctypes; argument marshalling only).

Every function here has the name of the C entry point it calls.  Tensors are
torch CUDA tensors (torch supplies device memory and the current stream);
codebooks are small host float32 arrays.  All arithmetic runs in the CUDA
library ``libvqflush.so``; if it is missing this module raises on first use,
there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvqflush.so")
_lib = None

VQ_OK = 0
VQ_ERR_INVALID_ARG = 1
VQ_ERR_UNSUPPORTED = 2
VQ_ERR_MISALIGNED = 3
VQ_ERR_ALIASING = 4
VQ_ERR_CUDA = 5
VQ_ERR_DEVICE = 6
VQ_DEVERR_WAIT_TIMEOUT = 0x1
VQ_DEVERR_BAD_OFFSET = 0x2

EXPORTED = ("vq_status_str", "vq_version", "vq_rvq_codebook", "vq_rvq_encode_pack",
            "vq_rvq_unpack_dequant", "vq_kivi_quant_pack", "vq_kivi_unpack_dequant",
            "vq_device_error", "vq_rvq_attend_workspace", "vq_rvq_attend", "vq_rvq_attend_noalloc",
            "vq_rvq_encode_pack_rs", "vq_rvq_unpack_dequant_rs", "vq_rvq_attend_rs",
            "vq_kivi_attend_workspace", "vq_kivi_attend", "vq_qjl_encode", "vq_flush_decode",
            "vq_paged_append", "vq_paged_gather", "vq_paged_attend_workspace", "vq_paged_attend",
            "vq_paged_attend_tree_workspace", "vq_paged_attend_tree",
            "vq_paged_attend_weigh_workspace", "vq_paged_attend_weigh", "vq_paged_select", "vq_paged_compact")
VQ_F16, VQ_BF16, VQ_E4M3 = 0, 1, 2
VQ_ATTEND_SCRATCH_BYTES = 16 * 1024 * 1024


class VQError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s" % (what, lib().vq_status_str(status).decode()))
        self.status = status


def lib():
    """Load libvqflush.so (raises OSError when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise OSError("libvqflush.so is not built (run __graft_entry__.build()): %s" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    P, I = ctypes.c_void_p, ctypes.c_int
    L.vq_status_str.argtypes = [I]
    L.vq_status_str.restype = ctypes.c_char_p
    L.vq_version.argtypes = []
    L.vq_version.restype = ctypes.c_char_p
    L.vq_rvq_codebook.argtypes = [I, I, P, P, P, P]
    L.vq_rvq_encode_pack.argtypes = [P, I, I, I, I, I, P, P, P, P, P, P, P, P, I, P]
    L.vq_rvq_unpack_dequant.argtypes = [P, P, P, I, I, I, I, I, P, P, P, P]
    L.vq_kivi_quant_pack.argtypes = [P, P, I, I, I, I, I, I, I, P, P, P, P, P, P, P, I, P]
    L.vq_kivi_unpack_dequant.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, P]
    L.vq_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
    L.vq_rvq_attend_workspace.argtypes = [I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
    L.vq_rvq_attend.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, ctypes.c_float, P, P,
                                ctypes.c_size_t, P]
    L.vq_rvq_attend_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, ctypes.c_float, P, P]
    L.vq_rvq_encode_pack_rs.argtypes = [P, I, I, I, I, I, P, P, P, P, P, P, P, P, I, P, P]
    L.vq_rvq_unpack_dequant_rs.argtypes = [P, P, P, I, I, I, I, I, P, P, P, P, P]
    L.vq_rvq_attend_rs.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, ctypes.c_float, P, P,
                                   ctypes.c_size_t, P]
    L.vq_kivi_attend_workspace.argtypes = [I, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
    L.vq_kivi_attend.argtypes = [P] * 11 + [I] * 8 + [ctypes.c_float, P, P, ctypes.c_size_t, P]
    L.vq_qjl_encode.argtypes = [P, I, I, P, I, P, P, P]
    L.vq_flush_decode.argtypes = [P, P, I, I, I, I, I, P, I, I, P, P, P, P, P, P, P, I, I,
                                  P, P, P, P, P, P, P, P, P, I, P]
    Q = ctypes.c_longlong
    L.vq_paged_append.argtypes = [P, Q, Q, P, Q, Q, I, I, P, P, P, P, P, I, I, I, I, I, P]
    L.vq_paged_gather.argtypes = [P, P, P, P, I, I, I, I, I, P, I, P, P, I, I, I, P, P, P]
    L.vq_paged_attend_workspace.argtypes = [I, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
    L.vq_paged_attend.argtypes = [P, Q, Q, I, P, P, P, P, I, I, I, I, I, P, I, P, P, I, I, I, I, I, I,
                                  ctypes.c_float, P, P, ctypes.c_size_t, P]
    L.vq_paged_attend_tree_workspace.argtypes = L.vq_paged_attend_workspace.argtypes
    L.vq_paged_attend_tree.argtypes = [P, Q, Q, I, P, P, P, P, I, I, I, I, I, P, I, P, P, P, I, I, I, I, I, I,
                                       ctypes.c_float, P, P, ctypes.c_size_t, P]
    L.vq_paged_attend_weigh_workspace.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
    L.vq_paged_attend_weigh.argtypes = [P, Q, Q, I, P, P, P, P, I, I, I, I, I, P, I, P, P, I, I, I, I, I, I, ctypes.c_float,
                                        P, I, ctypes.c_float, P, P, ctypes.c_size_t, P]
    L.vq_paged_select.argtypes = [P, I, I, I, P, I, P, I, I, I, I, P, P, P]
    L.vq_paged_compact.argtypes = [P, P, P, P, I, I, I, I, I, P, I, P, Q, Q, I, P, P, I, P, P]
    for name in EXPORTED[2:]:
        getattr(L, name).restype = I
    _lib = L
    return L


def _check(status: int, what: str):
    if status != VQ_OK:
        raise VQError(status, what)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _host(a):
    a = np.ascontiguousarray(a, dtype=np.float32)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _fp16(*tensors):
    """ValueError for keys or values of another floating type than the codecs read
    (a bf16 cache's blocks are read back as fp16 by vq_paged_gather)."""
    import torch
    for t in tensors:
        if t is not None and t.is_floating_point() and t.dtype != torch.float16:
            raise ValueError("keys and values of dtype %s: float16" % t.dtype)


def vq_status_str(status: int) -> str:
    return lib().vq_status_str(status).decode()


def vq_version() -> str:
    return lib().vq_version().decode()


def rvq_words(D: int, bits: int) -> int:
    """Packed words per row and stream: floor(32/b) codes per word."""
    return -(-D // (32 // bits))


def vq_rvq_codebook(D: int, bits: int):
    """(c1, b1, c2, b2) float32 host arrays: Gaussian stage-1 and Laplace-fit stage-2."""
    L = 1 << bits
    c1 = np.empty(L, np.float32)
    b1 = np.empty(L - 1, np.float32)
    c2 = np.empty(L, np.float32)
    b2 = np.empty(L - 1, np.float32)
    _check(lib().vq_rvq_codebook(D, bits, *[a.ctypes.data_as(ctypes.c_void_p) for a in (c1, b1, c2, b2)]),
           "vq_rvq_codebook")
    return c1, b1, c2, b2


def _sign_words(signs):
    s = np.ascontiguousarray(np.asarray(signs, dtype=np.uint32).ravel())
    if s.size != 4:
        raise ValueError("signs: 4 uint32 words (one bit per coordinate of D = 128)")
    return s


def vq_rvq_encode_pack(k, bits: int, c1, b1, c2, b2, packed1=None, packed2=None, norms=None,
                       dst_off=None, S_dst=None, stream=None, signs=None):
    """Encode fp16 keys k [B, H, S, D] into (packed1, packed2, norms); with
    `signs` (4 uint32 words) the randomised-sign rotation H diag(s)."""
    import torch
    _fp16(k)
    B, H, S, D = k.shape
    S_dst = S if S_dst is None else S_dst
    W = rvq_words(D, bits)
    if packed1 is None:
        packed1 = torch.empty((B, H, S_dst, W), dtype=torch.int32, device=k.device)
    if packed2 is None:
        packed2 = torch.empty((B, H, S_dst, W), dtype=torch.int32, device=k.device)
    if norms is None:
        norms = torch.empty((B, H, S_dst), dtype=torch.float32, device=k.device)
    keep = [_host(v) for v in (c1, b1, c2, b2)]
    if signs is None:
        _check(lib().vq_rvq_encode_pack(_ptr(k), B, H, S, D, bits, *[p for _, p in keep],
                                        _ptr(packed1), _ptr(packed2), _ptr(norms), _ptr(dst_off),
                                        S_dst, _stream(stream)), "vq_rvq_encode_pack")
    else:
        sw = _sign_words(signs)
        _check(lib().vq_rvq_encode_pack_rs(_ptr(k), B, H, S, D, bits, *[p for _, p in keep],
                                           _ptr(packed1), _ptr(packed2), _ptr(norms), _ptr(dst_off),
                                           S_dst, sw.ctypes.data_as(ctypes.c_void_p), _stream(stream)),
               "vq_rvq_encode_pack_rs")
    return packed1, packed2, norms


def vq_rvq_unpack_dequant(packed1, packed2, norms, bits: int, c1, c2, out=None, stream=None, signs=None,
                          D: int = 128):
    """Decode (packed1, packed2, norms) [B, H, S, W] back to fp16 keys [B, H, S, D]."""
    import torch
    B, H, S, _ = packed1.shape
    if out is None:
        out = torch.empty((B, H, S, D), dtype=torch.float16, device=packed1.device)
    keep = [_host(v) for v in (c1, c2)]
    if signs is None:
        _check(lib().vq_rvq_unpack_dequant(_ptr(packed1), _ptr(packed2), _ptr(norms), B, H, S, D, bits,
                                           keep[0][1], keep[1][1], _ptr(out), _stream(stream)),
               "vq_rvq_unpack_dequant")
    else:
        sw = _sign_words(signs)
        _check(lib().vq_rvq_unpack_dequant_rs(_ptr(packed1), _ptr(packed2), _ptr(norms), B, H, S, D, bits,
                                              keep[0][1], keep[1][1], sw.ctypes.data_as(ctypes.c_void_p),
                                              _ptr(out), _stream(stream)), "vq_rvq_unpack_dequant_rs")
    return out


def kivi_shapes(B, H, S_dst, D, bits, group):
    """Output shapes of vq_kivi_quant_pack for a destination of S_dst tokens."""
    NG = (S_dst + group - 1) // group
    return {
        "k_packed": (B, H, NG, group * bits // 32, D), "k_scale": (B, H, NG, D),
        "v_packed": (B, H, S_dst, D * bits // 32), "v_scale": (B, H, S_dst, D // group),
    }


def vq_rvq_attend_workspace(B: int, Hq: int, Hkv: int, S_cap: int) -> int:
    """Workspace bytes vq_rvq_attend wants for these shapes on the current device."""
    n = ctypes.c_size_t(0)
    _check(lib().vq_rvq_attend_workspace(B, Hq, Hkv, S_cap, ctypes.byref(n)), "vq_rvq_attend_workspace")
    return int(n.value)


def vq_rvq_attend(q, packed1, packed2, norms, v, bits: int, c1, c2, scale: float, lens=None, out=None,
                  workspace=None, stream=None, signs=None):
    """Decode-time attention of q [B, Hq, 128] over an RVQ key cache
    (packed1, packed2, norms [B, Hkv, S_cap, ...]) and fp16 values v
    [B, Hkv, S_cap, 128]; lens [B] int32 (device) or None.  Returns fp16
    [B, Hq, 128].  The workspace is allocated when not given."""
    import torch
    B, Hq, D = q.shape
    _, Hkv, S_cap, _ = packed1.shape
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float16, device=q.device)
    if workspace is None:
        nbytes = vq_rvq_attend_workspace(B, Hq, Hkv, S_cap)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=q.device)
    wbytes = workspace.numel() * workspace.element_size()
    keep = [_host(t) for t in (c1, c2)]
    if signs is None:
        _check(lib().vq_rvq_attend(_ptr(q), _ptr(packed1), _ptr(packed2), _ptr(norms), _ptr(v), _ptr(lens),
                                   B, Hq, Hkv, S_cap, D, bits, keep[0][1], keep[1][1], float(scale),
                                   _ptr(out), _ptr(workspace), wbytes, _stream(stream)), "vq_rvq_attend")
    else:
        sw = _sign_words(signs)
        _check(lib().vq_rvq_attend_rs(_ptr(q), _ptr(packed1), _ptr(packed2), _ptr(norms), _ptr(v), _ptr(lens),
                                      B, Hq, Hkv, S_cap, D, bits, keep[0][1], keep[1][1],
                                      sw.ctypes.data_as(ctypes.c_void_p), float(scale), _ptr(out),
                                      _ptr(workspace), wbytes, _stream(stream)), "vq_rvq_attend_rs")
    return out


def vq_rvq_attend_noalloc(q, packed1, packed2, norms, v, bits: int, c1, c2, scale: float, lens=None,
                          out=None, stream=None):
    """vq_rvq_attend with the library's static device scratch instead of a
    workspace (calls must not overlap in time on one device)."""
    import torch
    B, Hq, D = q.shape
    _, Hkv, S_cap, _ = packed1.shape
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float16, device=q.device)
    keep = [_host(t) for t in (c1, c2)]
    _check(lib().vq_rvq_attend_noalloc(_ptr(q), _ptr(packed1), _ptr(packed2), _ptr(norms), _ptr(v), _ptr(lens),
                                       B, Hq, Hkv, S_cap, D, bits, keep[0][1], keep[1][1], float(scale),
                                       _ptr(out), _stream(stream)), "vq_rvq_attend_noalloc")
    return out


def vq_kivi_attend_workspace(B: int, Hq: int, Hkv: int, S_cap: int, R: int) -> int:
    """Workspace bytes vq_kivi_attend wants for these shapes on the current device."""
    n = ctypes.c_size_t(0)
    _check(lib().vq_kivi_attend_workspace(B, Hq, Hkv, S_cap, R, ctypes.byref(n)), "vq_kivi_attend_workspace")
    return int(n.value)


def vq_kivi_attend(q, cache: dict, bits: int, group: int, scale: float, k_res=None, v_res=None, lens=None,
                   res_lens=None, out=None, workspace=None, stream=None):
    """Decode-time attention of q [B, Hq, 128] over a KIVI cache (`cache`: the
    dict vq_kivi_quant_pack returns, written with S_dst = S_cap) plus the fp16
    residual window k_res, v_res [B, Hkv, R, 128].  Returns fp16 [B, Hq, 128]."""
    import torch
    B, Hq, D = q.shape
    vp = cache["v_packed"]
    Hkv, S_cap = vp.shape[1], vp.shape[2]
    R = 0 if k_res is None else k_res.shape[2]
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float16, device=q.device)
    if workspace is None:
        nbytes = vq_kivi_attend_workspace(B, Hq, Hkv, S_cap, R)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=q.device)
    wbytes = workspace.numel() * workspace.element_size()
    c = cache
    _check(lib().vq_kivi_attend(_ptr(q), _ptr(c["k_packed"]), _ptr(c["k_scale"]), _ptr(c["k_zero"]),
                                _ptr(c["v_packed"]), _ptr(c["v_scale"]), _ptr(c["v_zero"]), _ptr(k_res),
                                _ptr(v_res), _ptr(lens), _ptr(res_lens), B, Hq, Hkv, S_cap, R, D, bits, group,
                                float(scale), _ptr(out), _ptr(workspace), wbytes, _stream(stream)),
           "vq_kivi_attend")
    return out


def vq_kivi_quant_pack(k, v, bits: int, group: int, residual_length: int, outs=None,
                       dst_off=None, S_dst=None, stream=None):
    """KIVI flush of k and/or v ([B, H, S, D] fp16; either may be None).

    Returns a dict with k_packed, k_scale, k_zero, v_packed, v_scale, v_zero
    (allocated when `outs` does not provide them)."""
    import torch
    _fp16(k, v)
    ref = k if k is not None else v
    B, H, S, D = ref.shape
    S_q = max(S - residual_length, 0)
    S_dst = S_q if S_dst is None else S_dst
    shp = kivi_shapes(B, H, S_dst, D, bits, group)
    outs = dict(outs or {})
    dev = ref.device
    if k is not None:
        outs.setdefault("k_packed", torch.empty(shp["k_packed"], dtype=torch.int32, device=dev))
        outs.setdefault("k_scale", torch.empty(shp["k_scale"], dtype=torch.float16, device=dev))
        outs.setdefault("k_zero", torch.empty(shp["k_scale"], dtype=torch.float16, device=dev))
    if v is not None:
        outs.setdefault("v_packed", torch.empty(shp["v_packed"], dtype=torch.int32, device=dev))
        outs.setdefault("v_scale", torch.empty(shp["v_scale"], dtype=torch.float16, device=dev))
        outs.setdefault("v_zero", torch.empty(shp["v_scale"], dtype=torch.float16, device=dev))
    g = outs.get
    _check(lib().vq_kivi_quant_pack(_ptr(k), _ptr(v), B, H, S, D, bits, group, residual_length,
                                    _ptr(g("k_packed") if k is not None else None),
                                    _ptr(g("k_scale") if k is not None else None),
                                    _ptr(g("k_zero") if k is not None else None),
                                    _ptr(g("v_packed") if v is not None else None),
                                    _ptr(g("v_scale") if v is not None else None),
                                    _ptr(g("v_zero") if v is not None else None),
                                    _ptr(dst_off), S_dst, _stream(stream)), "vq_kivi_quant_pack")
    return outs


def vq_kivi_unpack_dequant(packs: dict, B: int, H: int, S_q: int, bits: int, group: int,
                           k_out=None, v_out=None, want_k=True, want_v=True, stream=None):
    """Dequantize the KIVI storage in `packs` (keys and/or values) to fp16 [B, H, S_q, 128]."""
    import torch
    D = 128
    dk = want_k and "k_packed" in packs
    dv = want_v and "v_packed" in packs
    ref = packs["k_packed"] if dk else packs["v_packed"]
    if dk and k_out is None:
        k_out = torch.empty((B, H, S_q, D), dtype=torch.float16, device=ref.device)
    if dv and v_out is None:
        v_out = torch.empty((B, H, S_q, D), dtype=torch.float16, device=ref.device)
    _check(lib().vq_kivi_unpack_dequant(
        _ptr(packs["k_packed"]) if dk else None, _ptr(packs["k_scale"]) if dk else None,
        _ptr(packs["k_zero"]) if dk else None, _ptr(packs["v_packed"]) if dv else None,
        _ptr(packs["v_scale"]) if dv else None, _ptr(packs["v_zero"]) if dv else None,
        B, H, S_q, D, bits, group, _ptr(k_out) if dk else None, _ptr(v_out) if dv else None,
        _stream(stream)), "vq_kivi_unpack_dequant")
    return k_out, v_out


def vq_device_error(stream=None) -> int:
    """Wait for the stream; read and clear the library's device error bits."""
    code = ctypes.c_int(0)
    st = lib().vq_device_error(_stream(stream), ctypes.byref(code))
    if st not in (VQ_OK, VQ_ERR_DEVICE):
        raise VQError(st, "vq_device_error")
    return code.value


def vq_qjl_encode(x, s, packed=None, norms=None, stream=None):
    """QJL encode of the key rows x [..., 128] fp16 with the sketch s [m, 128]
    fp16: returns (packed [..., m/32] int32 sign words, norms [...] fp16)."""
    import torch
    D = x.shape[-1]
    lead = tuple(x.shape[:-1])
    N = 1
    for v in lead:
        N *= v
    m = s.shape[0]
    if packed is None:
        packed = torch.empty(lead + (m // 32,), dtype=torch.int32, device=x.device)
    if norms is None:
        norms = torch.empty(lead, dtype=torch.float16, device=x.device)
    _check(lib().vq_qjl_encode(_ptr(x), N, D, _ptr(s), m, _ptr(packed), _ptr(norms), _stream(stream)),
           "vq_qjl_encode")
    return packed, norms


def vq_flush_decode(k, v, residual_length: int, dst_off=None, S_dst=None, rvq=None, kivi=None,
                    window=None, stream=None):
    """The decode-time flush of one layer in one launch: k, v [B, H, T, 128]
    fp16 (either may be None when no part needs it); tokens [0, T - R) are
    quantized at the sequences' offsets, tokens [T - R, T) copied to the fp16
    window.  Parts (each optional, outputs allocated when absent):
      rvq = dict(bits, books=(c1, b1, c2, b2)[, packed1, packed2, norms])
      kivi = dict(bits, group[, keys=True, values=True, k_packed, ..., v_zero])
      window = dict([k_win, v_win, win_off, R_cap])
    Returns a dict with every output tensor."""
    import torch
    _fp16(k, v)
    ref = k if k is not None else v
    B, H, T, D = ref.shape
    R = int(residual_length)
    S_q = T - R
    S_dst = S_q if S_dst is None else S_dst
    dev = ref.device
    out = {}
    keep = []
    rb, rp = 0, [None] * 4
    if rvq is not None:
        rb = int(rvq["bits"])
        keep = [_host(a) for a in rvq["books"]]
        rp = [p_ for _, p_ in keep]
        W = rvq_words(D, rb)
        out["packed1"] = rvq.get("packed1", torch.empty((B, H, S_dst, W), dtype=torch.int32, device=dev))
        out["packed2"] = rvq.get("packed2", torch.empty((B, H, S_dst, W), dtype=torch.int32, device=dev))
        out["norms"] = rvq.get("norms", torch.empty((B, H, S_dst), dtype=torch.float32, device=dev))
    kb, G = 0, 0
    if kivi is not None:
        kb, G = int(kivi["bits"]), int(kivi["group"])
        shp = kivi_shapes(B, H, S_dst, D, kb, G)
        if kivi.get("keys", True):
            out["k_packed"] = kivi.get("k_packed", torch.empty(shp["k_packed"], dtype=torch.int32, device=dev))
            out["k_scale"] = kivi.get("k_scale", torch.empty(shp["k_scale"], dtype=torch.float16, device=dev))
            out["k_zero"] = kivi.get("k_zero", torch.empty(shp["k_scale"], dtype=torch.float16, device=dev))
        if kivi.get("values", True):
            out["v_packed"] = kivi.get("v_packed", torch.empty(shp["v_packed"], dtype=torch.int32, device=dev))
            out["v_scale"] = kivi.get("v_scale", torch.empty(shp["v_scale"], dtype=torch.float16, device=dev))
            out["v_zero"] = kivi.get("v_zero", torch.empty(shp["v_scale"], dtype=torch.float16, device=dev))
    win_off, R_cap = None, 0
    if window is not None and R > 0:
        R_cap = int(window.get("R_cap", R))
        win_off = window.get("win_off")
        if k is not None:
            out["k_win"] = window.get("k_win", torch.empty((B, H, R_cap, D), dtype=torch.float16, device=dev))
        if v is not None:
            out["v_win"] = window.get("v_win", torch.empty((B, H, R_cap, D), dtype=torch.float16, device=dev))
    g = out.get
    _check(lib().vq_flush_decode(_ptr(k), _ptr(v), B, H, T, D, R, _ptr(dst_off), S_dst, rb, *rp,
                                 _ptr(g("packed1")), _ptr(g("packed2")), _ptr(g("norms")), kb, G,
                                 _ptr(g("k_packed")), _ptr(g("k_scale")), _ptr(g("k_zero")),
                                 _ptr(g("v_packed")), _ptr(g("v_scale")), _ptr(g("v_zero")),
                                 _ptr(g("k_win")), _ptr(g("v_win")), _ptr(win_off), R_cap, _stream(stream)),
           "vq_flush_decode")
    return out


# The paged calls run once per layer and step, so the checks below are written to
# cost little: plain comparisons, no copies, the stream's handle without an object.
_DTYPE_CODES: dict = {}


def _dtype_code(dtype) -> int:
    """VQ_F16, VQ_BF16 or VQ_E4M3 of a torch dtype (ValueError for others)."""
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.float16: VQ_F16, torch.bfloat16: VQ_BF16, torch.float8_e4m3fn: VQ_E4M3})
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise ValueError("dtype %s: float16, bfloat16 or float8_e4m3fn" % dtype)
    return code


def _gpu(t, what) -> int:
    """The index of the GPU that t lies on (ValueError: on none)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s: a CUDA tensor" % what)
    return dev


def _typed(t, dtype, shape, what, dev=None):
    """The address of t; ValueError unless it is a contiguous CUDA tensor of this dtype
    and shape (on GPU dev)."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: a contiguous CUDA tensor %s of %s" % (what, tuple(shape), dtype))
    if (t.get_device() != dev) if dev is not None else not t.is_cuda:
        raise ValueError("%s: on the GPU of the other tensors" % what)
    return t.data_ptr()


def _rows_view(t, heads, D, what, dev):
    """(address, token stride, head stride) of a [T, heads, D] view on GPU dev whose rows are contiguous."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != D or t.get_device() != dev:
        raise ValueError("%s: a CUDA tensor [tokens, %d, %d] on the GPU of the other tensors" % (what, heads, D))
    st = t.stride()
    if st[2] != 1:
        raise ValueError("%s: the entries of a head have to be contiguous" % what)
    return t.data_ptr(), st[0], st[1]


def _raw_stream(stream, t):
    """The handle of `stream`, or of the current stream of t's device."""
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(t.device.index) if raw is not None else torch.cuda.current_stream().cuda_stream


def _empty(shape, dtype, device, stream, returned=True):
    """An empty tensor that a call on `stream`, not None, writes.  It is made on that
    stream: a block of the current stream's could still be in use by kernels queued
    there, and would go back to it while the call still runs.  What is returned is
    reserved for the current stream's use too."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned and current.cuda_stream != stream.cuda_stream:
        t.record_stream(current)
    return t


def paged_cache(num_pages: int, Hkv: int, page_size: int, dtype, device="cuda", D: int = 128) -> dict:
    """An empty paged cache: k_pages, v_pages [num_pages, Hkv, page_size, D] of
    dtype (float16, bfloat16 or float8_e4m3fn) and, for float8_e4m3fn, k_exp, v_exp
    [num_pages, Hkv, page_size] uint8 (None otherwise)."""
    import torch
    shape = (num_pages, Hkv, page_size, D)
    c = {x + "_pages": torch.zeros(shape, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype,
                                   device=device).view(dtype) for x in "kv"}
    q = _dtype_code(dtype) == VQ_E4M3
    for x in "kv":
        c[x + "_exp"] = torch.full(shape[:3], 127, dtype=torch.uint8, device=device) if q else None
    return c


_INT_MAX = (1 << 31) - 1  # (ctypes cuts larger numbers to other ones)
_gpus = 0  # how many this process sees; 0: not asked yet


def _on_gpu(dev, function):
    """`function` as it is called with GPU dev current, which a call's sizes and launches are for."""
    import torch
    global _gpus
    if _gpus == 0:
        _gpus = torch.cuda.device_count()
    if _gpus == 1 or torch.cuda.current_device() == dev:
        return function

    def there(*args):
        with torch.cuda.device(dev):
            return function(*args)
    return there


def _cache_args(cache, dev):
    """(k, v, k_exp, v_exp, dtype, num_pages, Hkv, page_size, D) of a cache dict on GPU dev."""
    k, v = cache["k_pages"], cache["v_pages"]
    dtype, shape = k.dtype, k.shape
    code = _dtype_code(dtype)
    if len(shape) != 4:
        raise ValueError("k_pages: [num_pages, Hkv, page_size, D]")
    kp, vp = _typed(k, dtype, shape, "k_pages", dev), _typed(v, dtype, shape, "v_pages", dev)
    ke = ve = None
    if code == VQ_E4M3:
        import torch
        ke, ve = cache.get("k_exp"), cache.get("v_exp")
        if ke is None or ve is None:
            raise ValueError("a float8_e4m3fn cache has k_exp and v_exp")
        ke, ve = _typed(ke, torch.uint8, shape[:3], "k_exp", dev), _typed(ve, torch.uint8, shape[:3], "v_exp", dev)
    return (kp, vp, ke, ve, code, *shape)


def vq_paged_append(k, v, cache: dict, slots, stream=None) -> dict:
    """Write the keys and values k, v [T, Hkv, 128] (fp16 or bf16, rows may be
    strided) of new tokens into the paged cache at slots [T] int64 (page *
    page_size + place; negative: not written).  Returns the cache."""
    import torch
    dev = _gpu(k, "k")
    args = _cache_args(cache, dev)
    T = k.shape[0]
    if k.dtype != v.dtype or v.shape[0] != T:
        raise ValueError("k and v: the same tokens and dtype")
    views = _rows_view(k, args[6], args[8], "k", dev) + _rows_view(v, args[6], args[8], "v", dev)
    _check(_on_gpu(dev, lib().vq_paged_append)(*views, _dtype_code(k.dtype), T,
                                               _typed(slots, torch.int64, (T,), "slots", dev), *args,
                                               _raw_stream(stream, k)), "vq_paged_append")
    return cache


def vq_paged_gather(cache: dict, block_table, lens, S_out: int, first=None, dtype=None, k_out=None, v_out=None,
                    want_k=True, want_v=True, stream=None):
    """Read tokens first[b] + [0, S_out) of every sequence back: (k, v)
    [B, Hkv, S_out, 128] of dtype (the cache's, float16 from an 8-bit one; float16,
    which the codecs take, from any), zeros past lens[b].  block_table [B, max_pages], lens and first [B] int32.
    stream: a torch stream or a handle; outputs made here are its memory."""
    import torch
    if S_out > _INT_MAX:
        raise ValueError("S_out: less than 2^31")
    gpu = _gpu(block_table, "block_table")
    args = _cache_args(cache, gpu)
    i32 = torch.int32
    B, max_pages = block_table.shape
    table = _typed(block_table, i32, (B, max_pages), "block_table", gpu)
    if dtype is None:
        dtype = torch.float16 if args[4] == VQ_E4M3 else cache["k_pages"].dtype
    shape = (B, args[6], S_out, args[8])
    dev = block_table.device
    ptrs = [None, None]
    outs = [k_out if want_k else None, v_out if want_v else None]
    for i, want in enumerate((want_k, want_v)):
        if not want:
            continue
        if outs[i] is None:
            outs[i] = torch.empty(shape, dtype=dtype, device=dev) if stream is None else _empty(shape, dtype, dev, stream)
            ptrs[i] = outs[i].data_ptr()
        else:
            ptrs[i] = _typed(outs[i], dtype, shape, "k_out, v_out", gpu)
    _check(_on_gpu(gpu, lib().vq_paged_gather)(*args, table, max_pages, _typed(lens, i32, (B,), "lens", gpu),
                                               None if first is None else _typed(first, i32, (B,), "first", gpu), B,
                                               S_out, _dtype_code(dtype), *ptrs, _raw_stream(stream, block_table)),
           "vq_paged_gather")
    return outs[0], outs[1]


def vq_paged_attend_workspace(T: int, B: int, Hq: int, Hkv: int, max_q: int) -> int:
    """Workspace bytes vq_paged_attend needs for these shapes on the current device."""
    n = ctypes.c_size_t(0)
    _check(lib().vq_paged_attend_workspace(T, B, Hq, Hkv, max_q, ctypes.byref(n)), "vq_paged_attend_workspace")
    return int(n.value)


_workspace_bytes: dict = {}  # sizes by shape and device: the call's own arithmetic, repeated every step


def _attend_args(sized, q, cache, block_table, cu_q, lens, max_q, window, sinks, out, workspace, stream, *more):
    """What the attention calls share: (out, gpu, arguments up to lens, (T, B, Hq, max_q,
    window, sinks), (out, workspace, bytes, stream)).  sized: the call's workspace
    function, which takes T, B, Hq, Hkv, max_q and `more`."""
    import torch
    if max_q > _INT_MAX or window > _INT_MAX or sinks > _INT_MAX:
        raise ValueError("max_q, window and sinks: less than 2^31")
    gpu = _gpu(q, "q")
    args = _cache_args(cache, gpu)
    i32 = torch.int32
    B, max_pages = block_table.shape
    T, Hq, _ = q.shape
    D, dtype, dev = args[8], q.dtype, q.device
    view = _rows_view(q, Hq, D, "q", gpu)
    table = _typed(block_table, i32, (B, max_pages), "block_table", gpu)
    cu, ln = _typed(cu_q, i32, (B + 1,), "cu_q", gpu), _typed(lens, i32, (B,), "lens", gpu)
    if out is None:
        shape = (T, Hq, D)
        out = torch.empty(shape, dtype=dtype, device=dev) if stream is None else _empty(shape, dtype, dev, stream)
        po = out.data_ptr()
    else:
        po = _typed(out, dtype, (T, Hq, D), "out", gpu)
    if workspace is None:
        key = (sized, T, B, Hq, args[6], max_q, gpu, more)
        wb = _workspace_bytes.get(key)
        if wb is None:
            if len(_workspace_bytes) > 4096:
                _workspace_bytes.clear()
            wb = _workspace_bytes[key] = _on_gpu(gpu, sized)(T, B, Hq, args[6], max_q, *more)
        wb = max(wb, 16)
        workspace = (torch.empty(wb, dtype=torch.uint8, device=dev) if stream is None
                     else _empty(wb, torch.uint8, dev, stream, returned=False))
    else:
        if workspace.get_device() != gpu or not workspace.is_contiguous():
            raise ValueError("workspace: a contiguous CUDA tensor on the GPU of the other tensors")
        wb = workspace.numel() * workspace.element_size()
    return (out, gpu, (*view, _dtype_code(dtype), *args, table, max_pages, cu, ln), (T, B, Hq, max_q, window, sinks),
            (po, workspace.data_ptr(), wb, _raw_stream(stream, q)), workspace)


def vq_paged_attend(q, cache: dict, block_table, cu_q, lens, scale: float, max_q: int, window: int = 0, sinks: int = 0,
                    out=None, workspace=None, stream=None):
    """Attention of new tokens q [T, Hq, 128] (rows may be strided) over a paged
    cache.  Sequence b has tokens cu_q[b] .. cu_q[b + 1] - 1 (at most max_q), the
    last of them at position lens[b] - 1; each sees the keys up to its own
    position, with a window those of the last `window` positions and the first
    `sinks`.  cu_q [B + 1], lens [B], block_table [B, max_pages] int32.  Returns
    [T, Hq, 128] of q's dtype; the workspace (uint8) is allocated when not given.
    stream: a torch stream or a handle; what is made here is its memory."""
    out, gpu, args, sizes, last, _held = _attend_args(vq_paged_attend_workspace, q, cache, block_table, cu_q, lens, max_q,
                                                      window, sinks, out, workspace, stream)
    _check(_on_gpu(gpu, lib().vq_paged_attend)(*args, *sizes, scale, *last), "vq_paged_attend")
    return out


def vq_paged_attend_tree_workspace(T: int, B: int, Hq: int, Hkv: int, max_q: int) -> int:
    """Workspace bytes vq_paged_attend_tree needs for these shapes on the current device."""
    n = ctypes.c_size_t(0)
    _check(lib().vq_paged_attend_tree_workspace(T, B, Hq, Hkv, max_q, ctypes.byref(n)), "vq_paged_attend_tree_workspace")
    return int(n.value)


def vq_paged_attend_tree(q, cache: dict, block_table, cu_q, lens, parents, scale: float, max_q: int, window: int = 0,
                         sinks: int = 0, out=None, workspace=None, stream=None):
    """Attention of a tree of drafted tokens of each sequence over a paged cache: as
    vq_paged_attend, but of the new tokens each sees itself and its ancestors.
    parents [T] int32: the new token of its sequence that a token follows (below
    its own index), or -1: the last token before the tree; a token's position is
    lens[b] - n_b plus its number of ancestors.  max_q: at most 256.  The drafted
    tokens are in the cache, in the order given; vq_paged_compact then moves an
    accepted path together."""
    import torch
    out, gpu, args, sizes, last, _held = _attend_args(vq_paged_attend_tree_workspace, q, cache, block_table, cu_q, lens,
                                                      max_q, window, sinks, out, workspace, stream)
    up = _typed(parents, torch.int32, (sizes[0],), "parents", gpu)
    _check(_on_gpu(gpu, lib().vq_paged_attend_tree)(*args, up, *sizes, scale, *last), "vq_paged_attend_tree")
    return out


def vq_paged_attend_weigh_workspace(T: int, B: int, Hq: int, Hkv: int, max_q: int, max_pages: int, page_size: int) -> int:
    """Workspace bytes vq_paged_attend_weigh needs for these shapes on the current device."""
    n = ctypes.c_size_t(0)
    _check(lib().vq_paged_attend_weigh_workspace(T, B, Hq, Hkv, max_q, max_pages, page_size, ctypes.byref(n)),
           "vq_paged_attend_weigh_workspace")
    return int(n.value)


def vq_paged_attend_weigh(q, cache: dict, weights, block_table, cu_q, lens, scale: float, max_q: int, window: int = 0,
                          sinks: int = 0, observe: int = 0, decay: float = 1.0, out=None, workspace=None, stream=None):
    """vq_paged_attend, which also adds up the softmax weight that each cached token
    gets: weights [num_pages, Hkv, page_size] (float32, updated in place) of every
    token that some new token sees become decay times what they were (of the new
    tokens: 0) plus the sum over the last `observe` new tokens of the sequence (0:
    all) and the query heads of the kv head.  decay acts once a call, however many
    tokens it has.  Sequences must not share pages.  The workspace grows with the
    block table's width (vq_paged_attend_weigh_workspace)."""
    import torch
    if observe > _INT_MAX:
        raise ValueError("observe: less than 2^31")
    shape = cache["k_pages"].shape
    w = _typed(weights, torch.float32, shape[:3], "weights", _gpu(q, "q"))
    out, gpu, args, sizes, last, _held = _attend_args(vq_paged_attend_weigh_workspace, q, cache, block_table, cu_q, lens,
                                                      max_q, window, sinks, out, workspace, stream, block_table.shape[1],
                                                      shape[2])
    _check(_on_gpu(gpu, lib().vq_paged_attend_weigh)(*args, *sizes, scale, w, observe, decay, *last), "vq_paged_attend_weigh")
    return out


def vq_paged_select(weights, block_table, lens, budget: int, recent: int = 0, sinks: int = 0, keep=None, counts=None,
                    stream=None):
    """The tokens that each sequence and kv head keeps by their accumulated weights
    [num_pages, Hkv, page_size] (float32): all, or the first `sinks`, the last
    `recent` and the heaviest in between, `budget` in all.  block_table
    [B, max_pages], lens [B] int32.  Returns (keep [B, Hkv, budget], ascending, -1
    behind the kept ones; counts [B]), int32.
    stream: a torch stream or a handle; outputs made here are its memory."""
    import torch
    if budget > _INT_MAX or recent > _INT_MAX or sinks > _INT_MAX:
        raise ValueError("budget, recent and sinks: less than 2^31")
    gpu = _gpu(block_table, "block_table")
    i32 = torch.int32
    NP, H, PS = weights.shape
    B, max_pages = block_table.shape
    w = _typed(weights, torch.float32, (NP, H, PS), "weights", gpu)
    table = _typed(block_table, i32, (B, max_pages), "block_table", gpu)
    ptrs, outs = [], [keep, counts]
    for i, (shape, name) in enumerate((((B, H, max(budget, 0)), "keep"), ((B,), "counts"))):
        if outs[i] is None:
            dev = block_table.device
            outs[i] = torch.empty(shape, dtype=i32, device=dev) if stream is None else _empty(shape, i32, dev, stream)
            ptrs.append(outs[i].data_ptr())
        else:
            ptrs.append(_typed(outs[i], i32, shape, name, gpu))
    _check(_on_gpu(gpu, lib().vq_paged_select)(w, NP, H, PS, table, max_pages, _typed(lens, i32, (B,), "lens", gpu), B,
                                               budget, recent, sinks, *ptrs, _raw_stream(stream, block_table)),
           "vq_paged_select")
    return outs[0], outs[1]


def vq_paged_compact(cache: dict, block_table, keep, counts, first=None, weights=None, stream=None) -> dict:
    """Move tokens of each sequence together, in place: token keep[b, h, i],
    i < counts[b], of kv head h goes to place first[b] + i (first None: i), with its
    exponents, and its weight in weights [num_pages, Hkv, page_size] (float32) where
    that is given.  keep [B, Hkv or 1, K] int32 (1: one list for all heads), rows
    ascending and contiguous, no token before its place; counts, first [B] and
    block_table [B, max_pages] int32.  Returns the cache."""
    import torch
    gpu = _gpu(block_table, "block_table")
    args = _cache_args(cache, gpu)
    i32 = torch.int32
    B, max_pages = block_table.shape
    table = _typed(block_table, i32, (B, max_pages), "block_table", gpu)
    shape = keep.shape
    if len(shape) != 3 or shape[0] != B or shape[1] not in (1, args[6]) or keep.dtype != i32 or keep.get_device() != gpu:
        raise ValueError("keep: an int32 CUDA tensor [%d, %d or 1, tokens] on the GPU of the other tensors" % (B, args[6]))
    st = keep.stride()
    if st[2] != 1 and shape[2] > 1:
        raise ValueError("keep: the entries of a list have to be contiguous")
    w = None if weights is None else _typed(weights, torch.float32, cache["k_pages"].shape[:3], "weights", gpu)
    _check(_on_gpu(gpu, lib().vq_paged_compact)(*args, table, max_pages, keep.data_ptr(), st[0],
                                                0 if shape[1] == 1 else st[1], shape[2],
                                                _typed(counts, i32, (B,), "counts", gpu),
                                                None if first is None else _typed(first, i32, (B,), "first", gpu), B, w,
                                                _raw_stream(stream, block_table)), "vq_paged_compact")
    return cache
