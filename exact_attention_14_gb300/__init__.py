"""GB300 (sm_103a) exact attention: fused forward (dense and packed
variable-length), backward, and split-KV decode (contiguous or paged cache); and
around it rotary positions, writing and reading the paged cache (bf16 or E4M3),
and attention of a tree of drafted tokens over that cache.

Thin ctypes binding over the C ABI in ``include/attn.h`` (library
``libgb300_attn.so`` built in-tree by ``_build.build()``).  The functions here
only marshal arguments -- shapes, data pointers and the CUDA stream -- and turn
status codes into exceptions; every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and streams.

There is no fallback: if the library is missing or was not built for this GPU,
the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

__all__ = [
    "ATTN_OUT_BF16", "ATTN_OUT_F32", "AttnError", "attn_fwd", "attn_fwd_workspace_size",
    "attn_fwd_varlen", "forward_varlen",
    "attn_fp8_quantize", "fp8_quantize", "attn_fwd_fp8", "forward_fp8", "attn_fp8_codes_bytes",
    "attn_fp8_descale_count",
    "attn_decode",
    "attn_decode_workspace_size", "attn_decode_noalloc", "attn_status_string", "attn_last_device_error",
    "attn_decode_num_splits", "attn_list_schedule", "attn_kv_tiles",
    "attn_fwd_num_units", "attn_fwd_schedule", "attn_fwd_split_plan", "attn_decode_kernel_launches",
    "attn_bwd", "attn_bwd_workspace_size", "backward", "attn_bwd_varlen",
    "attn_bwd_varlen_workspace_size", "backward_varlen", "attn_decode_paged", "decode_paged", "forward", "decode", "library_path", "load",
    "attn_rope", "rope", "rope_backward", "attn_rope_frequencies", "rope_frequencies",
    "attn_cache_write", "attn_cache_read", "cache_read", "attn_decode_tree",
    "attn_decode_tree_workspace_size", "decode_tree", "tree_mask_words",
]

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_TIMEOUT = 4
ATTN_ERR_WORKSPACE = 5
ATTN_OUT_BF16 = 0
ATTN_OUT_F32 = 1
ATTN_CACHE_BF16 = 0
ATTN_CACHE_E4M3 = 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgb300_attn.so")
_lib = None


class _Torch:
    """Stands in for torch until a call needs it: the host-only plans and
    frequencies work without torch and its import time."""
    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _Torch()

# Every symbol the header declares, with its ctypes signature.
_c_int, _c_ll, _c_sz, _c_f, _vp = (ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t,
                                   ctypes.c_float, ctypes.c_void_p)
SIGNATURES = {
    "attn_fwd": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                          _c_int, _c_int, _c_f, _c_int, _vp, _c_sz, _vp]),
    "attn_fwd_workspace_size": (_c_sz, [_c_int] * 7),
    "attn_fwd_varlen": (_c_int, [_vp] * 7 + [_c_int] * 9 + [_c_f, _c_int, _vp]),
    "attn_fp8_codes_bytes": (_c_sz, [_c_int] * 5),
    "attn_fp8_descale_count": (_c_sz, [_c_int] * 3),
    "attn_fp8_quantize": (_c_int, [_vp] * 4 + [_c_int] * 5 + [_vp]),
    "attn_fwd_fp8": (_c_int, [_vp] * 8 + [_c_int] * 7 + [_c_f, _c_int, _c_int, _vp]),
    "attn_selftest_bounded_wait": (_c_int, [_c_int, _vp, _vp]),
    "attn_decode_workspace_size": (_c_sz, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "attn_decode": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                             _c_int, _c_f, _c_int, _vp, _c_sz, _c_int, _vp]),
    "attn_decode_noalloc": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                     _c_int, _c_int, _c_f, _c_int, _c_int, _vp]),
    "attn_status_string": (ctypes.c_char_p, [_c_int]),
    "attn_last_device_error": (_c_int, [_vp]),
    "attn_decode_num_splits": (_c_int, [_c_int, _c_int, _c_int]),
    "attn_list_schedule": (_c_ll, [ctypes.POINTER(ctypes.c_int), _c_int, _c_int, _c_int,
                                   ctypes.POINTER(ctypes.c_longlong)]),
    "attn_kv_tiles": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "attn_fwd_num_units": (_c_ll, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "attn_fwd_schedule": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                   _c_int, _c_ll, ctypes.POINTER(ctypes.c_int),
                                   ctypes.POINTER(ctypes.c_int)]),
    "attn_decode_kernel_launches": (_c_int, [_c_int] * 6),
    "attn_bwd_workspace_size": (ctypes.c_size_t, [_c_int] * 6),
    "attn_bwd_varlen_workspace_size": (ctypes.c_size_t, [_c_int] * 5),
    "attn_bwd_varlen": (_c_int, [ctypes.c_void_p] * 11 + [_c_int] * 9 + [ctypes.c_float, _c_int, _c_int,
                                                                          ctypes.c_void_p, ctypes.c_size_t,
                                                                          ctypes.c_void_p]),
    "attn_decode_paged": (_c_int, [ctypes.c_void_p] * 7 + [_c_int, _c_int, _c_int, _c_ll, _c_int,
                                                            _c_int, _c_int, ctypes.c_float, _c_int,
                                                            ctypes.c_void_p, ctypes.c_size_t, _c_int,
                                                            ctypes.c_void_p]),
    "attn_bwd": (_c_int, [ctypes.c_void_p] * 9 + [_c_int] * 7 + [ctypes.c_float, _c_int, _c_int,
                                                                 ctypes.c_void_p, ctypes.c_size_t,
                                                                 ctypes.c_void_p]),
    "attn_rope_frequencies": (_c_int, [_c_int, ctypes.c_double, _c_int, ctypes.c_double, _c_int,
                                       ctypes.c_double, ctypes.c_double,
                                       ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_c_f)]),
    "attn_rope": (_c_int, [_vp] * 9 + [_c_ll, _vp] + [_c_int] * 8 + [_c_f, _c_int, _c_int, _vp]),
    "attn_cache_write": (_c_int, [_vp] * 9 + [_c_int] * 4 + [_c_ll, _c_int, _c_int, _vp]),
    "attn_cache_read": (_c_int, [_vp] * 8 + [_c_int] * 3 + [_c_ll] + [_c_int] * 5 + [_vp]),
    "attn_decode_tree_workspace_size": (_c_sz, [_c_int] * 8),
    "attn_decode_tree": (_c_int, [_vp] * 11 + [_c_int] * 4 + [_c_ll] + [_c_int] * 3 +
                         [_c_f, _c_int, _vp, _c_sz, _c_int, _vp]),
    "attn_fwd_split_plan": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                     _c_int, ctypes.POINTER(ctypes.c_int),
                                     ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
}


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {attn_status_string(code)} ({code})")


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` "
                "(there is no CPU fallback)")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def attn_status_string(code: int) -> str:
    return load().attn_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != ATTN_OK:
        raise AttnError(code, where)


def _current_stream(device):
    """Handle of a device's current stream; without a Stream object (2 us of a small
    call's 20) where torch has the call that its generated code makes."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream


def _stream_ptr(stream):
    if stream is None:   # the current stream of the current device
        return _current_stream(torch.cuda.current_device())
    return ctypes.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(ws):
    """(pointer, bytes) of an optional workspace tensor."""
    if ws is None:
        return None, 0
    _need(ws, ws.dtype, "workspace")
    return _ptr(ws), ws.numel() * ws.element_size()


def _one_device(*tensors):
    """The device of the given tensors (None entries skipped): the library
    launches on the current CUDA device, so every operand must live on one
    device, which the call then makes current."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"operands on different devices: {dev} and {t.device}")
    return dev


class _Here:
    """No change of device."""
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(dev):
    if dev.index == torch.cuda.current_device():   # (a switch and back costs more than a launch)
        return _HERE
    return torch.cuda.device(dev)


def attn_fwd_workspace_size(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int,
                            causal: bool) -> int:
    """Bytes of workspace attn_fwd needs for this shape on the current device
    (0 when it splits no unit)."""
    return int(load().attn_fwd_workspace_size(B, Hq, Hkv, Nq, Nk, d, int(bool(causal))))


def attn_fwd(q, k, v, o, lse=None, *, causal: bool = False, scale: float | None = None,
             workspace=None, stream=None):
    """Fused forward into caller-provided outputs.

    q [B,Hq,Nq,d] bf16; k, v [B,Hkv,Nk,d] bf16; o [B,Hq,Nq,d] bf16 or fp32;
    lse [B,Hq,Nq] fp32 or None; workspace: a CUDA tensor of at least
    attn_fwd_workspace_size(...) bytes, or None (then one is allocated with
    torch when the shape needs it).  Asynchronous on ``stream`` (default: the
    current torch stream)."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    if o.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("o must be bfloat16 or float32")
    _need(o, o.dtype, "o")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Hkv, Nk, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k/v shape mismatch")
    if tuple(o.shape) != (B, Hq, Nq, d):
        raise ValueError("o shape mismatch")
    if lse is not None and tuple(lse.shape) != (B, Hq, Nq):
        raise ValueError("lse shape mismatch")
    if scale is None:
        scale = d ** -0.5
    odt = ATTN_OUT_F32 if o.dtype == torch.float32 else ATTN_OUT_BF16
    dev = _one_device(q, k, v, o, lse, workspace)
    with _on(dev):
        if workspace is None:
            need = attn_fwd_workspace_size(B, Hq, Hkv, Nq, Nk, d, causal)
            if need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
                if isinstance(stream, torch.cuda.Stream):
                    workspace.record_stream(stream)   # freed only after that stream's use
        ws_ptr, ws_bytes = _workspace(workspace)
        rc = load().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d,
                             int(bool(causal)), float(scale), odt, ws_ptr, ws_bytes,
                             _stream_ptr(stream))
    _check(rc, "attn_fwd")
    return o, lse


def attn_fwd_varlen(q, k, v, o, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                    max_seqlen_k: int, lse=None, *, causal: bool = False,
                    scale: float | None = None, stream=None):
    """Packed variable-length forward into caller-provided outputs.

    q [total_q,Hq,d] bf16; k, v [total_k,Hkv,d] bf16; o [total_q,Hq,d] bf16 or
    fp32; cu_seqlens_q / cu_seqlens_k int32 [B+1] on the device (sequence b is
    rows cu[b]..cu[b+1]); lse [Hq,total_q] fp32 or None.  Asynchronous."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    for t, n in ((cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k")):
        _need(t, torch.int32, n)
    if o.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("o must be bfloat16 or float32")
    _need(o, o.dtype, "o")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    total_q, Hq, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    if tuple(k.shape) != (total_k, Hkv, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k/v shape mismatch")
    if tuple(o.shape) != tuple(q.shape):
        raise ValueError("o shape mismatch")
    B = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != B + 1 or B < 1:
        raise ValueError("cu_seqlens_q / cu_seqlens_k must both have B + 1 entries")
    if lse is not None and tuple(lse.shape) != (Hq, total_q):
        raise ValueError("lse shape mismatch")
    if scale is None:
        scale = d ** -0.5
    odt = ATTN_OUT_F32 if o.dtype == torch.float32 else ATTN_OUT_BF16
    with _on(_one_device(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k)):
        rc = load().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                    _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, Hq, Hkv, total_q,
                                    total_k, int(max_seqlen_q), int(max_seqlen_k), d,
                                    int(bool(causal)), float(scale), odt, _stream_ptr(stream))
    _check(rc, "attn_fwd_varlen")
    return o, lse


def forward_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                   *, causal: bool = False, scale: float | None = None, out_dtype=None,
                   return_lse: bool = True, stream=None):
    """Allocate O (and LSE [Hq, total_q]) with torch and run attn_fwd_varlen."""
    import torch
    out_dtype = out_dtype or torch.bfloat16
    o = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    lse = (torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
           if return_lse else None)
    return attn_fwd_varlen(q, k, v, o, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                           lse, causal=causal, scale=scale, stream=stream)


def attn_fp8_codes_bytes(B: int, H: int, N: int, d: int, transpose: bool = False) -> int:
    return int(load().attn_fp8_codes_bytes(B, H, N, d, int(bool(transpose))))


def attn_fp8_descale_count(B: int, H: int, N: int) -> int:
    return int(load().attn_fp8_descale_count(B, H, N))


def attn_fp8_quantize(x, codes, descale, signs=None, *, transpose: bool = False, stream=None):
    """Block-quantize x [B,H,N,d] bf16 into caller-provided E4M3 codes (uint8
    [B,H,N,d], or [B,H,d,Np] when transpose) and descale [B,H,ceil(N/128)]
    fp32; signs: None or an int8 tensor of d values +-1 (rotate first)."""
    import torch
    _need(x, torch.bfloat16, "x")
    _need(codes, torch.uint8, "codes")
    _need(descale, torch.float32, "descale")
    if signs is not None:
        _need(signs, torch.int8, "signs")
    B, H, N, d = x.shape
    if signs is not None and signs.numel() != d:
        raise ValueError("signs must hold d values")
    npad = (N + 15) // 16 * 16
    want = (B, H, d, npad) if transpose else (B, H, N, d)
    if tuple(codes.shape) != want:
        raise ValueError(f"codes must be {want}")
    if tuple(descale.shape) != (B, H, (N + 127) // 128):
        raise ValueError("descale shape mismatch")
    with _on(_one_device(x, codes, descale, signs)):
        rc = load().attn_fp8_quantize(_ptr(x), _ptr(codes), _ptr(descale), _ptr(signs), B, H, N, d,
                                      int(bool(transpose)), _stream_ptr(stream))
    _check(rc, "attn_fp8_quantize")
    return codes, descale


def fp8_quantize(x, signs=None, *, transpose: bool = False, stream=None):
    """Allocate the codes and scales with torch and run attn_fp8_quantize."""
    import torch
    B, H, N, d = x.shape
    npad = (N + 15) // 16 * 16
    shape = (B, H, d, npad) if transpose else (B, H, N, d)
    codes = (torch.zeros if transpose else torch.empty)(shape, dtype=torch.uint8, device=x.device)
    descale = torch.empty((B, H, (N + 127) // 128), dtype=torch.float32, device=x.device)
    return attn_fp8_quantize(x, codes, descale, signs, transpose=transpose, stream=stream)


def attn_fwd_fp8(q8, k8, vt8, q_descale, k_descale, v_descale, o, lse=None, *,
                 causal: bool = False, scale: float | None = None, rotated: bool = False,
                 stream=None):
    """Forward on E4M3 operands into caller-provided outputs: q8 [B,Hq,Nq,128],
    k8 [B,Hkv,Nk,128], vt8 [B,Hkv,128,Np] (uint8 codes), descales fp32
    [B,H,ceil(N/128)]; o [B,Hq,Nq,128] bf16/fp32; lse [B,Hq,Nq] or None.
    scale is the original problem's softmax scale; rotated: Q and K were
    quantized with the same Hadamard signs (the library then divides the
    scale by d)."""
    import torch
    for t, n in ((q8, "q8"), (k8, "k8"), (vt8, "vt8")):
        _need(t, torch.uint8, n)
    for t, n in ((q_descale, "q_descale"), (k_descale, "k_descale"), (v_descale, "v_descale")):
        _need(t, torch.float32, n)
    if o.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("o must be bfloat16 or float32")
    _need(o, o.dtype, "o")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    B, Hq, Nq, d = q8.shape
    Hkv, Nk = k8.shape[1], k8.shape[2]
    if tuple(k8.shape) != (B, Hkv, Nk, d) or tuple(vt8.shape) != (B, Hkv, d, (Nk + 15) // 16 * 16):
        raise ValueError("k8 / vt8 shape mismatch")
    if tuple(o.shape) != (B, Hq, Nq, d):
        raise ValueError("o shape mismatch")
    if lse is not None and tuple(lse.shape) != (B, Hq, Nq):
        raise ValueError("lse shape mismatch")
    nbq, nbk = (Nq + 127) // 128, (Nk + 127) // 128
    if (tuple(q_descale.shape) != (B, Hq, nbq) or tuple(k_descale.shape) != (B, Hkv, nbk)
            or tuple(v_descale.shape) != (B, Hkv, nbk)):
        raise ValueError("descale shape mismatch")
    if scale is None:
        scale = d ** -0.5
    odt = ATTN_OUT_F32 if o.dtype == torch.float32 else ATTN_OUT_BF16
    with _on(_one_device(q8, k8, vt8, q_descale, k_descale, v_descale, o, lse)):
        rc = load().attn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(vt8), _ptr(q_descale), _ptr(k_descale),
                                 _ptr(v_descale), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d,
                                 int(bool(causal)), float(scale), int(bool(rotated)), odt,
                                 _stream_ptr(stream))
    _check(rc, "attn_fwd_fp8")
    return o, lse


def forward_fp8(q, k, v, *, causal: bool = False, scale: float | None = None, signs=None,
                out_dtype=None, return_lse: bool = True, stream=None):
    """bf16 q, k, v -> E4M3 (Q and K rotated by diag(signs) H when signs is
    given: an int8 tensor of d values +-1) -> attn_fwd_fp8.  Returns (O, LSE)."""
    import torch
    d = q.shape[-1]
    if scale is None:
        scale = d ** -0.5
    q8, qd = fp8_quantize(q, signs, stream=stream)
    k8, kd = fp8_quantize(k, signs, stream=stream)
    vt8, vd = fp8_quantize(v, None, transpose=True, stream=stream)
    out_dtype = out_dtype or torch.bfloat16
    o = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    lse = (torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
           if return_lse else None)
    return attn_fwd_fp8(q8, k8, vt8, qd, kd, vd, o, lse, causal=causal, scale=scale,
                        rotated=signs is not None, stream=stream)


def attn_bwd_workspace_size(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    return int(load().attn_bwd_workspace_size(B, Hq, Hkv, Nq, Nk, d))


def attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, *, causal: bool = False,
             scale: float | None = None, workspace=None, stream=None):
    """Backward into caller-provided gradients.

    q, dout [B,Hq,Nq,d] bf16; k, v [B,Hkv,Nk,d] bf16; o [B,Hq,Nq,d] bf16 or
    fp32 (the forward's output); lse [B,Hq,Nq] fp32 (the forward's natural-log
    logsumexp); dq [B,Hq,Nq,d] and dk, dv [B,Hkv,Nk,d], all bf16 or all fp32;
    workspace: uint8 of attn_bwd_workspace_size bytes.  Asynchronous."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _need(t, torch.bfloat16, n)
    if o.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("o must be bfloat16 or float32")
    _need(o, o.dtype, "o")
    _need(lse, torch.float32, "lse")
    gdt = dq.dtype
    if gdt not in (torch.bfloat16, torch.float32) or dk.dtype != gdt or dv.dtype != gdt:
        raise TypeError("dq, dk, dv must all be bfloat16 or all float32")
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, gdt, n)
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if (tuple(k.shape) != (B, Hkv, Nk, d) or tuple(v.shape) != tuple(k.shape)
            or tuple(dk.shape) != tuple(k.shape) or tuple(dv.shape) != tuple(k.shape)):
        raise ValueError("k/v/dk/dv shape mismatch")
    if tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape) \
            or tuple(dq.shape) != tuple(q.shape):
        raise ValueError("o/dout/dq shape mismatch")
    if tuple(lse.shape) != (B, Hq, Nq):
        raise ValueError("lse shape mismatch")
    if scale is None:
        scale = d ** -0.5
    need = attn_bwd_workspace_size(B, Hq, Hkv, Nq, Nk, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if isinstance(stream, torch.cuda.Stream):
            workspace.record_stream(stream)   # freed only after that stream's use
    odt = ATTN_OUT_F32 if o.dtype == torch.float32 else ATTN_OUT_BF16
    g32 = ATTN_OUT_F32 if gdt == torch.float32 else ATTN_OUT_BF16
    with _on(_one_device(q, k, v, o, dout, lse, dq, dk, dv, workspace)):
        rc = load().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                             _ptr(dk), _ptr(dv), B, Hq, Hkv, Nq, Nk, d, int(bool(causal)),
                             float(scale), odt, g32, _ptr(workspace), workspace.numel(),
                             _stream_ptr(stream))
    _check(rc, "attn_bwd")
    return dq, dk, dv


def backward(q, k, v, o, dout, lse, *, causal: bool = False, scale: float | None = None,
             grad_dtype=None, stream=None):
    """Allocate dQ, dK, dV (and the workspace) with torch and run attn_bwd."""
    import torch
    grad_dtype = grad_dtype or torch.bfloat16
    dq = torch.empty(q.shape, dtype=grad_dtype, device=q.device)
    dk = torch.empty(k.shape, dtype=grad_dtype, device=q.device)
    dv = torch.empty(v.shape, dtype=grad_dtype, device=q.device)
    return attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, causal=causal, scale=scale,
                    stream=stream)


def attn_bwd_varlen_workspace_size(B: int, Hq: int, Hkv: int, total_q: int, d: int) -> int:
    return int(load().attn_bwd_varlen_workspace_size(B, Hq, Hkv, total_q, d))


def attn_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k,
                    max_seqlen_q: int, max_seqlen_k: int, *, causal: bool = False,
                    scale: float | None = None, workspace=None, stream=None):
    """Packed variable-length backward into caller-provided gradients.

    q, dout [total_q,Hq,d] bf16; k, v [total_k,Hkv,d] bf16; o [total_q,Hq,d]
    bf16 or fp32 and lse [Hq,total_q] fp32 from attn_fwd_varlen; dq
    [total_q,Hq,d] and dk, dv [total_k,Hkv,d], all bf16 or all fp32;
    cu_seqlens_q / cu_seqlens_k int32 [B+1] on the device; workspace: uint8 of
    attn_bwd_varlen_workspace_size bytes.  Asynchronous."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _need(t, torch.bfloat16, n)
    for t, n in ((cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k")):
        _need(t, torch.int32, n)
    if o.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("o must be bfloat16 or float32")
    _need(o, o.dtype, "o")
    _need(lse, torch.float32, "lse")
    gdt = dq.dtype
    if gdt not in (torch.bfloat16, torch.float32) or dk.dtype != gdt or dv.dtype != gdt:
        raise TypeError("dq, dk, dv must all be bfloat16 or all float32")
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, gdt, n)
    total_q, Hq, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    if (tuple(k.shape) != (total_k, Hkv, d) or tuple(v.shape) != tuple(k.shape)
            or tuple(dk.shape) != tuple(k.shape) or tuple(dv.shape) != tuple(k.shape)):
        raise ValueError("k/v/dk/dv shape mismatch")
    if tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape) \
            or tuple(dq.shape) != tuple(q.shape):
        raise ValueError("o/dout/dq shape mismatch")
    B = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != B + 1 or B < 1:
        raise ValueError("cu_seqlens_q / cu_seqlens_k must both have B + 1 entries")
    if tuple(lse.shape) != (Hq, total_q):
        raise ValueError("lse shape mismatch")
    if scale is None:
        scale = d ** -0.5
    dev = _one_device(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, workspace)
    with _on(dev):
        if workspace is None:
            workspace = torch.empty(attn_bwd_varlen_workspace_size(B, Hq, Hkv, total_q, d),
                                    dtype=torch.uint8, device=dev)
            if isinstance(stream, torch.cuda.Stream):
                workspace.record_stream(stream)   # freed only after that stream's use
        ws_ptr, ws_bytes = _workspace(workspace)
        odt = ATTN_OUT_F32 if o.dtype == torch.float32 else ATTN_OUT_BF16
        g32 = ATTN_OUT_F32 if gdt == torch.float32 else ATTN_OUT_BF16
        rc = load().attn_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                    _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens_q),
                                    _ptr(cu_seqlens_k), B, Hq, Hkv, total_q, total_k,
                                    int(max_seqlen_q), int(max_seqlen_k), d, int(bool(causal)),
                                    float(scale), odt, g32, ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(rc, "attn_bwd_varlen")
    return dq, dk, dv


def backward_varlen(q, k, v, o, dout, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                    max_seqlen_k: int, *, causal: bool = False, scale: float | None = None,
                    grad_dtype=None, stream=None):
    """Allocate dQ, dK, dV (and the workspace) with torch and run attn_bwd_varlen."""
    import torch
    grad_dtype = grad_dtype or torch.bfloat16
    dq = torch.empty(q.shape, dtype=grad_dtype, device=q.device)
    dk = torch.empty(k.shape, dtype=grad_dtype, device=q.device)
    dv = torch.empty(v.shape, dtype=grad_dtype, device=q.device)
    return attn_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k,
                           max_seqlen_q, max_seqlen_k, causal=causal, scale=scale, stream=stream)


def forward(q, k, v, *, causal: bool = False, scale: float | None = None,
            out_dtype=None, return_lse: bool = True, stream=None):
    """Allocate O (and LSE) with torch and run attn_fwd."""
    import torch
    out_dtype = out_dtype or torch.bfloat16
    o = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    lse = (torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
           if return_lse else None)
    return attn_fwd(q, k, v, o, lse, causal=causal, scale=scale, stream=stream)


def attn_decode_workspace_size(B: int, Hq: int, Hkv: int, Nmax: int, d: int,
                               num_splits: int = 0) -> int:
    return int(load().attn_decode_workspace_size(B, Hq, Hkv, Nmax, d, num_splits))


def _check_decode_args(q, k_cache, v_cache, seqlens, o, lse):
    """Types and shapes of a contiguous-cache decode call (everything the
    kernels index by): q [B,Hq,1,d] bf16, caches [B,Hkv,Nmax,d] bf16, seqlens
    [B] int32, o [B,Hq,1,d] bf16/fp32, lse [B,Hq,1] fp32 or None.  Returns
    (B, Hq, Hkv, Nmax, d)."""
    import torch
    named = [(q, "q", torch.bfloat16), (k_cache, "k_cache", torch.bfloat16),
             (v_cache, "v_cache", torch.bfloat16), (seqlens, "seqlens", torch.int32)]
    if lse is not None:
        named.append((lse, "lse", torch.float32))
    # types, then shapes, then placement: each is checked before any pointer
    # reaches the library
    for t, n, dt in named:
        if not isinstance(t, torch.Tensor) or t.dtype != dt:
            raise TypeError(f"{n} must be a {dt} tensor")
    if not isinstance(o, torch.Tensor) or o.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("o must be a bfloat16 or float32 tensor")
    if q.ndim != 4 or k_cache.ndim != 4:
        raise ValueError("q and the caches must be 4-D")
    B, Hq, one, d = q.shape
    Hkv, Nmax = k_cache.shape[1], k_cache.shape[2]
    if one != 1 or tuple(k_cache.shape) != (B, Hkv, Nmax, d) or v_cache.shape != k_cache.shape:
        raise ValueError("decode shape mismatch")
    if tuple(o.shape) != (B, Hq, 1, d) or tuple(seqlens.shape) != (B,):
        raise ValueError("decode output/seqlens shape mismatch")
    if lse is not None and tuple(lse.shape) != (B, Hq, 1):
        raise ValueError("lse shape mismatch")
    for t, n, dt in named + [(o, "o", o.dtype)]:
        _need(t, dt, n)
    return B, Hq, Hkv, Nmax, d


def attn_decode(q, k_cache, v_cache, seqlens, o, lse=None, *, scale: float | None = None,
                num_splits: int = 0, workspace=None, stream=None):
    """Split-KV decode into caller-provided outputs.

    q [B,Hq,1,d] bf16; caches [B,Hkv,Nmax,d] bf16; seqlens [B] int32 (device);
    o [B,Hq,1,d] bf16/fp32; lse [B,Hq,1] fp32 or None; workspace: a uint8
    CUDA tensor of at least attn_decode_workspace_size(...) bytes."""
    import torch
    B, Hq, Hkv, Nmax, d = _check_decode_args(q, k_cache, v_cache, seqlens, o, lse)
    if scale is None:
        scale = d ** -0.5
    ws_ptr, ws_bytes = _workspace(workspace)
    odt = ATTN_OUT_F32 if o.dtype == torch.float32 else ATTN_OUT_BF16
    with _on(_one_device(q, k_cache, v_cache, seqlens, o, lse)):
        rc = load().attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), _ptr(o),
                                _ptr(lse), B, Hq, Hkv, Nmax, d, float(scale), int(num_splits),
                                ws_ptr, ws_bytes, odt, _stream_ptr(stream))
    _check(rc, "attn_decode")
    return o, lse


def decode(q, k_cache, v_cache, seqlens, *, scale=None, num_splits: int = 0,
           out_dtype=None, stream=None):
    """Allocate O, LSE and the workspace with torch and run attn_decode."""
    import torch
    out_dtype = out_dtype or torch.bfloat16
    B, Hq, _, d = q.shape
    Hkv, Nmax = k_cache.shape[1], k_cache.shape[2]
    ws = torch.empty(attn_decode_workspace_size(B, Hq, Hkv, Nmax, d, num_splits),
                     dtype=torch.uint8, device=q.device)
    o = torch.empty((B, Hq, 1, d), dtype=out_dtype, device=q.device)
    lse = torch.empty((B, Hq, 1), dtype=torch.float32, device=q.device)
    return attn_decode(q, k_cache, v_cache, seqlens, o, lse, scale=scale,
                       num_splits=num_splits, workspace=ws, stream=stream)


def attn_decode_noalloc(q, k_cache, v_cache, seqlens, o, lse=None, *,
                        scale: float | None = None, num_splits: int = 0, stream=None):
    """attn_decode without a workspace argument, for callers that cannot
    allocate device memory: the library's fixed 16 MiB per-device scratch array
    holds the split partials.  Calls that overlap on the GPU share that array
    and race; calls ordered on one stream do not.  The first call on a device
    must come before any stream capture."""
    import torch
    B, Hq, Hkv, Nmax, d = _check_decode_args(q, k_cache, v_cache, seqlens, o, lse)
    if scale is None:
        scale = d ** -0.5
    odt = ATTN_OUT_F32 if o.dtype == torch.float32 else ATTN_OUT_BF16
    with _on(_one_device(q, k_cache, v_cache, seqlens, o, lse)):
        rc = load().attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), _ptr(o),
                                        _ptr(lse), B, Hq, Hkv, Nmax, d, float(scale),
                                        int(num_splits), odt, _stream_ptr(stream))
    _check(rc, "attn_decode_noalloc")
    return o, lse


def attn_selftest_bounded_wait(mode: int, result, stream=None) -> None:
    """Run the bounded-wait diagnostic (mode 0: time out; mode 1: abort flag)
    writing its outcome into `result` (an int32 CUDA tensor of one element)."""
    import torch
    _need(result, torch.int32, "result")
    with _on(_one_device(result)):
        _check(load().attn_selftest_bounded_wait(int(mode), _ptr(result), _stream_ptr(stream)),
               "attn_selftest_bounded_wait")


def attn_last_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return int(load().attn_last_device_error(_stream_ptr(stream)))


# ------------------------- host-side scheduling logic -------------------------
def attn_decode_num_splits(units: int, num_sms: int, max_splits: int = 128) -> int:
    return int(load().attn_decode_num_splits(units, num_sms, max_splits))


def attn_list_schedule(costs, workers: int, lpt: bool):
    """Returns (makespan, per-worker loads)."""
    n = len(costs)
    arr = (ctypes.c_int * max(n, 1))(*[int(c) for c in costs])
    loads = (ctypes.c_longlong * workers)()
    mk = load().attn_list_schedule(arr, n, workers, int(bool(lpt)), loads)
    if mk < 0:
        raise ValueError("attn_list_schedule rejected its arguments")
    return int(mk), [int(x) for x in loads]


def attn_kv_tiles(row0: int, rows: int, Nq: int, Nk: int, causal: bool, block: int) -> int:
    return int(load().attn_kv_tiles(row0, rows, Nq, Nk, int(bool(causal)), block))


def attn_fwd_num_units(B, Hq, Hkv, Nq, Nk, d, causal) -> int:
    return int(load().attn_fwd_num_units(B, Hq, Hkv, Nq, Nk, d, int(bool(causal))))


def attn_fwd_schedule(B, Hq, Hkv, Nq, Nk, d, causal, num_sms: int = 0):
    """Returns ([(b, hq, m_block), ...] in walk order, [cost, ...]) for a GPU
    with num_sms SMs (0: the fixed section widths)."""
    n = attn_fwd_num_units(B, Hq, Hkv, Nq, Nk, d, causal)
    units = (ctypes.c_int * (3 * n))()
    costs = (ctypes.c_int * n)()
    rc = load().attn_fwd_schedule(B, Hq, Hkv, Nq, Nk, d, int(bool(causal)), int(num_sms), n,
                                  units, costs)
    if rc != 0:
        raise ValueError("attn_fwd_schedule rejected its arguments")
    return [tuple(units[3 * i:3 * i + 3]) for i in range(n)], list(costs)


def attn_fwd_split_plan(B, Hq, Hkv, Nq, Nk, d, causal, num_sms):
    """Returns (n_full, n_split, parts): the tail split attn_fwd applies on a
    GPU with num_sms SMs."""
    out = [ctypes.c_int() for _ in range(3)]
    rc = load().attn_fwd_split_plan(B, Hq, Hkv, Nq, Nk, d, int(bool(causal)), num_sms,
                                    *(ctypes.byref(o) for o in out))
    if rc != 0:
        raise ValueError("attn_fwd_split_plan rejected its arguments")
    return tuple(o.value for o in out)


def attn_decode_kernel_launches(B, Hq, Hkv, Nmax, d, num_splits=0) -> int:
    """Kernels attn_decode launches for this shape: 1 (the split kernel merges)
    or 2 (split + combine)."""
    n = int(load().attn_decode_kernel_launches(B, Hq, Hkv, Nmax, d, num_splits))
    if n < 0:
        raise ValueError("attn_decode_kernel_launches rejected its arguments")
    return n


def attn_decode_paged(q, k_pages, v_pages, block_table, seqlens, o, lse=None, *,
                      scale: float | None = None, num_splits: int = 0, workspace=None,
                      stream=None):
    """Decode over a paged KV cache into caller-provided outputs.

    q [B,Hq,1,d] bf16; k_pages, v_pages [num_blocks, page_size, Hkv, d] bf16;
    block_table [B, max_blocks] int32; seqlens [B] int32; o [B,Hq,1,d] bf16
    or fp32; lse [B,Hq,1] fp32 or None.  Asynchronous."""
    import torch
    named = [(q, "q", torch.bfloat16), (k_pages, "k_pages", torch.bfloat16),
             (v_pages, "v_pages", torch.bfloat16), (block_table, "block_table", torch.int32),
             (seqlens, "seqlens", torch.int32)]
    if lse is not None:
        named.append((lse, "lse", torch.float32))
    for t, n, dt in named:   # types, then shapes, then placement
        if not isinstance(t, torch.Tensor) or t.dtype != dt:
            raise TypeError(f"{n} must be a {dt} tensor")
    if not isinstance(o, torch.Tensor) or o.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("o must be a bfloat16 or float32 tensor")
    if q.ndim != 4 or k_pages.ndim != 4:
        raise ValueError("q and the pages must be 4-D")
    B, Hq, one, d = q.shape
    num_blocks, page_size, Hkv, dk = k_pages.shape
    if one != 1 or dk != d or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("q / page shapes mismatch")
    if block_table.ndim != 2 or block_table.shape[0] != B or tuple(seqlens.shape) != (B,):
        raise ValueError("block_table must be [B, max_blocks] and seqlens [B]")
    if tuple(o.shape) != (B, Hq, 1, d):
        raise ValueError("o shape mismatch")
    if lse is not None and tuple(lse.shape) != (B, Hq, 1):
        raise ValueError("lse shape mismatch")
    for t, n, dt in named + [(o, "o", o.dtype)]:
        _need(t, dt, n)
    max_blocks = block_table.shape[1]
    if scale is None:
        scale = d ** -0.5
    need = attn_decode_workspace_size(B, Hq, Hkv, max_blocks * page_size, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    odt = ATTN_OUT_F32 if o.dtype == torch.float32 else ATTN_OUT_BF16
    with _on(_one_device(q, k_pages, v_pages, block_table, seqlens, o, lse, workspace)):
        rc = load().attn_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                                      _ptr(seqlens), _ptr(o), _ptr(lse), B, Hq, Hkv, num_blocks,
                                      page_size, max_blocks, d, float(scale), num_splits,
                                      _ptr(workspace), workspace.numel(), odt, _stream_ptr(stream))
    _check(rc, "attn_decode_paged")
    return o, lse


def decode_paged(q, k_pages, v_pages, block_table, seqlens, *, scale: float | None = None,
                 num_splits: int = 0, out_dtype=None, stream=None):
    """Allocate O and LSE with torch and run attn_decode_paged."""
    import torch
    out_dtype = out_dtype or torch.bfloat16
    B, Hq, _, d = q.shape
    o = torch.empty((B, Hq, 1, d), dtype=out_dtype, device=q.device)
    lse = torch.empty((B, Hq, 1), dtype=torch.float32, device=q.device)
    return attn_decode_paged(q, k_pages, v_pages, block_table, seqlens, o, lse, scale=scale,
                             num_splits=num_splits, stream=stream)


# ------------------- positions, the paged cache, drafted tokens -------------------
_Strides = ctypes.c_longlong * 3


def _tensor(t, dtypes, name):
    """A CUDA tensor of one of the given dtypes (any layout)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _at(t):
    """Address of an optional tensor."""
    return None if t is None else t.data_ptr()


def _rows(t, name):
    """(B, H, N, d) and the host strides {batch, head, token} (None: contiguous)
    of a [B,H,N,d] view or a packed [total,H,d] one (B = 1), whose rows are
    contiguous and 16-byte aligned."""
    nd = t.ndim
    if nd == 4:
        B, H, N, d = shape = t.shape
        if t.is_contiguous() and B and H and N and d and not t.data_ptr() % 16:
            return shape, None   # (row lengths that are no multiple of 16 bytes the library refuses)
        sb, sh, sn, sd = t.stride()
        if B == 1:
            sb = 0
    elif nd == 3:
        N, H, d = t.shape
        sn, sh, sd = t.stride()
        B, sb = 1, 0
    else:
        raise ValueError(f"{name} must be [B, H, N, d] or packed [total, H, d]")
    if not (B and H and N and d):
        raise ValueError(f"{name} is empty")
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if H == 1:
        sh = 0
    if N == 1:
        sn = 0
    if (sb | sh | sn) % (16 // t.element_size()) or t.data_ptr() % 16:
        raise ValueError(f"{name}: rows must be 16-byte aligned")
    return (B, H, N, d), _Strides(sb, sh, sn)


def _made_on(stream, dev):
    """Where the outputs and workspaces of a call on ``stream`` are allocated: on
    that stream, since a block of the current stream's may still be in use by work
    queued there."""
    if stream is None:
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        at = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(at, device=dev) if at else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


def _used_here(dev, *tensors):
    """Outputs made on a stream of the caller's, which are read on the current one
    too: a block is given out again only after that use."""
    here = torch.cuda.current_stream(dev)
    for t in tensors:
        if t is not None:
            t.record_stream(here)


def attn_rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none",
                          factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0,
                          beta_slow: float = 1.0):
    """([inv_freq, ...] in radians per position, magnitude) as Python floats.
    scaling: "none", "linear", "ntk" or "by_parts" (the last needs
    original_len, the trained context)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    out = (ctypes.c_double * max(int(rotary_dim) // 2, 1))()
    mag = _c_f()
    _check(load().attn_rope_frequencies(int(rotary_dim), float(base), ROPE_SCALINGS[scaling],
                                        float(factor), int(original_len), float(beta_fast),
                                        float(beta_slow), out, ctypes.byref(mag)),
           "attn_rope_frequencies")
    return list(out), mag.value


def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none",
                     factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, device="cuda"):
    """(inv_freq float64 tensor [rotary_dim / 2] on ``device``, magnitude) for
    rope() and rope_backward(); see attn_rope_frequencies."""
    f, mag = attn_rope_frequencies(rotary_dim, base, scaling=scaling, factor=factor,
                                   original_len=original_len, beta_fast=beta_fast,
                                   beta_slow=beta_slow)
    return torch.tensor(f, dtype=torch.float64, device=device), mag


def _rope_inputs(q, k):
    """Checks q and k; returns (B, Hq, Hkv, N, d) and their strides."""
    _tensor(q, (torch.bfloat16, torch.float32), "q")
    (B, Hq, N, d), qs = _rows(q, "q")
    if k is None:
        return B, Hq, 0, N, d, qs, None
    _tensor(k, (q.dtype,), "k")
    (Bk, Hkv, Nk, dk), ks = _rows(k, "k")
    if Bk != B or Nk != N or dk != d or k.ndim != q.ndim:
        raise ValueError("q / k shape mismatch")
    return B, Hq, Hkv, N, d, qs, ks


def _rope_call(q, k, q_out, k_out, positions, inv_freq, shape, qos, kos, interleaved, inverse,
               magnitude, stream):
    """attn_rope once q, k and the outputs are known to be good."""
    B, Hq, Hkv, N, d, qs, ks = shape
    _tensor(positions, (torch.int32,), "positions")
    _need(inv_freq, torch.float64, "inv_freq")
    if positions.shape == (N,):
        pos_stride = 0
    elif positions.shape == (B, N):
        pos_stride = positions.stride(0) if B > 1 else 0
    else:
        raise ValueError("positions must be [B, N] or [N]")
    if N > 1 and positions.stride(-1) != 1:
        raise ValueError("positions: the last dimension must be contiguous")
    pairs = inv_freq.shape[0] if inv_freq.ndim == 1 else 0
    if not 1 <= pairs <= d // 2:
        raise ValueError("inv_freq must hold rotary_dim / 2 <= d / 2 frequencies")
    idt = ATTN_OUT_F32 if q.dtype == torch.float32 else ATTN_OUT_BF16
    odt = ATTN_OUT_F32 if q_out.dtype == torch.float32 else ATTN_OUT_BF16
    with _on(_one_device(q, k, q_out, k_out, positions, inv_freq)):
        rc = load().attn_rope(q.data_ptr(), _at(k), q_out.data_ptr(), _at(k_out), qs, ks, qos, kos,
                              positions.data_ptr(), pos_stride, inv_freq.data_ptr(), B, Hq, Hkv, N, d,
                              2 * pairs, 1 if interleaved else 0, 1 if inverse else 0, magnitude, idt,
                              odt, _stream_ptr(stream))
    _check(rc, "attn_rope")
    return q_out, k_out


def attn_rope(q, k, q_out, k_out, positions, inv_freq, *, interleaved: bool = False,
              inverse: bool = False, magnitude: float = 1.0, stream=None):
    """Rotary positions on q and k (k and k_out may be None) into caller-provided
    outputs, one launch.

    q, q_out [B,Hq,N,d] and k, k_out [B,Hkv,N,d], or packed [total,H,d]; bf16 or
    fp32 (q and k alike, the outputs alike); any strides with contiguous,
    16-byte-aligned rows, so a slice of a projection's [B,N,H,d] output works as
    q.transpose(1, 2).  positions int32 [B,N] or [N] ([total] for packed
    tensors); inv_freq float64 [rotary_dim / 2] (rope_frequencies); the columns
    past rotary_dim are copied.  inverse: the gradient.  In place when an output
    is its input.  Asynchronous on ``stream``."""
    shape = _rope_inputs(q, k)
    B, Hq, Hkv, N, d = shape[:5]
    _tensor(q_out, (torch.bfloat16, torch.float32), "q_out")
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    if q_out.shape != q.shape:
        raise ValueError("q_out shape mismatch")
    _, qos = _rows(q_out, "q_out")
    kos = None
    if k is not None:
        _tensor(k_out, (q_out.dtype,), "k_out")
        if k_out.shape != k.shape:
            raise ValueError("k_out shape mismatch")
        _, kos = _rows(k_out, "k_out")
    return _rope_call(q, k, q_out, k_out, positions, inv_freq, shape, qos, kos, interleaved,
                      inverse, magnitude, stream)


def _new_rows(x, dtype, H, N, d):
    """A contiguous output of x's shape and its strides."""
    if dtype == x.dtype and x.is_contiguous():
        out = torch.empty_like(x)
    else:
        out = torch.empty(x.shape, dtype=dtype, device=x.device)
    return out, None if x.ndim == 4 else _Strides(0, d if H > 1 else 0, H * d if N > 1 else 0)


def rope(q, k, positions, inv_freq, *, interleaved: bool = False, magnitude: float = 1.0,
         out_dtype=None, stream=None, inverse: bool = False):
    """Allocate the outputs (contiguous, of q's and k's shapes) with torch and
    run attn_rope.  Returns (q_out, k_out); k may be None."""
    shape = _rope_inputs(q, k)
    _, Hq, Hkv, N, d = shape[:5]
    out_dtype = out_dtype or q.dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    with _made_on(stream, q.device):
        q_out, qos = _new_rows(q, out_dtype, Hq, N, d)
        k_out, kos = (None, None) if k is None else _new_rows(k, out_dtype, Hkv, N, d)
    if stream is not None:
        _used_here(q.device, q_out, k_out)
    return _rope_call(q, k, q_out, k_out, positions, inv_freq, shape, qos, kos, interleaved,
                      inverse, magnitude, stream)


def rope_backward(dq_out, dk_out, positions, inv_freq, *, interleaved: bool = False,
                  magnitude: float = 1.0, grad_dtype=None, stream=None):
    """The gradients of rope()'s q and k from those of its outputs (attn_bwd's
    dQ and dK): (dq, dk), dk None when dk_out is."""
    return rope(dq_out, dk_out, positions, inv_freq, interleaved=interleaved, magnitude=magnitude,
                out_dtype=grad_dtype, stream=stream, inverse=True)


def _check_pages(k_pages, v_pages, k_descale, v_descale):
    """Types, shapes and placement of a paged cache; returns (num_blocks,
    page_size, Hkv, d, cache dtype)."""
    _tensor(k_pages, (torch.bfloat16, torch.uint8), "k_pages")
    _need(k_pages, k_pages.dtype, "k_pages")
    _need(v_pages, k_pages.dtype, "v_pages")
    if k_pages.ndim != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must both be [num_blocks, page_size, Hkv, d]")
    num_blocks, page_size, Hkv, d = k_pages.shape
    if k_pages.dtype == torch.bfloat16:
        if k_descale is not None or v_descale is not None:
            raise ValueError("a bf16 cache has no descales")
        return num_blocks, page_size, Hkv, d, ATTN_CACHE_BF16
    for t, n in ((k_descale, "k_descale"), (v_descale, "v_descale")):
        _need(t, torch.float32, n)
        if t.shape != (num_blocks, Hkv, page_size):
            raise ValueError(f"{n} must be [num_blocks, Hkv, page_size]")
    return num_blocks, page_size, Hkv, d, ATTN_CACHE_E4M3


def attn_cache_write(k, v, k_pages, v_pages, slots, k_descale=None, v_descale=None, *, stream=None):
    """Write keys and values into a paged cache (in place).

    k, v bf16 [B,Hkv,N,d] or packed [total,Hkv,d], any strides with contiguous,
    16-byte-aligned rows; k_pages, v_pages [num_blocks,page_size,Hkv,d] bf16, or
    uint8 E4M3 codes with k_descale, v_descale fp32 [num_blocks,Hkv,page_size];
    slots int64 [B,N] (or [total]): page * page_size + key in the page, distinct,
    -1 for tokens to leave out.  Asynchronous."""
    _tensor(k, (torch.bfloat16,), "k")
    _tensor(v, (torch.bfloat16,), "v")
    num_blocks, page_size, Hkv, d, kind = _check_pages(k_pages, v_pages, k_descale, v_descale)
    (B, H, N, dk), ks = _rows(k, "k")
    if v.shape != k.shape or (H, dk) != (Hkv, d):
        raise ValueError("k / v / page shapes mismatch")
    _, vs = _rows(v, "v")
    _need(slots, torch.int64, "slots")
    if slots.shape != (k.shape[:1] if k.ndim == 3 else (B, N)):
        raise ValueError("slots must be [B, N] ([total] for packed keys)")
    with _on(_one_device(k, v, k_pages, v_pages, slots, k_descale, v_descale)):
        rc = load().attn_cache_write(_at(k), _at(v), ks, vs, _at(k_pages), _at(v_pages),
                                     _at(k_descale), _at(v_descale), _at(slots), B, N, Hkv, d,
                                     num_blocks, page_size, kind, _stream_ptr(stream))
    _check(rc, "attn_cache_write")


def _read_call(k_pages, v_pages, block_table, cu_seqlens, k_out, v_out, k_descale, v_descale,
               cache, stream):
    """attn_cache_read once the cache and the outputs are known to be good."""
    num_blocks, page_size, Hkv, d, kind = cache
    _need(block_table, torch.int32, "block_table")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    if block_table.ndim != 2 or cu_seqlens.shape != (block_table.shape[0] + 1,):
        raise ValueError("block_table must be [B, max_blocks] and cu_seqlens [B + 1]")
    B, max_blocks = block_table.shape
    odt = ATTN_OUT_F32 if k_out.dtype == torch.float32 else ATTN_OUT_BF16
    with _on(_one_device(k_pages, v_pages, block_table, cu_seqlens, k_out, v_out, k_descale, v_descale)):
        rc = load().attn_cache_read(k_pages.data_ptr(), v_pages.data_ptr(), _at(k_descale),
                                    _at(v_descale), block_table.data_ptr(), cu_seqlens.data_ptr(),
                                    k_out.data_ptr(), v_out.data_ptr(), B, Hkv, k_out.shape[0],
                                    num_blocks, page_size, max_blocks, d, kind, odt,
                                    _stream_ptr(stream))
    _check(rc, "attn_cache_read")
    return k_out, v_out


def attn_cache_read(k_pages, v_pages, block_table, cu_seqlens, k_out, v_out, k_descale=None,
                    v_descale=None, *, stream=None):
    """Read a paged cache back into packed k_out, v_out [total,Hkv,d] (bf16 or
    fp32), which attn_fwd_varlen takes: keys 0.. of sequence b to rows
    cu_seqlens[b]..cu_seqlens[b+1].  block_table int32 [B,max_blocks],
    cu_seqlens int32 [B+1], both on the device.  Rows outside every sequence
    stay as they were.  Asynchronous."""
    cache = _check_pages(k_pages, v_pages, k_descale, v_descale)
    _tensor(k_out, (torch.bfloat16, torch.float32), "k_out")
    _need(k_out, k_out.dtype, "k_out")
    _need(v_out, k_out.dtype, "v_out")
    if k_out.ndim != 3 or k_out.shape[1:] != cache[2:4] or v_out.shape != k_out.shape:
        raise ValueError("k_out and v_out must both be [total, Hkv, d]")
    return _read_call(k_pages, v_pages, block_table, cu_seqlens, k_out, v_out, k_descale, v_descale,
                      cache, stream)


def cache_read(k_pages, v_pages, block_table, cu_seqlens, total: int, k_descale=None,
               v_descale=None, *, out_dtype=None, stream=None):
    """Allocate k and v [total,Hkv,d] with torch and run attn_cache_read (total
    = cu_seqlens[-1], known to the host)."""
    cache = _check_pages(k_pages, v_pages, k_descale, v_descale)
    out_dtype = out_dtype or torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    shape = (total, cache[2], cache[3])
    with _made_on(stream, k_pages.device):
        k = torch.empty(shape, dtype=out_dtype, device=k_pages.device)
        v = torch.empty(shape, dtype=out_dtype, device=k_pages.device)
    if stream is not None:
        _used_here(k_pages.device, k, v)
    return _read_call(k_pages, v_pages, block_table, cu_seqlens, k, v, k_descale, v_descale, cache,
                      stream)


def tree_mask_words(mask):
    """bool [B,T,T] (mask[b, t, u]: drafted token t sees drafted token u) ->
    the int64 words [B,T,ceil(T/64)] that attn_decode_tree takes."""
    if mask.ndim != 3 or mask.shape[1] != mask.shape[2] or mask.dtype != torch.bool:
        raise ValueError("mask must be bool [B, T, T]")
    B, T, _ = mask.shape
    W = (T + 63) // 64
    bits = torch.zeros((B, T, W * 64), dtype=torch.int64, device=mask.device)
    bits[..., :T] = mask
    return (bits.view(B, T, W, 64) << torch.arange(64, device=mask.device)).sum(-1)


def attn_decode_tree_workspace_size(B: int, Hq: int, Hkv: int, T: int, max_blocks: int,
                                    page_size: int, d: int, e4m3: bool = False) -> int:
    return int(load().attn_decode_tree_workspace_size(B, Hq, Hkv, T, max_blocks, page_size, d,
                                                      int(bool(e4m3))))


@functools.lru_cache(maxsize=1024)
def _tree_workspace_known(Hq, Hkv, T, d, kind, device_index):
    n = int(load().attn_decode_tree_workspace_size(1, Hq, Hkv, T, 1, 16, d, kind))
    if n == 0:
        raise LookupError   # (not remembered)
    return n


def _tree_workspace(Hq, Hkv, T, d, kind, device_index):
    """attn_decode_tree_workspace_size on the current device (device_index), which
    depends on nothing else.  0, for what the library will refuse or when the device
    does not answer, is asked for again the next time."""
    try:
        return _tree_workspace_known(Hq, Hkv, T, d, kind, device_index)
    except LookupError:
        return 0


def _tree_call(q, k_pages, v_pages, block_table, seqlens, o, lse, tree_mask, q_lens, k_descale,
               v_descale, scale, workspace, stream):
    """attn_decode_tree once o and lse are known to be good."""
    _need(q, torch.bfloat16, "q")
    num_blocks, page_size, Hkv, d, kind = _check_pages(k_pages, v_pages, k_descale, v_descale)
    _need(block_table, torch.int32, "block_table")
    _need(seqlens, torch.int32, "seqlens")
    if q.ndim != 4 or q.shape[3] != d:
        raise ValueError("q / page shapes mismatch")
    B, Hq, T, _ = q.shape
    if block_table.ndim != 2 or block_table.shape[0] != B or seqlens.shape != (B,):
        raise ValueError("block_table must be [B, max_blocks] and seqlens [B]")
    if tree_mask is not None:
        _need(tree_mask, torch.int64, "tree_mask")
        if tree_mask.shape != (B, T, (T + 63) // 64):
            raise ValueError("tree_mask must be [B, T, ceil(T / 64)]")
    if q_lens is not None:
        _need(q_lens, torch.int32, "q_lens")
        if q_lens.shape != (B,):
            raise ValueError("q_lens must be [B]")
    if scale is None:
        scale = d ** -0.5
    max_blocks = block_table.shape[1]
    odt = ATTN_OUT_F32 if o.dtype == torch.float32 else ATTN_OUT_BF16
    dev = _one_device(q, k_pages, v_pages, block_table, seqlens, o, lse, tree_mask, q_lens,
                      k_descale, v_descale, workspace)
    lib = load()
    with _on(dev):
        if workspace is None:
            with _made_on(stream, dev):
                workspace = torch.empty(_tree_workspace(Hq, Hkv, T, d, kind, dev.index), dtype=torch.uint8,
                                        device=dev)
        elif not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        rc = lib.attn_decode_tree(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                  _at(k_descale), _at(v_descale), block_table.data_ptr(),
                                  seqlens.data_ptr(), _at(q_lens), _at(tree_mask), o.data_ptr(),
                                  _at(lse), B, Hq, Hkv, T, num_blocks, page_size, max_blocks, d,
                                  scale, kind, workspace.data_ptr(), workspace.nbytes, odt,
                                  _stream_ptr(stream))
    _check(rc, "attn_decode_tree")
    return o, lse


def attn_decode_tree(q, k_pages, v_pages, block_table, seqlens, o, lse=None, tree_mask=None,
                     q_lens=None, k_descale=None, v_descale=None, *, scale: float | None = None,
                     workspace=None, stream=None):
    """Attention of up to T drafted tokens per sequence over a paged cache that
    holds their keys and values already, into caller-provided outputs.

    q [B,Hq,T,d] bf16; the cache as for attn_cache_write; block_table int32
    [B,max_blocks]; seqlens int32 [B], drafted tokens included; o [B,Hq,T,d]
    bf16 or fp32; lse [B,Hq,T] fp32 or None; tree_mask int64 [B,T,ceil(T/64)]
    (tree_mask_words) or None for a chain; q_lens int32 [B] drafted tokens of
    each sequence, or None for T; workspace: a CUDA tensor of at least
    attn_decode_tree_workspace_size(...) bytes, or None (then one is allocated
    with torch).  T = 1 is plain decode.  Asynchronous."""
    _tensor(o, (torch.bfloat16, torch.float32), "o")
    _need(o, o.dtype, "o")
    if o.shape != q.shape:
        raise ValueError("o shape mismatch")
    if lse is not None:
        _need(lse, torch.float32, "lse")
        if lse.shape != q.shape[:3]:
            raise ValueError("lse shape mismatch")
    return _tree_call(q, k_pages, v_pages, block_table, seqlens, o, lse, tree_mask, q_lens, k_descale,
                      v_descale, scale, workspace, stream)


def decode_tree(q, k_pages, v_pages, block_table, seqlens, tree_mask=None, q_lens=None,
                k_descale=None, v_descale=None, *, scale: float | None = None, out_dtype=None,
                return_lse: bool = True, stream=None):
    """Allocate O (and LSE) with torch and run attn_decode_tree."""
    out_dtype = out_dtype or torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    with _made_on(stream, q.device):
        o = torch.empty(q.shape, dtype=out_dtype, device=q.device)
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device) if return_lse else None
    if stream is not None:
        _used_here(q.device, o, lse)
    return _tree_call(q, k_pages, v_pages, block_table, seqlens, o, lse, tree_mask, q_lens, k_descale,
                      v_descale, scale, None, stream)
