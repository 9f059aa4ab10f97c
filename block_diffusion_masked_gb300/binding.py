"""ctypes binding of libdfa.so: argument marshalling only.

Every function here has the name of the C entry point it calls (see
``include/dfa.h``) and does nothing but check tensor shapes, dtypes and
devices, allocate outputs with PyTorch, and pass raw pointers, sizes and the
current CUDA stream to the library.  Every step of the computation runs in
the library's CUDA kernels; there is no other implementation to fall back to,
so a missing or unloadable library raises.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdfa.so")

DFA_OK = 0
DFA_EINVAL = -1
DFA_EUNSUPPORTED = -2
DFA_ECUDA = -3
DFA_ETIMEOUT = -4
DFA_EDEVICE = -5
DFA_DETERMINISTIC = 1
DFA_NOISY_DIAG_PASS = 2
DFA_ROTARY_INTERLEAVED = 1
DFA_ROTARY_INVERSE = 2
DFA_ROTARY_CLEAR = 4
MODE_DIFFUSION = 0
MODE_CAUSAL = 1

_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_SIGNATURES = {
    "dfa_version": (_I, []),
    "dfa_error_string": (ctypes.c_char_p, [_I]),
    "dfa_last_cuda_error": (ctypes.c_char_p, []),
    "dfa_forward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "dfa_backward": (_I, [_P] * 9 + [_I, _I, _I, _I, _I, _P]),
    "dfa_forward_gqa": (_I, [_P] * 5 + [_I] * 6 + [_P]),
    "dfa_backward_gqa": (_I, [_P] * 9 + [_I] * 6 + [_P]),
    "dfa_forward_varlen": (_I, [_P] * 6 + [_I] * 5 + [_P]),
    "dfa_backward_varlen": (_I, [_P] * 10 + [_I] * 5 + [_P]),
    "dfa_backward_ex": (_I, [_P] * 10 + [_I] * 7 + [_P]),
    "dfa_forward_fp8": (_I, [_P] * 5 + [ctypes.c_float] * 3 + [_I] * 6 + [_P]),
    "dfa_fp8_vt_bytes": (ctypes.c_longlong, [_I] * 4),
    "dfa_fp8_transpose_v": (_I, [_P] * 2 + [_I] * 4 + [_P]),
    "dfa_forward_fp8_vt": (_I, [_P] * 5 + [ctypes.c_float] * 3 + [_I] * 6 + [_P]),
    "dfa_causal_forward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "dfa_causal_backward": (_I, [_P] * 9 + [_I, _I, _I, _I, _P]),
    "dfa_rotary": (_I, [_P] * 6 + [_I] * 8 + [_P] * 2 + [_I, _P]),
    "dfa_cache_plan": (_I, [_P] * 10 + [_I] * 5 + [_P]),
    "dfa_cache_release": (_I, [_P] * 5 + [_I] * 4 + [_P]),
    "dfa_cache_append": (_I, [_P] * 9 + [_I] * 8 + [_P] * 3),
    "dfa_cache_workspace_bytes": (ctypes.c_longlong, [_I] * 8),
    "dfa_cache_forward": (_I, [_P] * 13 + [ctypes.c_longlong] + [_I] * 10 + [_P] * 4),
    "dfa_cache_scale_exp": (_I, [ctypes.c_uint]),
    "dfa_cache_page_ok": (_I, [_I] * 2),
    "dfa_cache_append_pages": (_I, [_I] * 2),
    "dfa_cache_append_span": (_I, [_I] * 4 + [ctypes.POINTER(_I)]),
    "dfa_cache_units": (_I, [_I] * 4),
    "dfa_cache_blocks": (_I, [ctypes.c_longlong, _I]),
    "dfa_cache_run": (ctypes.c_longlong, [_I, ctypes.c_longlong, _I]),
    "dfa_cache_owner": (_I, [ctypes.c_longlong, ctypes.c_longlong, _I]),
    "dfa_cache_own_end": (_I, [_I] * 4),
    "dfa_status": (_I, [_P]),
    "dfa_selftest_wait_timeout": (_I, [_I, _P]),
    "dfa_fwd_main": (_I, [_P] * 6 + [_I] * 6 + [_P]),
    "dfa_bwd_preprocess": (_I, [_P] * 4 + [_I] * 4 + [_P]),
    "dfa_bwd_main": (_I, [_P] * 9 + [_I] * 6 + [_P]),
    "dfa_bwd_dq_convert": (_I, [_P] * 2 + [_I] * 4 + [_P]),
    "dfa_bwd_preprocess_ex": (_I, [_P] * 4 + [_I] * 5 + [_P]),
    "dfa_bwd_dq_convert_ex": (_I, [_P] * 2 + [_I] * 5 + [_P]),
    "dfa_fwd_main_gqa": (_I, [_P] * 6 + [_I] * 7 + [_P]),
    "dfa_bwd_main_gqa": (_I, [_P] * 9 + [_I] * 7 + [_P]),
    "dfa_bwd_main_ex": (_I, [_P] * 9 + [_I] * 8 + [_P]),
    "dfa_fwd_segments": (_I, [_I] * 7 + [ctypes.POINTER(_I)]),
    "dfa_bwd_segments": (_I, [_I] * 7 + [ctypes.POINTER(_I)]),
    "dfa_tile_full": (_I, [_I] * 7),
    "dfa_tile_visits": (ctypes.c_longlong, [_I] * 6),
    "dfa_tile_shape": (_I, [_I] + [ctypes.POINTER(_I)] * 4),
    "dfa_work_item": (_I, [_I] * 7 + [ctypes.POINTER(_I)]),
}


class DfaError(RuntimeError):
    def __init__(self, fn, code):
        msg = lib().dfa_error_string(code).decode()
        if code == DFA_ECUDA:
            msg += ": " + lib().dfa_last_cuda_error().decode()
        super().__init__(f"{fn} failed: {msg} ({code})")
        self.code = code


def lib():
    """Load libdfa.so (built in-tree by ``build()``) once and return it."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdfa.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(fn, rc):
    if rc != DFA_OK:
        raise DfaError(fn, rc)


def _stream_ptr(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _check_buf(t, shape, dtype, device, name):
    """A caller-supplied buffer must be exactly what the library will write."""
    if (not isinstance(t, torch.Tensor) or tuple(t.shape) != tuple(shape) or t.dtype != dtype
            or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {device}")
    return t


def _out_or_new(t, shape, dtype, device, name):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _check_buf(t, shape, dtype, device, name)


def _check_qkv(*ts):
    q = ts[0]
    if q.dim() != 4:
        raise ValueError("expected (batch, seqlen, heads, headdim) tensors")
    for t in ts:
        if t.shape != q.shape:
            raise ValueError("all tensors must have the shape of q")
        if t.dtype != torch.bfloat16:
            raise TypeError("tensors must be bfloat16")
        if not t.is_cuda or t.device != q.device:
            raise ValueError("tensors must live on the same CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def dfa_forward(q, k, v, block_size, out=None, lse=None):
    """Block-diffusion attention forward.  q, k, v: (B, 2n, H, d) bf16 CUDA.

    Returns (out, lse) with out (B, 2n, H, d) bf16 and lse (B, H, 2n) fp32.
    """
    _check_qkv(q, k, v)
    B, L, H, d = q.shape
    if L % 2:
        raise ValueError("the sequence must be [noisy | clean] with an even length 2n")
    out = _out_or_new(out, q.shape, torch.bfloat16, q.device, "out")
    lse = _out_or_new(lse, (B, H, L), torch.float32, q.device, "lse")
    with torch.cuda.device(q.device):
        rc = lib().dfa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, L // 2, H, d,
                               int(block_size), _stream_ptr(q))
    _check("dfa_forward", rc)
    return out, lse


def dfa_backward(q, k, v, out, dout, lse, block_size, dq=None, dk=None, dv=None):
    """Block-diffusion attention backward; returns (dq, dk, dv) bf16."""
    _check_qkv(q, k, v, out, dout)
    B, L, H, d = q.shape
    if L % 2:
        raise ValueError("the sequence must be [noisy | clean] with an even length 2n")
    _check_buf(lse, (B, H, L), torch.float32, q.device, "lse")
    dq = _out_or_new(dq, q.shape, torch.bfloat16, q.device, "dq")
    dk = _out_or_new(dk, k.shape, torch.bfloat16, q.device, "dk")
    dv = _out_or_new(dv, v.shape, torch.bfloat16, q.device, "dv")
    with torch.cuda.device(q.device):
        rc = lib().dfa_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
                                _ptr(dq), _ptr(dk), _ptr(dv), B, L // 2, H, d, int(block_size),
                                _stream_ptr(q))
    _check("dfa_backward", rc)
    return dq, dk, dv


def _check_grouped(q, k, v, *more):
    """q (and ``more``) share one shape, k and v another with fewer heads."""
    _check_qkv(q, *more)
    _check_qkv(k, v)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected (batch, seqlen, heads, headdim) tensors")
    if k.device != q.device:
        raise ValueError("tensors must live on the same CUDA device")
    B, L, H, d = q.shape
    Hk = k.shape[2]
    if k.shape[0] != B or k.shape[1] != L or k.shape[3] != d:
        raise ValueError("k and v must be (batch, seqlen, kv_heads, headdim) like q")
    if Hk < 1 or H % Hk:
        raise ValueError("kv_heads must divide the query heads")
    return Hk


def dfa_forward_gqa(q, k, v, block_size, out=None, lse=None):
    """Forward with grouped key/value heads: q (B, 2n, H, d), k, v (B, 2n, Hk, d).

    Query head h reads key/value head h // (H // Hk).  Returns (out, lse)
    like :func:`dfa_forward`.
    """
    Hk = _check_grouped(q, k, v)
    B, L, H, d = q.shape
    if L % 2:
        raise ValueError("the sequence must be [noisy | clean] with an even length 2n")
    out = _out_or_new(out, q.shape, torch.bfloat16, q.device, "out")
    lse = _out_or_new(lse, (B, H, L), torch.float32, q.device, "lse")
    with torch.cuda.device(q.device):
        rc = lib().dfa_forward_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, L // 2, H,
                                   Hk, d, int(block_size), _stream_ptr(q))
    _check("dfa_forward_gqa", rc)
    return out, lse


def dfa_backward_gqa(q, k, v, out, dout, lse, block_size, dq=None, dk=None, dv=None):
    """Backward with grouped key/value heads; dk, dv have the shape of k.

    The gradient of a key/value head sums over its query heads.
    """
    Hk = _check_grouped(q, k, v, out, dout)
    B, L, H, d = q.shape
    if L % 2:
        raise ValueError("the sequence must be [noisy | clean] with an even length 2n")
    _check_buf(lse, (B, H, L), torch.float32, q.device, "lse")
    dq = _out_or_new(dq, q.shape, torch.bfloat16, q.device, "dq")
    dk = _out_or_new(dk, k.shape, torch.bfloat16, q.device, "dk")
    dv = _out_or_new(dv, v.shape, torch.bfloat16, q.device, "dv")
    with torch.cuda.device(q.device):
        rc = lib().dfa_backward_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
                                    _ptr(dq), _ptr(dk), _ptr(dv), B, L // 2, H, Hk, d,
                                    int(block_size), _stream_ptr(q))
    _check("dfa_backward_gqa", rc)
    return dq, dk, dv


def _cu_array(cu_seqlens, rows):
    """Host int32 copy of cu_seqlens (list, NumPy array or tensor) as a ctypes array."""
    if isinstance(cu_seqlens, torch.Tensor):
        cu_seqlens = cu_seqlens.detach().cpu().tolist()
    cu = [int(x) for x in cu_seqlens]
    if len(cu) < 1 or cu[0] != 0 or cu[-1] != rows:
        raise ValueError("cu_seqlens must start at 0 and end at the packed rows")
    return (ctypes.c_int * len(cu))(*cu), len(cu) - 1


def _check_packed(q, k, v, *more):
    for t in (q, k, v) + more:
        if t.dim() != 3:
            raise ValueError("expected packed (rows, heads, headdim) tensors")
    _check_qkv(q[None], *(t[None] for t in more))
    _check_qkv(k[None], v[None])
    if k.device != q.device or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("k and v must be (rows, kv_heads, headdim) like q")
    if k.shape[1] < 1 or q.shape[1] % k.shape[1]:
        raise ValueError("kv_heads must divide the query heads")
    return k.shape[1]


def dfa_forward_varlen(q, k, v, cu_seqlens, block_size, out=None, lse=None):
    """Forward on a packed batch: q (rows, H, d), k, v (rows, Hk, d) bf16 CUDA.

    ``cu_seqlens`` (host: list, array or tensor) holds batch + 1 prefix sums;
    every sample length is even ([noisy | clean]).  Returns out (rows, H, d)
    and lse (H, rows) float32.
    """
    Hk = _check_packed(q, k, v)
    rows, H, d = q.shape
    cu, batch = _cu_array(cu_seqlens, rows)
    out = _out_or_new(out, q.shape, torch.bfloat16, q.device, "out")
    lse = _out_or_new(lse, (H, rows), torch.float32, q.device, "lse")
    with torch.cuda.device(q.device):
        rc = lib().dfa_forward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), cu, batch,
                                      H, Hk, d, int(block_size), _stream_ptr(q))
    _check("dfa_forward_varlen", rc)
    return out, lse


def dfa_backward_varlen(q, k, v, out, dout, lse, cu_seqlens, block_size, dq=None, dk=None,
                        dv=None):
    """Backward on a packed batch; returns (dq, dk, dv) bf16."""
    Hk = _check_packed(q, k, v, out, dout)
    rows, H, d = q.shape
    _check_buf(lse, (H, rows), torch.float32, q.device, "lse")
    cu, batch = _cu_array(cu_seqlens, rows)
    dq = _out_or_new(dq, q.shape, torch.bfloat16, q.device, "dq")
    dk = _out_or_new(dk, k.shape, torch.bfloat16, q.device, "dk")
    dv = _out_or_new(dv, v.shape, torch.bfloat16, q.device, "dv")
    with torch.cuda.device(q.device):
        rc = lib().dfa_backward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout),
                                       _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), cu, batch, H, Hk,
                                       d, int(block_size), _stream_ptr(q))
    _check("dfa_backward_varlen", rc)
    return dq, dk, dv


def dfa_forward_fp8(q, k, v, q_descale, k_descale, v_descale, block_size, out=None, lse=None):
    """FP8 forward: q (B, 2n, H, 128), k, v (B, 2n, Hk, 128) float8_e4m3fn CUDA tensors.

    The attention of q * q_descale, k * k_descale, v * v_descale; returns
    out (B, 2n, H, 128) bf16 and lse (B, H, 2n) float32.
    """
    for t in (q, k, v):
        if t.dtype != torch.float8_e4m3fn or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous float8_e4m3fn CUDA tensors")
    if q.dim() != 4 or k.shape != v.shape or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3]:
        raise ValueError("q (B, 2n, H, d), k and v (B, 2n, Hk, d)")
    B, L, H, d = q.shape
    Hk = k.shape[2]
    if L % 2 or H % Hk:
        raise ValueError("even 2n and kv_heads dividing heads required")
    if k.device != q.device or v.device != q.device:
        raise ValueError("q, k, v must live on the same CUDA device")
    out = _out_or_new(out, q.shape, torch.bfloat16, q.device, "out")
    lse = _out_or_new(lse, (B, H, L), torch.float32, q.device, "lse")
    with torch.cuda.device(q.device):
        rc = lib().dfa_forward_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                   float(q_descale), float(k_descale), float(v_descale), B, L // 2,
                                   H, Hk, d, int(block_size), _stream_ptr(q))
    _check("dfa_forward_fp8", rc)
    return out, lse


def dfa_fp8_transpose_v(v, vt=None):
    """V^T of an e4m3 v (B, 2n, Hk, 128) for dfa_forward_fp8_vt (a uint8 tensor).

    A caller-supplied ``vt`` must be a contiguous uint8 tensor on v's device
    with exactly dfa_fp8_vt_bytes(B, n, Hk, 128) elements.
    """
    if (v.dtype != torch.float8_e4m3fn or v.dim() != 4 or not v.is_contiguous()
            or not v.is_cuda):
        raise ValueError("v must be a contiguous float8_e4m3fn (B, 2n, Hk, 128) CUDA tensor")
    B, L, Hk, d = v.shape
    if L % 2:
        raise ValueError("the sequence must be [noisy | clean] with an even length 2n")
    nbytes = lib().dfa_fp8_vt_bytes(B, L // 2, Hk, d)
    if nbytes < 0:
        raise DfaError("dfa_fp8_vt_bytes", int(nbytes))
    vt = _out_or_new(vt, (int(nbytes),), torch.uint8, v.device, "vt")
    with torch.cuda.device(v.device):
        rc = lib().dfa_fp8_transpose_v(_ptr(v), _ptr(vt), B, L // 2, Hk, d, _stream_ptr(v))
    _check("dfa_fp8_transpose_v", rc)
    return vt


def dfa_forward_fp8_vt(q, k, vt, kv_heads, q_descale, k_descale, v_descale, block_size,
                       out=None, lse=None):
    """dfa_forward_fp8 on a V^T from dfa_fp8_transpose_v (no scratch).

    ``kv_heads`` must equal k.shape[2]; ``vt`` must be the uint8 tensor
    dfa_fp8_transpose_v wrote for a v of k's shape.
    """
    for t in (q, k):
        if t.dtype != torch.float8_e4m3fn or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k must be contiguous float8_e4m3fn CUDA tensors")
    if q.dim() != 4 or k.dim() != 4 or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3]:
        raise ValueError("q (B, 2n, H, d), k (B, 2n, Hk, d)")
    if k.device != q.device:
        raise ValueError("q and k must live on the same CUDA device")
    B, L, H, d = q.shape
    if L % 2:
        raise ValueError("the sequence must be [noisy | clean] with an even length 2n")
    Hk = k.shape[2]
    if int(kv_heads) != Hk:
        raise ValueError(f"kv_heads ({kv_heads}) must equal k.shape[2] ({Hk})")
    if H % Hk:
        raise ValueError("kv_heads must divide the query heads")
    nbytes = lib().dfa_fp8_vt_bytes(B, L // 2, Hk, d)
    if nbytes < 0:
        raise DfaError("dfa_fp8_vt_bytes", int(nbytes))
    _check_buf(vt, (int(nbytes),), torch.uint8, q.device, "vt")
    out = _out_or_new(out, q.shape, torch.bfloat16, q.device, "out")
    lse = _out_or_new(lse, (B, H, L), torch.float32, q.device, "lse")
    with torch.cuda.device(q.device):
        rc = lib().dfa_forward_fp8_vt(_ptr(q), _ptr(k), _ptr(vt), _ptr(out), _ptr(lse),
                                      float(q_descale), float(k_descale), float(v_descale), B,
                                      L // 2, H, Hk, d, int(block_size), _stream_ptr(q))
    _check("dfa_forward_fp8_vt", rc)
    return out, lse


def dfa_backward_ex(q, k, v, out, dout, lse, block_size, cu_seqlens=None, deterministic=False,
                    dq=None, dk=None, dv=None, noisy_diag_pass=False):
    """Backward with options: batched (q 4-D) or packed (q 3-D, ``cu_seqlens``).

    ``deterministic``: dQ contributions are added in a fixed order, so the
    results are bitwise reproducible.  ``noisy_diag_pass``: the noisy key
    tiles in a launch of their own before the clean ones, where the block
    size allows it (DFA_NOISY_DIAG_PASS).
    """
    if cu_seqlens is None:
        Hk = _check_grouped(q, k, v, out, dout)
        B, L, H, d = q.shape
        if lse.shape != (B, H, L):
            raise ValueError("lse must be (B, H, 2n)")
        cu, batch, n = None, B, L // 2
    else:
        Hk = _check_packed(q, k, v, out, dout)
        rows, H, d = q.shape
        if lse.shape != (H, rows):
            raise ValueError("lse must be (heads, rows)")
        cu, batch = _cu_array(cu_seqlens, rows)
        n = 0
    if lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    flags = (DFA_DETERMINISTIC if deterministic else 0) | \
        (DFA_NOISY_DIAG_PASS if noisy_diag_pass else 0)
    with torch.cuda.device(q.device):
        rc = lib().dfa_backward_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
                                   _ptr(dq), _ptr(dk), _ptr(dv), cu, batch, n, H, Hk, d,
                                   int(block_size), flags, _stream_ptr(q))
    _check("dfa_backward_ex", rc)
    return dq, dk, dv


def dfa_causal_forward(q, k, v, out=None, lse=None):
    """Causal attention on (Bc, L, H, d), any Bc: the yardstick."""
    _check_qkv(q, k, v)
    B, L, H, d = q.shape
    out = _out_or_new(out, q.shape, torch.bfloat16, q.device, "out")
    lse = _out_or_new(lse, (B, H, L), torch.float32, q.device, "lse")
    with torch.cuda.device(q.device):
        rc = lib().dfa_causal_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, L, H, d,
                                      _stream_ptr(q))
    _check("dfa_causal_forward", rc)
    return out, lse


def dfa_causal_backward(q, k, v, out, dout, lse, dq=None, dk=None, dv=None):
    _check_qkv(q, k, v, out, dout)
    B, L, H, d = q.shape
    _check_buf(lse, (B, H, L), torch.float32, q.device, "lse")
    dq = _out_or_new(dq, q.shape, torch.bfloat16, q.device, "dq")
    dk = _out_or_new(dk, k.shape, torch.bfloat16, q.device, "dk")
    dv = _out_or_new(dv, v.shape, torch.bfloat16, q.device, "dv")
    with torch.cuda.device(q.device):
        rc = lib().dfa_causal_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout),
                                       _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), B, L, H, d,
                                       _stream_ptr(q))
    _check("dfa_causal_backward", rc)
    return dq, dk, dv


def _ptr_or_null(t):
    return ctypes.c_void_p(None) if t is None else _ptr(t)


def _step_shape(q, mode):
    """(batch, n, rows per batch entry) of a step-API tensor for `mode`.

    Diffusion: q is (B, 2n, H, d); causal: q is (Bc, n, H, d), Bc sequences.
    """
    B, L, H, d = q.shape
    if mode == MODE_CAUSAL:
        return B, L, L
    if mode != MODE_DIFFUSION:
        raise ValueError("mode must be MODE_DIFFUSION or MODE_CAUSAL")
    if L % 2:
        raise ValueError("the sequence must be [noisy | clean] with an even length 2n")
    return B, L // 2, L


def _check_scratch(q, lse, delta, dq_acc):
    B, L, H, d = q.shape
    if lse is not None:
        _check_buf(lse, (B, H, L), torch.float32, q.device, "lse")
    if delta is not None:
        _check_buf(delta, (B, H, L), torch.float32, q.device, "delta")
    if dq_acc is not None:
        _check_buf(dq_acc, q.shape, torch.float32, q.device, "dq_acc")


def dfa_fwd_main(q, k, v, out, lse, dq_acc, block_size, mode=MODE_DIFFUSION):
    """The forward step; also zeroes dq_acc (float32, shape of q) unless None.

    Diffusion: q, k, v, out (B, 2n, H, d) bf16, lse (B, H, 2n) fp32.  Causal:
    q, k, v, out (Bc, n, H, d), lse (Bc, H, n), as dfa_causal_forward.
    """
    _check_qkv(q, k, v, out)
    B, n, L = _step_shape(q, mode)
    H, d = q.shape[2], q.shape[3]
    _check_scratch(q, lse, None, dq_acc)
    with torch.cuda.device(q.device):
        rc = lib().dfa_fwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                _ptr_or_null(dq_acc), B, n, H, d, int(block_size), int(mode),
                                _stream_ptr(q))
    _check("dfa_fwd_main", rc)


def dfa_bwd_preprocess(out, dout, delta, dq_acc, mode=MODE_DIFFUSION):
    """Step 1 of the backward: delta = rowsum(dout * out); dq_acc = 0 unless None."""
    _check_qkv(out, dout)
    B, n, L = _step_shape(out, mode)
    H, d = out.shape[2], out.shape[3]
    _check_scratch(out, None, delta, dq_acc)
    with torch.cuda.device(out.device):
        rc = lib().dfa_bwd_preprocess_ex(_ptr(out), _ptr(dout), _ptr(delta),
                                         _ptr_or_null(dq_acc), B, n, H, d, int(mode),
                                         _stream_ptr(out))
    _check("dfa_bwd_preprocess_ex", rc)


def dfa_bwd_main(q, k, v, dout, lse, delta, dq_acc, dk, dv, block_size, mode=MODE_DIFFUSION):
    """Step 2 of the backward: the tensor-core kernel (dk, dv, dq_acc += dq)."""
    _check_qkv(q, k, v, dout, dk, dv)
    B, n, L = _step_shape(q, mode)
    H, d = q.shape[2], q.shape[3]
    _check_scratch(q, lse, delta, dq_acc)
    with torch.cuda.device(q.device):
        rc = lib().dfa_bwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lse), _ptr(delta),
                                _ptr(dq_acc), _ptr(dk), _ptr(dv), B, n, H, d,
                                int(block_size), int(mode), _stream_ptr(q))
    _check("dfa_bwd_main", rc)


def dfa_fwd_main_gqa(q, k, v, out, lse, dq_acc, block_size, mode=MODE_DIFFUSION):
    """dfa_fwd_main with k, v of fewer heads (grouped key/value heads)."""
    Hk = _check_grouped(q, k, v, out)
    B, n, L = _step_shape(q, mode)
    H, d = q.shape[2], q.shape[3]
    _check_scratch(q, lse, None, dq_acc)
    with torch.cuda.device(q.device):
        rc = lib().dfa_fwd_main_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                    _ptr_or_null(dq_acc), B, n, H, Hk, d, int(block_size),
                                    int(mode), _stream_ptr(q))
    _check("dfa_fwd_main_gqa", rc)


def dfa_bwd_main_gqa(q, k, v, dout, lse, delta, dq_acc, dk, dv, block_size, mode=MODE_DIFFUSION):
    """dfa_bwd_main with k, v, dk, dv of fewer heads (grouped key/value heads)."""
    Hk = _check_grouped(q, k, v, dout)
    B, n, L = _step_shape(q, mode)
    H, d = q.shape[2], q.shape[3]
    _check_scratch(q, lse, delta, dq_acc)
    _check_buf(dk, k.shape, torch.bfloat16, q.device, "dk")
    _check_buf(dv, v.shape, torch.bfloat16, q.device, "dv")
    with torch.cuda.device(q.device):
        rc = lib().dfa_bwd_main_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lse),
                                    _ptr(delta), _ptr(dq_acc), _ptr(dk), _ptr(dv), B, n, H,
                                    Hk, d, int(block_size), int(mode), _stream_ptr(q))
    _check("dfa_bwd_main_gqa", rc)


def dfa_bwd_main_ex(q, k, v, dout, lse, delta, dq_acc, dk, dv, block_size, mode=MODE_DIFFUSION,
                    noisy_diag_pass=False):
    """dfa_bwd_main_gqa with flags (``noisy_diag_pass``: DFA_NOISY_DIAG_PASS)."""
    Hk = _check_grouped(q, k, v, dout)
    B, n, L = _step_shape(q, mode)
    H, d = q.shape[2], q.shape[3]
    _check_scratch(q, lse, delta, dq_acc)
    _check_buf(dk, k.shape, torch.bfloat16, q.device, "dk")
    _check_buf(dv, v.shape, torch.bfloat16, q.device, "dv")
    flags = DFA_NOISY_DIAG_PASS if noisy_diag_pass else 0
    with torch.cuda.device(q.device):
        rc = lib().dfa_bwd_main_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lse),
                                   _ptr(delta), _ptr(dq_acc), _ptr(dk), _ptr(dv), B, n, H,
                                   Hk, d, int(block_size), int(mode), flags, _stream_ptr(q))
    _check("dfa_bwd_main_ex", rc)


def dfa_bwd_dq_convert(dq_acc, dq, mode=MODE_DIFFUSION):
    """Step 3 of the backward: dq = bf16(dq_acc)."""
    _check_qkv(dq)
    B, n, L = _step_shape(dq, mode)
    H, d = dq.shape[2], dq.shape[3]
    _check_scratch(dq, None, None, dq_acc)
    with torch.cuda.device(dq.device):
        rc = lib().dfa_bwd_dq_convert_ex(_ptr(dq_acc), _ptr(dq), B, n, H, d, int(mode),
                                         _stream_ptr(dq))
    _check("dfa_bwd_dq_convert_ex", rc)


# ------------------------------------------- rotary positions, sampling cache
# A sampling step is many small calls, so these keep to few Python operations:
# the checks read attributes only, and the device is made current only where
# it is not.

_INT_MAX = (1 << 31) - 1


def _int32(x):
    """An integer argument in 32 bits, which ctypes would wrap it to: one past them
    is the largest, and any negative one, which no entry point takes, -1."""
    return max(min(int(x), _INT_MAX), -1)


_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(fn, device, *args):
    """Call entry point ``fn`` with ``device`` current, on its current stream."""
    handle = _lib or lib()
    index = device.index
    if index == _get_device():
        stream = _raw_stream(index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
        rc = getattr(handle, fn)(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = getattr(handle, fn)(*args, torch.cuda.current_stream(device).cuda_stream)
    if rc != DFA_OK:
        raise DfaError(fn, rc)


def _check_dense(t, shape, dtype, device, name):
    """A contiguous input of the given shape on a CUDA device."""
    try:
        if (t.dtype is dtype and t.get_device() == device.index and t.shape == shape
                and t.is_contiguous()):
            return
    except AttributeError:  # not a tensor
        pass
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                     f"on {device}")


def _check_dims(t, dim, name):
    if not isinstance(t, torch.Tensor) or t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-dimensional tensor")
    return t.shape


def _check_heads(t, dim, name, device=None):
    """A bf16 input of ``dim`` dimensions on a CUDA device; returns its shape."""
    try:
        shape = t.shape
        if (t.dtype is torch.bfloat16 and len(shape) == dim
                and (t.is_cuda if device is None else t.get_device() == device.index)):
            return shape
    except AttributeError:  # not a tensor
        pass
    where = "a CUDA device" if device is None else str(device)
    raise ValueError(f"{name} must be a {dim}-dimensional bfloat16 tensor on {where}")


@functools.lru_cache(maxsize=1024)
def _stride_array(lead, *strides):
    """Host array of ``lead`` zeros and the leading strides; None for strides the
    kernels do not take."""
    if strides[-1] != 1 or any(x & 7 for x in strides[:-1]):
        return None
    return (ctypes.c_longlong * (lead + len(strides) - 1))(*[0] * lead, *strides[:-1])


def _strides(t, name, lead=0):
    """Host array of a tensor's leading strides (behind ``lead`` zeros), None where
    it is contiguous.

    The last dimension must be contiguous and the others multiples of 8
    elements (16 bytes), as must be the address of the first element.
    """
    if t.is_contiguous():
        return None
    array = _stride_array(lead, *t.stride())
    if array is None:
        raise ValueError(f"{name}: the last dimension must be contiguous and the other strides "
                         "multiples of 8 elements")
    return array


def dfa_rotary(q, k, table, positions=None, period=None, interleaved=False, inverse=False,
               q_out=None, k_out=None, clear=False):
    """Rotary positions of q (B, L, H, d) and k (B, L, Hk, d), bf16; k may be None.

    ``table``: float32 (max_pos, rot_dim), cosines then sines.  ``positions``:
    int32 (B, L), or None: row r has position r mod ``period`` (default L // 2,
    the [noisy | clean] layout).  Packed rows: q (rows, H, d), k (rows, Hk, d),
    positions (rows,).  q and k may be strided views (the last dimension
    contiguous).  Returns contiguous (q_out, k_out); rows of negative positions
    are not written, or set to zero with ``clear``.  ``inverse`` is the
    transposed map.
    """
    sizes = _rotary_sizes(q, k, table, positions, period)
    if q_out is not None:
        _check_dense(q_out, q.shape, torch.bfloat16, q.device, "q_out")
    if k is not None and k_out is not None:
        _check_dense(k_out, k.shape, torch.bfloat16, q.device, "k_out")
    flags = ((DFA_ROTARY_INTERLEAVED if interleaved else 0)
             | (DFA_ROTARY_INVERSE if inverse else 0) | (DFA_ROTARY_CLEAR if clear else 0))
    return _rotary_launch(q, k, table, positions, sizes, flags, q_out, k_out)


def _rotary_sizes(q, k, table, positions, period):
    """Check dfa_rotary's inputs; returns its integer arguments."""
    packed = isinstance(q, torch.Tensor) and q.dim() == 3
    shape = _check_heads(q, 3 if packed else 4, "q")
    dev = q.device
    if packed:
        L, H, d = shape
        B = 1
    else:
        B, L, H, d = shape
    Hk = 0
    if k is not None:
        kshape = _check_heads(k, 3 if packed else 4, "k", dev)
        Hk = kshape[-2]
        if kshape[0] != shape[0] or kshape[-3] != L or kshape[-1] != d:
            raise ValueError("k must be (batch, seqlen, kv_heads, headdim) like q")
    max_pos, rot = _check_dims(table, 2, "table")
    _check_dense(table, (max_pos, rot), torch.float32, dev, "table")
    if positions is not None:
        _check_dense(positions, (L,) if packed else (B, L), torch.int32, dev, "positions")
        period = 1
    elif packed:
        raise ValueError("packed rows need positions")
    elif period is None:
        if L % 2:
            raise ValueError("the sequence must be [noisy | clean] with an even length 2n")
        period = max(L // 2, 1)
    return B, L, _int32(period), H, Hk, d, rot, max_pos


def _rotary_launch(q, k, table, positions, sizes, flags, q_out=None, k_out=None):
    """dfa_rotary of tensors that _rotary_sizes (or a call like it) has checked."""
    shape, dev = q.shape, q.device
    lead = 1 if len(shape) == 3 else 0  # packed rows: a batch of one
    q_str, k_str, kp, kop = _strides(q, "q", lead), None, None, None
    if q_out is None:
        q_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
        k_str, kp, kop = _strides(k, "k", lead), k.data_ptr(), k_out.data_ptr()
    _call("dfa_rotary", dev, q.data_ptr(), kp, q_out.data_ptr(), kop, table.data_ptr(),
          None if positions is None else positions.data_ptr(), *sizes, q_str, k_str, flags)
    return q_out, k_out


def _check_pages(cache_lens, per_request, block_table, free_pages, free_count, name):
    """The int32 state of a page table; returns (device, batch, max_pages, free entries)."""
    i32 = torch.int32
    (B,) = _check_dims(cache_lens, 1, "cache_lens")
    dev = cache_lens.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a CUDA device")
    _check_dense(cache_lens, (B,), i32, dev, "cache_lens")
    _check_dense(per_request, (B,), i32, dev, name)
    maxp = _check_dims(block_table, 2, "block_table")[1]
    _check_dense(block_table, (B, maxp), i32, dev, "block_table")
    (F,) = _check_dims(free_pages, 1, "free_pages")
    _check_dense(free_pages, (F,), i32, dev, "free_pages")
    _check_dense(free_count, (1,), i32, dev, "free_count")
    return dev, B, maxp, F


def dfa_cache_plan(cache_lens, new_lens, block_table, free_pages, free_count, page_size, rows):
    """The pages of a sampling step (see dfa.h).  int32 CUDA tensors: cache_lens,
    new_lens (B,), block_table (B, max_pages), free_pages (F,), free_count (1,).

    Writes the new pages into ``block_table`` and returns (block_table, cu_new
    (B + 1,), positions (rows,), next_lens (B,), next_free (1,), missing (1,)).
    The caller's next step passes next_lens and next_free.
    """
    dev, B, maxp, F = _check_pages(cache_lens, new_lens, block_table, free_pages, free_count,
                                   "new_lens")
    rows = int(rows)
    if not 0 <= rows <= 1 << 30:
        raise ValueError("rows must be 0 to 2^30")
    buf = torch.empty(2 * B + 3 + rows, dtype=torch.int32, device=dev)
    # integers, of which autograd keeps no versions: views without its bookkeeping
    cu_new, next_lens, next_free, missing, positions = torch.unsafe_split_with_sizes(
        buf, (B + 1, B, 1, 1, rows))
    at = buf.data_ptr()
    _call("dfa_cache_plan", dev, cache_lens.data_ptr(), new_lens.data_ptr(),
          block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), at,
          at + 4 * (2 * B + 3), at + 4 * (B + 1), at + 4 * (2 * B + 1), at + 4 * (2 * B + 2), B,
          maxp, F, _int32(page_size), rows)
    return block_table, cu_new, positions, next_lens, next_free, missing


def dfa_cache_release(finished, cache_lens, block_table, free_pages, free_count, page_size):
    """Requests with finished != 0 give their pages back (in place; see dfa.h)."""
    dev, B, maxp, F = _check_pages(cache_lens, finished, block_table, free_pages, free_count,
                                   "finished")
    _call("dfa_cache_release", dev, finished.data_ptr(), cache_lens.data_ptr(),
          block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), B, maxp, F,
          _int32(page_size))


def _check_cache(k_cache, v_cache, k_scale, v_scale, block_table, cache_lens, cu_new, dev, d):
    """Shapes of a cache and its tables; returns (batch, kv_heads, page_size, pages, max_pages)."""
    shape = _check_dims(k_cache, 4, "k_cache")
    P, Hk, ps, dc = shape
    if dc != d:
        raise ValueError("the cache must have the head dimension of the rows")
    _check_dense(k_cache, shape, torch.float8_e4m3fn, dev, "k_cache")
    _check_dense(v_cache, shape, torch.float8_e4m3fn, dev, "v_cache")
    _check_dense(k_scale, (P, Hk), torch.float32, dev, "k_scale")
    _check_dense(v_scale, (P, Hk), torch.float32, dev, "v_scale")
    B, maxp = _check_dims(block_table, 2, "block_table")
    _check_dense(block_table, (B, maxp), torch.int32, dev, "block_table")
    _check_dense(cache_lens, (B,), torch.int32, dev, "cache_lens")
    _check_dense(cu_new, (B + 1,), torch.int32, dev, "cu_new")
    return B, Hk, ps, P, maxp


def dfa_cache_append(k, v, cu_new, cache_lens, block_table, k_cache, v_cache, k_scale, v_scale,
                     max_new):
    """Append packed tokens k, v (rows, Hk, d) bf16 to the cache, in place (see dfa.h).

    ``max_new``: a bound on the rows of one request, known to the host.
    """
    rows, Hk, d = shape = _check_heads(k, 3, "k")
    dev = k.device
    vshape = _check_heads(v, 3, "v", dev)
    B, Hc, ps, P, maxp = _check_cache(k_cache, v_cache, k_scale, v_scale, block_table, cache_lens,
                                      cu_new, dev, d)
    if vshape != shape or Hc != Hk:
        raise ValueError("k and v must be (rows, kv_heads, headdim) with the cache's heads")
    _call("dfa_cache_append", dev, k.data_ptr(), v.data_ptr(), cu_new.data_ptr(),
          cache_lens.data_ptr(), block_table.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          k_scale.data_ptr(), v_scale.data_ptr(), B, rows, _int32(max_new), Hk,
          d, ps, P, maxp, _strides(k, "k"), _strides(v, "v"))


def dfa_cache_workspace_bytes(batch, rows, max_new, heads, kv_heads, headdim, page_size,
                              max_pages):
    """Bytes of workspace dfa_cache_forward needs on the current device (0: none)."""
    n = lib().dfa_cache_workspace_bytes(*map(_int32, (batch, rows, max_new, heads, kv_heads, headdim,
                                                      page_size, max_pages)))
    if n < 0:
        raise DfaError("dfa_cache_workspace_bytes", int(n))
    return int(n)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(device_index, *sizes):
    """dfa_cache_workspace_bytes on a device, which sizes alone determine."""
    with torch.cuda.device(device_index):
        return dfa_cache_workspace_bytes(*sizes)


def dfa_cache_forward(q, k_cache, v_cache, k_scale, v_scale, block_table, cache_lens, cu_new,
                      max_new, k=None, v=None, block_size=1, out=None, lse=None, workspace=None):
    """Attention of packed new rows q (rows, H, d) over the cache and, with k and v
    (rows, Hk, d) bf16, over their own blocks (see dfa.h).

    ``max_new``: a bound on the rows of one request.  Returns out (rows, H, d)
    bf16 and lse (H, rows) float32.  ``workspace``: a uint8 tensor of at least
    dfa_cache_workspace_bytes(...) bytes; by default one is allocated.  For
    sampling: no gradients, the outputs are detached from q, k and v.
    """
    rows, H, d = shape = _check_heads(q, 3, "q")
    dev = q.device
    B, Hk, ps, P, maxp = _check_cache(k_cache, v_cache, k_scale, v_scale, block_table, cache_lens,
                                      cu_new, dev, d)
    if Hk < 1 or H % Hk:
        raise ValueError("kv_heads must divide the query heads")
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    kp = vp = ks = vs = None
    if k is not None:
        own = (rows, Hk, d)
        if _check_heads(k, 3, "k", dev) != own or _check_heads(v, 3, "v", dev) != own:
            raise ValueError("k and v must be (rows, kv_heads, headdim)")
        kp, vp, ks, vs = k.data_ptr(), v.data_ptr(), _strides(k, "k"), _strides(v, "v")
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        _check_dense(out, shape, torch.bfloat16, dev, "out")
    if lse is None:
        lse = torch.empty((H, rows), dtype=torch.float32, device=dev)
    else:
        _check_dense(lse, (H, rows), torch.float32, dev, "lse")
    max_new = _int32(max_new)
    if workspace is None:
        nwork = _workspace_bytes(dev.index, B, rows, max_new, H, Hk, d, ps, maxp)
        if nwork:
            workspace = torch.empty(nwork, dtype=torch.uint8, device=dev)
    else:
        nwork = workspace.numel()
        _check_dense(workspace, (nwork,), torch.uint8, dev, "workspace")
    _call("dfa_cache_forward", dev, q.data_ptr(), kp, vp, k_cache.data_ptr(), v_cache.data_ptr(),
          k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), cache_lens.data_ptr(),
          cu_new.data_ptr(), out.data_ptr(), lse.data_ptr(),
          None if workspace is None else workspace.data_ptr(), nwork, B, rows, max_new, H, Hk, d,
          _int32(block_size), ps, P, maxp, _strides(q, "q"), ks, vs)
    return out, lse


def dfa_selftest_wait_timeout(limit_us=20000):
    """Run the bounded-wait self-test on the current stream (see dfa.h)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        rc = lib().dfa_selftest_wait_timeout(int(limit_us),
                                             ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream))
    _check("dfa_selftest_wait_timeout", rc)


def dfa_status(device=None):
    """Synchronise the current stream and return (and clear) the device status code."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        return lib().dfa_status(ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream))


# ------------------------------------------------------------- geometry

def dfa_fwd_segments(mode, n, block_size, block_m, block_n, q_half, q_tile):
    buf = (_I * 8)()
    cnt = lib().dfa_fwd_segments(mode, n, block_size, block_m, block_n, q_half, q_tile, buf)
    _check("dfa_fwd_segments", 0 if cnt >= 0 else cnt)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(cnt)]


def dfa_bwd_segments(mode, n, block_size, block_m, block_n, k_half, k_tile):
    buf = (_I * 8)()
    cnt = lib().dfa_bwd_segments(mode, n, block_size, block_m, block_n, k_half, k_tile, buf)
    _check("dfa_bwd_segments", 0 if cnt >= 0 else cnt)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(cnt)]


def dfa_tile_full(rule, n, block_size, q_start, block_m, k_start, block_n):
    return lib().dfa_tile_full(rule, n, block_size, q_start, block_m, k_start, block_n)


def dfa_tile_visits(mode, n, block_size, block_m, block_n, pass_):
    return lib().dfa_tile_visits(mode, n, block_size, block_m, block_n, pass_)


def dfa_work_item(pass_, mode, w, batch, heads, tiles, group):
    """(batch, head, half, tile) of the w-th work item of a pass (0 forward, 1 backward)."""
    buf = (_I * 4)()
    _check("dfa_work_item", lib().dfa_work_item(pass_, mode, w, batch, heads, tiles, group, buf))
    return tuple(buf)


def dfa_tile_shape(headdim):
    vals = [_I() for _ in range(4)]
    _check("dfa_tile_shape", lib().dfa_tile_shape(headdim, *[ctypes.byref(x) for x in vals]))
    return tuple(x.value for x in vals)
