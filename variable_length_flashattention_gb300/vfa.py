"""Python binding of libvfa (include/vfa.h): argument marshalling only.

Every function takes torch tensors that already live on the current CUDA
device, passes their data pointers and the current torch stream to the C ABI,
and raises ``VfaError`` on a non-OK status.  All computation happens in the
library's kernels; there is no fallback of any kind: if ``libvfa.so`` has not
been built (``python -m variable_length_flashattention_gb300.build``) the
first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading
from fractions import Fraction
from typing import Optional, Tuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libvfa.so")
_lock = threading.Lock()
_lib = None

STATUS_NAMES = {
    0: "VFA_OK",
    1: "VFA_ERR_INVALID_ARG",
    2: "VFA_ERR_UNSUPPORTED",
    3: "VFA_ERR_ARCH",
    4: "VFA_ERR_CUDA",
    5: "VFA_ERR_BAD_SEQLENS",
    6: "VFA_ERR_BAD_BLOCK",
    7: "VFA_ERR_TIMEOUT",
    8: "VFA_ERR_WORKSPACE",
    9: "VFA_ERR_NO_PAGES",
}
VFA_OK, VFA_ERR_INVALID_ARG, VFA_ERR_UNSUPPORTED, VFA_ERR_ARCH, VFA_ERR_CUDA = 0, 1, 2, 3, 4
VFA_ERR_BAD_SEQLENS, VFA_ERR_BAD_BLOCK, VFA_ERR_TIMEOUT, VFA_ERR_WORKSPACE = 5, 6, 7, 8
VFA_ERR_NO_PAGES = 9

# Every symbol include/vfa.h declares: (name, restype, argtypes).
_P, _I, _F, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_L = ctypes.c_int64
SIGNATURES = [
    ("vfa_last_error", ctypes.c_char_p, []),
    ("vfa_version", ctypes.c_char_p, []),
    ("vfa_varlen_fwd_workspace_bytes", _S, [_I, _I, _I, _I, _I]),
    ("vfa_varlen_fwd_tile_shape", _I, [_I, _P, _P, _P]),
    ("vfa_varlen_fwd", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _P, _P,
                            _S, _P]),
    ("vfa_varlen_fwd_sinks", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I,
                                  _P, _P, _P, _S, _P]),
    ("vfa_varlen_fwd_fp8", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _F, _F, _I,
                                _I, _P, _P, _P, _S, _P]),
    ("vfa_varlen_fwd_noalloc", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P,
                                    _P, _P, _P]),
    ("vfa_varlen_schedule", _I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _I, _P, _P, _P,
                                 _S, _P]),
    ("vfa_varlen_bwd_workspace_bytes", _S, [_I, _I, _I, _I]),
    ("vfa_varlen_bwd", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I,
                            _P, _P, _P, _P, _S, _P]),
    ("vfa_varlen_bwd_sinks_workspace_bytes", _S, [_I, _I, _I, _I, _I]),
    ("vfa_varlen_bwd_sinks", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I,
                                  _I, _I, _P, _P, _P, _P, _S, _P]),
    ("vfa_paged_decode_init", _I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    ("vfa_paged_decode_step", _I, [_P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P,
                                   _P, _P, _P, _P]),
    ("vfa_paged_decode_step_split", _I, [_P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F,
                                         _P, _P, _P, _P, _I, _P, _S, _P]),
    ("vfa_paged_decode_split_workspace_bytes", _S, [_I, _I, _I, _I, _I]),
    ("vfa_paged_decode_split_count", _I, [_I, _I, _I, _P]),
    ("vfa_paged_decode_finalize", _I, [_P, _P, _I, _I, _I, _P, _P]),
    ("vfa_debug_paged_gather", _I, [_P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    ("vfa_debug_bounded_wait", _I, [_P, _P]),
    ("vfa_qk_norm_rope_fwd", _I, [_P, _P, _L, _L, _P, _I, _P, _I, _I, _P, _P, _F, _I, _I, _I, _I,
                                  _P, _P, _L, _L, _P]),
    ("vfa_qk_norm_rope_bwd_workspace_bytes", _S, [_I]),
    ("vfa_qk_norm_rope_bwd", _I, [_P, _P, _L, _L, _P, _P, _L, _L, _P, _I, _P, _I, _I, _P, _P, _F,
                                  _I, _I, _I, _I, _P, _P, _L, _L, _P, _P, _P, _S, _P]),
    ("vfa_kv4_block_bytes", _S, [_I, _I]),
    ("vfa_kv4_write", _I, [_P, _P, _L, _L, _I, _P, _I, _P, _I, _P, _P, _I, _I, _I, _F, _F, _P,
                           _P]),
    ("vfa_kv4_gather", _I, [_P, _P, _L, _L, _I, _P, _I, _P, _I, _P, _P, _I, _I, _I, _F, _F, _P,
                            _P]),
    ("vfa_kv4_decode_workspace_bytes", _S, [_I, _I, _I, _I]),
    ("vfa_kv4_decode", _I, [_P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _F, _F, _F, _P, _P, _P, _P,
                            _S, _P]),
    ("vfa_pages_workspace_bytes", _S, [_I, _I, _I]),
    ("vfa_pages_extend", _I, [_P, _I, _P, _I, _P, _I, _P, _I, _P, _S, _P, _P]),
    ("vfa_pages_fork", _I, [_P, _I, _P, _I, _P, _I, _P, _P, _I, _P, _P, _I, _I, _P, _S, _P, _P]),
    ("vfa_pages_free", _I, [_P, _I, _P, _I, _P, _I, _P, _I, _I, _P, _P]),
    ("vfa_pages_compact", _I, [_P, _I, _P, _I, _P, _I, _P, _P, _I, _I, _P, _P, _P, _P, _S, _P,
                               _P]),
    ("vfa_pages_copy", _I, [_P, _P, _I, _P, _P, _I, _I, _P, _P]),
    ("vfa_pages_truncate", _I, [_P, _I, _P, _I, _P, _I, _P, _I, _P, _P, _P, _S, _P, _P]),
    ("vfa_paged_decode_workspace_bytes", _S, [_I, _I, _I, _I, _I]),
    ("vfa_paged_decode", _I, [_P, _P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P,
                              _P, _P, _P, _S, _P]),
    ("vfa_varlen_key_weights_workspace_bytes", _S, [_I, _I, _I, _I, _I]),
    ("vfa_varlen_key_weights", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I,
                                    _P, _P, _L, _P, _S, _P]),
    ("vfa_cache_evict_workspace_bytes", _S, [_I, _I, _I]),
    ("vfa_cache_evict", _I, [_P, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _P, _P, _P, _I, _I, _P, _P,
                             _P, _P, _P, _S, _P, _P]),
    ("vfa_read_status", _I, [_P, _P, _P]),
]


class VfaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"libvfa.so is not built ({_LIB_PATH}); run "
                "`python -m variable_length_flashattention_gb300.build` first")
        L = ctypes.CDLL(_LIB_PATH)
        for name, res, args in SIGNATURES:
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
        return L


def _check(st: int):
    if st != VFA_OK:
        raise VfaError(st, lib().vfa_last_error().decode(errors="replace"))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _plain(t: torch.Tensor, dtype, dev: int) -> bool:
    """What _dense asks for, in one expression (it says what is wrong)."""
    return t.get_device() == dev and t.dtype is dtype and t.is_contiguous()


def _packed_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k):
    """(total_q, H, D, total_k, Hkv, batch) of packed q and k, v, checked against each other."""
    qshape, kshape = q.shape, k.shape
    if (len(qshape) != 3 or kshape != v.shape or len(kshape) != 3 or qshape[2] != kshape[2] or
            kshape[1] == 0 or qshape[1] % kshape[1] != 0):
        raise ValueError("q, k, v must be [tokens, heads, head_dim]; k/v heads must divide q heads")
    batch = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != batch + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    _fits(*qshape, kshape[0], batch)
    return (*qshape, kshape[0], kshape[1], batch)


def _shaped(t: torch.Tensor, dtype, shape, name: str, dev: int):
    """A caller's tensor that is read or written whole."""
    if not _plain(t, dtype, dev):
        _dense(t, dtype, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _scratch(t: torch.Tensor, dev: int):
    """A caller's workspace: its bytes are counted, of any type."""
    if t.get_device() != dev or not t.is_contiguous():
        _dense(t, t.dtype, "workspace", dev)


def _int32(n, name) -> int:
    """n as the C ABI takes it; ctypes would cut a larger one without a word."""
    n = int(n)
    if not -0x80000000 <= n <= 0x7fffffff:
        raise ValueError(f"{name} {n} does not fit 32 bits")
    return n


def version() -> str:
    return lib().vfa_version().decode()


# ----------------------------------------------------------------- varlen forward

def tile_shape(head_dim: int) -> Tuple[int, int, bool]:
    """(q tile rows, key tile rows, two q tiles per work item) for head_dim."""
    bq, bk, pr = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib().vfa_varlen_fwd_tile_shape(head_dim, ctypes.byref(bq), ctypes.byref(bk),
                                           ctypes.byref(pr)))
    return bq.value, bk.value, bool(pr.value)


def workspace_bytes(batch: int, total_q: int, total_k: int, num_heads: int, head_dim: int) -> int:
    n = lib().vfa_varlen_fwd_workspace_bytes(batch, total_q, total_k, num_heads, head_dim)
    if n == 0:
        raise VfaError(VFA_ERR_INVALID_ARG, "no workspace size for these arguments")
    return int(n)


def alloc_workspace(batch: int, total_q: int, total_k: int, num_heads: int, head_dim: int,
                    device=None) -> torch.Tensor:
    n = workspace_bytes(batch, total_q, total_k, num_heads, head_dim)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def varlen_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
               cu_seqlens_k: torch.Tensor, max_seqlen_q: int, softmax_scale: float,
               causal, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None, window_left: int = -1, sink_tokens: int = 0):
    """out bf16 [Tq, H, D], lse f32 [Tq, H] = varlen attention forward (vfa_varlen_fwd).

    k, v may hold fewer heads than q (a divisor of H): query head h reads kv
    head h // (H // Hkv).  causal: 0 / False, 1 / True (top-left), 2
    (bottom-right); window_left >= 0 adds a sliding window (needs causal), past
    which the first sink_tokens keys stay visible (vfa_varlen_fwd_sinks)."""
    bf16, i32 = torch.bfloat16, torch.int32
    dev = _device(q, "q")
    if not (_plain(q, bf16, dev) and _plain(k, bf16, dev) and _plain(v, bf16, dev) and
            _plain(cu_seqlens_q, i32, dev) and _plain(cu_seqlens_k, i32, dev)):
        for t, d, n in ((q, bf16, "q"), (k, bf16, "k"), (v, bf16, "v"),
                        (cu_seqlens_q, i32, "cu_seqlens_q"), (cu_seqlens_k, i32, "cu_seqlens_k")):
            _dense(t, d, n, dev)
    total_q, H, D, total_k, Hkv, batch = _packed_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k)
    if out is None:
        out = torch.empty_like(q)
    else:
        _shaped(out, bf16, q.shape, "out", dev)
    if lse is None:
        lse = torch.empty((total_q, H), dtype=torch.float32, device=q.device)
    else:
        _shaped(lse, torch.float32, (total_q, H), "lse", dev)
    if workspace is None:
        with _of(stream):
            workspace = alloc_workspace(batch, total_q, total_k, H, D, device=q.device)
    else:
        _scratch(workspace, dev)
    ins = (q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
           total_q, total_k, _int32(max_seqlen_q, "max_seqlen_q"), batch, H, Hkv, D, float(softmax_scale),
           _int32(causal, "causal"), _int32(window_left, "window_left"))
    outs = (out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes,
            _raw_stream(stream, dev))
    if sink_tokens != 0:
        sinks = _int32(sink_tokens, "sink_tokens")
        st = (_lib or lib()).vfa_varlen_fwd_sinks(*ins, sinks, *outs)
    else:
        st = (_lib or lib()).vfa_varlen_fwd(*ins, *outs)
    if st:
        _check(st)
    return out, lse


def varlen_fwd_fp8(q8: torch.Tensor, k8: torch.Tensor, v: torch.Tensor,
                   cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, max_seqlen_q: int,
                   softmax_scale: float, descale_q: float, descale_k: float, causal,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None,
                   window_left: int = -1):
    """vfa_varlen_fwd_fp8: q8, k8 uint8 E4M3 codes [T, H(kv), 128], v bf16; returns (out, lse)."""
    dev = _device(q8, "q8")
    for t, d, n in ((q8, _U8, "q8"), (k8, _U8, "k8"), (v, _BF16, "v"), (cu_seqlens_q, _I32, "cu_seqlens_q"),
                    (cu_seqlens_k, _I32, "cu_seqlens_k")):
        _dense(t, d, n, dev)
    total_q, H, D, total_k, Hkv, batch = _packed_shapes(q8, k8, v, cu_seqlens_q, cu_seqlens_k)
    if out is None:
        out = torch.empty(q8.shape, dtype=torch.bfloat16, device=q8.device)
    else:
        _shaped(out, _BF16, q8.shape, "out", dev)
    if lse is None:
        lse = torch.empty((total_q, H), dtype=torch.float32, device=q8.device)
    else:
        _shaped(lse, _F32, (total_q, H), "lse", dev)
    if workspace is None:
        with _of(stream):
            workspace = alloc_workspace(batch, total_q, total_k, H, D, device=q8.device)
    else:
        _scratch(workspace, dev)
    st = lib().vfa_varlen_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v), _ptr(cu_seqlens_q),
                                  _ptr(cu_seqlens_k), total_q, total_k,
                                  _int32(max_seqlen_q, "max_seqlen_q"), batch, H, Hkv, D,
                                  float(softmax_scale), float(descale_q), float(descale_k),
                                  _int32(causal, "causal"), _int32(window_left, "window_left"),
                                  _ptr(out), _ptr(lse), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st)
    return out, lse


def alloc_bwd_workspace(batch: int, total_q: int, num_heads: int, head_dim: int,
                        device="cuda", sink_tokens: int = 0) -> torch.Tensor:
    if sink_tokens != 0:
        n = lib().vfa_varlen_bwd_sinks_workspace_bytes(batch, total_q, num_heads, head_dim,
                                                       _int32(sink_tokens, "sink_tokens"))
    else:
        n = lib().vfa_varlen_bwd_workspace_bytes(batch, total_q, num_heads, head_dim)
    if n == 0:
        raise VfaError(VFA_ERR_UNSUPPORTED, "backward workspace size query rejected its arguments")
    return torch.empty(n, dtype=torch.uint8, device=device)


def varlen_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
               dout: torch.Tensor, lse: torch.Tensor, cu_seqlens_q: torch.Tensor,
               cu_seqlens_k: torch.Tensor, softmax_scale: float, causal,
               window_left: int = -1, dq: Optional[torch.Tensor] = None,
               dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None, sink_tokens: int = 0):
    """(dq, dk, dv) bf16 = gradients of varlen_fwd for upstream gradient dout (vfa_varlen_bwd;
    with sink_tokens vfa_varlen_bwd_sinks, and a workspace made for as many)."""
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    dev = _device(q, "q")
    if not (_plain(q, bf16, dev) and _plain(k, bf16, dev) and _plain(v, bf16, dev) and
            _plain(out, bf16, dev) and _plain(dout, bf16, dev) and _plain(lse, f32, dev) and
            _plain(cu_seqlens_q, i32, dev) and _plain(cu_seqlens_k, i32, dev)):
        for t, d, n in ((q, bf16, "q"), (k, bf16, "k"), (v, bf16, "v"), (out, bf16, "out"),
                        (dout, bf16, "dout"), (lse, f32, "lse"), (cu_seqlens_q, i32, "cu_seqlens_q"),
                        (cu_seqlens_k, i32, "cu_seqlens_k")):
            _dense(t, d, n, dev)
    total_q, H, D, total_k, Hkv, batch = _packed_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k)
    if out.shape != q.shape or dout.shape != q.shape or lse.shape != (total_q, H):
        raise ValueError("out and dout must have q's shape [Tq, H, D] and lse [Tq, H]")
    if dq is None:
        dq = torch.empty_like(q)
    else:
        _shaped(dq, bf16, q.shape, "dq", dev)
    if dk is None:
        dk = torch.empty_like(k)
    else:
        _shaped(dk, bf16, k.shape, "dk", dev)
    if dv is None:
        dv = torch.empty_like(v)
    else:
        _shaped(dv, bf16, v.shape, "dv", dev)
    if workspace is None:
        with _of(stream):
            workspace = alloc_bwd_workspace(batch, total_q, H, D, device=q.device,
                                            sink_tokens=max(sink_tokens, 0))
    else:
        _scratch(workspace, dev)
    ins = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), dout.data_ptr(), lse.data_ptr(),
           cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), total_q, total_k, batch, H, Hkv, D,
           float(softmax_scale), _int32(causal, "causal"), _int32(window_left, "window_left"))
    outs = (dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), workspace.nbytes,
            _raw_stream(stream, dev))
    if sink_tokens != 0:
        sinks = _int32(sink_tokens, "sink_tokens")
        st = (_lib or lib()).vfa_varlen_bwd_sinks(*ins, sinks, *outs)
    else:
        st = (_lib or lib()).vfa_varlen_bwd(*ins, *outs)
    if st:
        _check(st)
    return dq, dk, dv, workspace


def varlen_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, max_seqlen_q: int,
                       softmax_scale: float, causal: bool, out: torch.Tensor, lse: torch.Tensor,
                       device_status: Optional[torch.Tensor] = None, stream=None,
                       window_left: int = -1):
    """vfa_varlen_fwd_noalloc: the forward with the library's static scratch.

    For callers that cannot allocate device memory: the caller passes only
    inputs and outputs (allocated however it likes); the library allocates
    nothing.  Calls that can overlap on the GPU must not use it concurrently.
    """
    dev = _device(q, "q")
    for t, d, n in ((q, _BF16, "q"), (k, _BF16, "k"), (v, _BF16, "v"), (cu_seqlens_q, _I32, "cu_seqlens_q"),
                    (cu_seqlens_k, _I32, "cu_seqlens_k")):
        _dense(t, d, n, dev)
    total_q, H, D, total_k, Hkv, batch = _packed_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k)
    _shaped(out, _BF16, q.shape, "out", dev)
    _shaped(lse, _F32, (total_q, H), "lse", dev)
    if device_status is not None:
        _dense(device_status, _I32, "device_status", dev)
    st = lib().vfa_varlen_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_q),
                                      _ptr(cu_seqlens_k), total_q, total_k,
                                      _int32(max_seqlen_q, "max_seqlen_q"), batch, H, Hkv, D,
                                      float(softmax_scale), _int32(causal, "causal"),
                                      _int32(window_left, "window_left"), _ptr(out), _ptr(lse),
                                      _ptr(device_status),
                                      _stream(stream))
    _check(st)
    return out, lse


def schedule(cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, total_q: int, total_k: int,
             max_seqlen_q: int, num_heads: int, block_q: int, block_k: int, causal: bool,
             pair: bool = False, stream=None, window_left: int = -1):
    """Runs the device tile scheduler alone; returns (items int32 [n, 8] on device, status)."""
    batch = cu_seqlens_q.numel() - 1
    cap = num_heads * (total_q // block_q + batch)
    dev = cu_seqlens_q.device
    items = torch.full((max(cap, 1), 8), -7, dtype=torch.int32, device=dev)
    n_items = torch.zeros(1, dtype=torch.int32, device=dev)
    status = torch.full((1,), -1, dtype=torch.int32, device=dev)
    # scratch of vfa_varlen_fwd_workspace_bytes() bytes covers any tile shape
    nbytes = workspace_bytes(batch, total_q, total_k, num_heads, 128)
    scratch = torch.empty((nbytes + 3) // 4, dtype=torch.int32, device=dev)
    st = lib().vfa_varlen_schedule(_ptr(cu_seqlens_q), _ptr(cu_seqlens_k), total_q, total_k,
                                   _int32(max_seqlen_q, "max_seqlen_q"), batch, num_heads, block_q,
                                   block_k, _int32(causal, "causal"),
                                   _int32(window_left, "window_left"), int(bool(pair)), _ptr(items),
                                   cap,
                                   _ptr(n_items), _ptr(status), _ptr(scratch), scratch.numel() * 4,
                                   _stream(stream))
    _check(st)
    n = int(n_items.item())
    return items[:n], int(status.item())


def read_status(word: torch.Tensor, stream=None) -> int:
    """The int32 at word.data_ptr() (workspace status word or decode status)."""
    out = ctypes.c_int32()
    _check(lib().vfa_read_status(_ptr(word), _stream(stream), ctypes.byref(out)))
    return int(out.value)


# ----------------------------------------------------------------- paged decode

def decode_init(m: torch.Tensor, l: torch.Tensor, o: torch.Tensor,
                status: Optional[torch.Tensor] = None, stream=None):
    S, Hq, D = o.shape
    for t, n in ((m, "m"), (l, "l"), (o, "o")):
        _need(t, torch.float32, n)
    _check(lib().vfa_paged_decode_init(_ptr(m), _ptr(l), _ptr(o), S, Hq, D, _ptr(status),
                                       _stream(stream)))


def decode_step(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                tile_blocks: torch.Tensor, tile_block_counts: torch.Tensor,
                m: torch.Tensor, l: torch.Tensor, o: torch.Tensor,
                status: Optional[torch.Tensor] = None, stream=None,
                tile_token_counts: Optional[torch.Tensor] = None, softmax_scale: float = 0.0):
    """vfa_paged_decode_step; tile_token_counts (int32 [S], optional) and
    softmax_scale (<= 0: 1/sqrt(D)) as in include/vfa.h."""
    _need(q, torch.bfloat16, "q")
    if tile_token_counts is not None:
        _need(tile_token_counts, torch.int32, "tile_token_counts")
    _need(k_pool, torch.bfloat16, "k_pool")
    _need(v_pool, torch.bfloat16, "v_pool")
    _need(tile_blocks, torch.int32, "tile_blocks")
    _need(tile_block_counts, torch.int32, "tile_block_counts")
    S, Hq, D = q.shape
    nb, bs, Hkv, D2 = k_pool.shape
    if D2 != D or v_pool.shape != k_pool.shape or tile_blocks.shape[0] != S:
        raise ValueError("inconsistent decode shapes")
    _check(lib().vfa_paged_decode_step(_ptr(q), _ptr(k_pool), _ptr(v_pool), nb, _ptr(tile_blocks),
                                       _ptr(tile_block_counts), _ptr(tile_token_counts),
                                       tile_blocks.shape[1], S, Hq, Hkv, D, bs,
                                       float(softmax_scale), _ptr(m), _ptr(l), _ptr(o),
                                       _ptr(status), _stream(stream)))


def decode_split_count(num_seqs: int, num_kv_heads: int, tile_capacity: int) -> int:
    """vfa_paged_decode_split_count: a run count for the current device."""
    n = ctypes.c_int()
    _check(lib().vfa_paged_decode_split_count(num_seqs, num_kv_heads, tile_capacity,
                                              ctypes.byref(n)))
    return n.value


def alloc_decode_split_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                 head_dim: int, num_splits: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for vfa_paged_decode_step_split (the tickets start at zero)."""
    n = lib().vfa_paged_decode_split_workspace_bytes(num_seqs, num_q_heads, num_kv_heads,
                                                     head_dim, num_splits)
    if n == 0:
        raise VfaError(VFA_ERR_UNSUPPORTED, "no split workspace for these sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode_step_split(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                      tile_blocks: torch.Tensor, tile_block_counts: torch.Tensor,
                      m: torch.Tensor, l: torch.Tensor, o: torch.Tensor, num_splits: int,
                      workspace: torch.Tensor, status: Optional[torch.Tensor] = None,
                      stream=None, tile_token_counts: Optional[torch.Tensor] = None,
                      softmax_scale: float = 0.0):
    """vfa_paged_decode_step_split: the step with each tile cut into num_splits runs."""
    _need(q, torch.bfloat16, "q")
    if tile_token_counts is not None:
        _need(tile_token_counts, torch.int32, "tile_token_counts")
    _need(k_pool, torch.bfloat16, "k_pool")
    _need(v_pool, torch.bfloat16, "v_pool")
    _need(tile_blocks, torch.int32, "tile_blocks")
    _need(tile_block_counts, torch.int32, "tile_block_counts")
    _need(workspace, torch.uint8, "workspace")
    S, Hq, D = q.shape
    nb, bs, Hkv, D2 = k_pool.shape
    if D2 != D or v_pool.shape != k_pool.shape or tile_blocks.shape[0] != S:
        raise ValueError("inconsistent decode shapes")
    _check(lib().vfa_paged_decode_step_split(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), nb, _ptr(tile_blocks), _ptr(tile_block_counts),
        _ptr(tile_token_counts), tile_blocks.shape[1], S, Hq, Hkv, D, bs, float(softmax_scale),
        _ptr(m), _ptr(l), _ptr(o), _ptr(status), int(num_splits), _ptr(workspace),
        workspace.numel(), _stream(stream)))


def decode_finalize(l: torch.Tensor, o: torch.Tensor, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    S, Hq, D = o.shape
    if out is None:
        out = torch.empty((S, Hq, D), dtype=torch.bfloat16, device=o.device)
    _check(lib().vfa_paged_decode_finalize(_ptr(l), _ptr(o), S, Hq, D, _ptr(out),
                                           _stream(stream)))
    return out


# ----------------------------------------------------------------- norm and rotation

# 1 / (2 pi) to 60 digits: the table's steps are rounded once, from this.
_INV_2PI = Fraction("0.159154943091895335768883763372514362034459645740456448747667")


# The operators below are called once per layer of a step, often on little
# data, where the host's time is the call's time: a check is one expression per
# tensor, and the message is worked out only where it fails.

_BF16, _F32, _I32, _I64, _U8 = (torch.bfloat16, torch.float32, torch.int32, torch.int64,
                                torch.uint8)


def _refuse(t, dtype, name, dev):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev or dev != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current device (cuda:{torch.cuda.current_device()}), "
                         f"like the other tensors; got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _fits(*sizes):
    """The C ABI takes sizes as int32, and ctypes would cut a larger one without a word."""
    for n in sizes:
        if n > 0x7fffffff:
            raise ValueError(f"size {n} does not fit 32 bits")


def _device(t: torch.Tensor, name: str) -> int:
    """The current device, which must be t's: kernels are launched there."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _refuse(t, t.dtype, name, dev)
    return dev


def _dense(t: torch.Tensor, dtype, name: str, dev: int):
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous():
        _refuse(t, dtype, name, dev)


def _rows(t: torch.Tensor, shape, name: str, dev: int) -> int:
    """t: bf16 [tokens, heads, head_dim], heads and dims contiguous; returns the token stride
    in elements (one or no token has no neighbour: the packed distance)."""
    if t.dtype is not _BF16 or t.get_device() != dev:
        _refuse(t, _BF16, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] = {tuple(shape)}, got "
                         f"{tuple(t.shape)}")
    T, H, D = shape
    st, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{name} must have contiguous heads and dims")
    return st if T > 1 else H * D


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _of(stream):
    """Allocations belong to the stream the call's kernels run on: the block of a workspace that is
    dropped on return is handed out again to work behind them, not beside them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An allocation that belongs to the stream the call's kernels run on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_rows(like, stream) -> torch.Tensor:
    """A packed tensor shaped like `like`, whose token stride is its largest."""
    if stream is None:
        return torch.empty_like(like)
    with torch.cuda.stream(stream):
        return torch.empty_like(like)


def _address(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def rope_table(inv_freq, axes=None, device="cuda") -> torch.Tensor:
    """The table of vfa_qk_norm_rope_fwd: int64 [len(inv_freq), 2].

    inv_freq: radians per position of each rotated pair (rotary_dim / 2 finite
    numbers); axes: the position axis each pair follows (default: all 0)."""
    inv_freq = [float(f) for f in inv_freq]
    axes = [0] * len(inv_freq) if axes is None else [int(a) for a in axes]
    if len(axes) != len(inv_freq):
        raise ValueError("axes must give one axis per frequency")
    if any(a < 0 for a in axes):
        raise ValueError("axes must be >= 0")
    rows = []
    for f, a in zip(inv_freq, axes):
        if not math.isfinite(f):
            raise ValueError("inv_freq must be finite")
        step = round(Fraction(f) * _INV_2PI * 2 ** 64) % 2 ** 64
        rows.append((step - 2 ** 64 if step >= 2 ** 63 else step, a))
    return torch.tensor(rows, dtype=torch.int64, device=device).reshape(len(rows), 2)


def _rope_inputs(q, k, positions, table, q_weight, k_weight):
    """Checks; (device, q's and k's token strides, position axes, rotated dims)."""
    dev = q.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _refuse(q, _BF16, "q", dev)
    qshape, kshape = q.shape, k.shape
    if len(qshape) != 3 or len(kshape) != 3 or qshape[0] != kshape[0] or qshape[2] != kshape[2]:
        raise ValueError("q [T, Hq, D] and k [T, Hkv, D] must agree in tokens and head_dim")
    qs, ks = _rows(q, qshape, "q", dev), _rows(k, kshape, "k", dev)
    T, _, D = qshape
    axes = rot = 0
    if table is not None:
        tshape = table.shape
        if table.get_device() != dev or table.dtype is not _I64 or not table.is_contiguous():
            _refuse(table, _I64, "table", dev)
        if len(tshape) != 2 or tshape[1] != 2:
            raise ValueError("table must be [rotary_dim / 2, 2], as rope_table makes it")
        rot = 2 * tshape[0]
        if positions is None:
            raise ValueError("a rotation needs positions")
        if positions.get_device() != dev or positions.dtype is not _I32 or \
                not positions.is_contiguous():
            _refuse(positions, _I32, "positions", dev)
        pshape = positions.shape
        axes = 1 if len(pshape) == 1 else pshape[0]
        if not 1 <= len(pshape) <= 2 or pshape[-1] != T or axes > 0x7fffffff:
            raise ValueError("positions must be [tokens] or [axes, tokens]")
    if q_weight is not None:
        _rope_weight(q_weight, "q_weight", D, dev)
    if k_weight is not None:
        _rope_weight(k_weight, "k_weight", D, dev)
    return dev, qs, ks, axes, rot


def _rope_weight(w, name, D, dev):
    if w.get_device() != dev or w.dtype is not _F32 or not w.is_contiguous():
        _refuse(w, _F32, name, dev)
    if w.shape != (D,):
        raise ValueError(f"{name} must be [head_dim]")


def _row_output(given, like, name, dev, stream):
    """(the output, its token stride): the given one checked, or a new one shaped like `like`."""
    if given is None:
        shape = like.shape
        return _empty_rows(like, stream), shape[1] * shape[2]
    return given, _rows(given, like.shape, name, dev)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor],
                 table: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, stream=None):
    """(q_out, k_out) bf16 = per-head RMS norm and position rotation (vfa_qk_norm_rope_fwd).

    q [T, Hq, D], k [T, Hkv, D] bf16, views with a token stride included;
    positions int32 [T] or [axes, T]; table from rope_table (None: no rotation);
    weights f32 [D] (None: no norm); q_out / k_out may be q / k."""
    dev, qs, ks, axes, rot = _rope_inputs(q, k, positions, table, q_weight, k_weight)
    q_out, qos = _row_output(q_out, q, "q_out", dev, stream)
    k_out, kos = _row_output(k_out, k, "k_out", dev, stream)
    T, Hq, D = q.shape
    st = (_lib or lib()).vfa_qk_norm_rope_fwd(
        q.data_ptr(), k.data_ptr(), qs, ks, _address(positions), axes, _address(table), rot,
        1 if interleaved else 0, _address(q_weight), _address(k_weight), eps, T, Hq, k.shape[1], D,
        q_out.data_ptr(), k_out.data_ptr(), qos, kos, _raw_stream(stream, dev))
    if st:
        _check(st)
    return q_out, k_out


def alloc_qk_norm_rope_bwd_workspace(head_dim: int, device="cuda") -> torch.Tensor:
    n = (_lib or lib()).vfa_qk_norm_rope_bwd_workspace_bytes(head_dim)
    if n == 0:
        raise VfaError(VFA_ERR_UNSUPPORTED, f"no workspace size for head_dim {head_dim}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, dq_out: torch.Tensor, dk_out: torch.Tensor,
                     positions: Optional[torch.Tensor], table: Optional[torch.Tensor],
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     interleaved: bool = False, dq: Optional[torch.Tensor] = None,
                     dk: Optional[torch.Tensor] = None, dq_weight: Optional[torch.Tensor] = None,
                     dk_weight: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """(dq, dk, dq_weight, dk_weight) = gradients of qk_norm_rope (vfa_qk_norm_rope_bwd).

    dq_out, dk_out: upstream gradients; dq / dk may be dq_out / dk_out.  The
    weight gradients are f32 [D], None where there is no weight."""
    dev, qs, ks, axes, rot = _rope_inputs(q, k, positions, table, q_weight, k_weight)
    dqos, dkos = _rows(dq_out, q.shape, "dq_out", dev), _rows(dk_out, k.shape, "dk_out", dev)
    dq, dqs = _row_output(dq, q, "dq", dev, stream)
    dk, dks = _row_output(dk, k, "dk", dev, stream)
    grads = [None, None]
    for i, (w, g, n) in enumerate(((q_weight, dq_weight, "dq_weight"),
                                   (k_weight, dk_weight, "dk_weight"))):
        if w is None:
            continue
        if g is None:
            g = _empty(w.shape, torch.float32, w.device, stream)
        else:
            _dense(g, _F32, n, dev)
            if g.shape != w.shape:
                raise ValueError(f"{n} must be [head_dim]")
        grads[i] = g
    if workspace is not None:
        _dense(workspace, workspace.dtype, "workspace", dev)
    elif q_weight is not None or k_weight is not None:
        n = (_lib or lib()).vfa_qk_norm_rope_bwd_workspace_bytes(q.shape[2])
        workspace = _empty(n, torch.uint8, q.device, stream)
    T, Hq, D = q.shape
    st = (_lib or lib()).vfa_qk_norm_rope_bwd(
        q.data_ptr(), k.data_ptr(), qs, ks, dq_out.data_ptr(), dk_out.data_ptr(), dqos, dkos,
        _address(positions), axes, _address(table), rot, 1 if interleaved else 0,
        _address(q_weight), _address(k_weight), eps, T, Hq, k.shape[1], D, dq.data_ptr(),
        dk.data_ptr(), dqs, dks, _address(grads[0]), _address(grads[1]), _address(workspace),
        _nbytes(workspace), _raw_stream(stream, dev))
    if st:
        _check(st)
    return dq, dk, grads[0], grads[1]


# ----------------------------------------------------------------- 4-bit cache

def kv4_block_bytes(num_kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of 16 tokens (vfa_kv4_block_bytes)."""
    n = (_lib or lib()).vfa_kv4_block_bytes(num_kv_heads, head_dim)
    if n == 0:
        raise VfaError(VFA_ERR_UNSUPPORTED, "no 4-bit page size for these arguments")
    return int(n)


def alloc_kv4_pool(num_blocks: int, num_kv_heads: int, head_dim: int,
                   device="cuda") -> torch.Tensor:
    """A zero-filled 4-bit pool, uint8 [num_blocks, num_kv_heads, 18 * head_dim]."""
    kv4_block_bytes(num_kv_heads, head_dim)
    return torch.zeros(num_blocks, num_kv_heads, 18 * head_dim, dtype=torch.uint8, device=device)


def _kv4_pool(pool, tables, status):
    """Checks; (device, head_dim)."""
    dev = _device(pool, "pool")
    _dense(pool, _U8, "pool", dev)
    _dense(tables, _I32, "tables", dev)
    if status is not None:
        _dense(status, _I32, "status", dev)
    if pool.dim() != 3 or tables.dim() != 2:
        raise ValueError("pool must be [num_blocks, num_kv_heads, 18 * head_dim], tables "
                         "[num_seqs, capacity]")
    _fits(*tables.shape)
    D, rest = divmod(pool.shape[2], 18)
    if rest:
        raise ValueError("pool pages must hold 18 * head_dim bytes per kv head")
    return dev, D


def _token_map(cu_seqlens, start_positions, tables, dev):
    _dense(cu_seqlens, _I32, "cu_seqlens", dev)
    _dense(start_positions, _I32, "start_positions", dev)
    S = tables.shape[0]
    if cu_seqlens.numel() != S + 1 or start_positions.numel() != S:
        raise ValueError("cu_seqlens [num_seqs + 1] and start_positions [num_seqs] must match "
                         "tables")


def kv4_write(k: torch.Tensor, v: torch.Tensor, pool: torch.Tensor, tables: torch.Tensor,
              cu_seqlens: torch.Tensor, start_positions: torch.Tensor, descale_k: float = 1.0,
              descale_v: float = 1.0, status: Optional[torch.Tensor] = None, stream=None):
    """Quantises packed k, v bf16 [T, Hkv, D] into a 4-bit pool (vfa_kv4_write).

    Token i of sequence s (row cu_seqlens[s] + i) becomes position
    start_positions[s] + i of its table row; rows past cu_seqlens[-1] are padding."""
    dev, D = _kv4_pool(pool, tables, status)
    _token_map(cu_seqlens, start_positions, tables, dev)
    blocks, Hkv, _ = pool.shape
    T = k.shape[0]
    ks, vs = _rows(k, (T, Hkv, D), "k", dev), _rows(v, (T, Hkv, D), "v", dev)
    st = (_lib or lib()).vfa_kv4_write(
        k.data_ptr(), v.data_ptr(), ks, vs, T, pool.data_ptr(), blocks, tables.data_ptr(),
        tables.shape[1], cu_seqlens.data_ptr(), start_positions.data_ptr(), tables.shape[0], Hkv, D,
        descale_k, descale_v, _address(status), _raw_stream(stream, dev))
    if st:
        _check(st)


def kv4_gather(pool: torch.Tensor, tables: torch.Tensor, cu_seqlens: torch.Tensor,
               start_positions: torch.Tensor, total_tokens: int, descale_k: float = 1.0,
               descale_v: float = 1.0, k_out: Optional[torch.Tensor] = None,
               v_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               stream=None):
    """(k, v) bf16 [total_tokens, Hkv, D] read back from a 4-bit pool, exactly (vfa_kv4_gather).

    Rows without a place in the cache are left as they were (unset if allocated here)."""
    dev, D = _kv4_pool(pool, tables, status)
    _token_map(cu_seqlens, start_positions, tables, dev)
    blocks, Hkv, _ = pool.shape
    shape = (total_tokens, Hkv, D)
    if k_out is None:
        k_out, ks = _empty(shape, torch.bfloat16, pool.device, stream), Hkv * D
    else:
        ks = _rows(k_out, shape, "k_out", dev)
    if v_out is None:
        v_out, vs = _empty(shape, torch.bfloat16, pool.device, stream), Hkv * D
    else:
        vs = _rows(v_out, shape, "v_out", dev)
    st = (_lib or lib()).vfa_kv4_gather(
        k_out.data_ptr(), v_out.data_ptr(), ks, vs, total_tokens, pool.data_ptr(), blocks,
        tables.data_ptr(), tables.shape[1], cu_seqlens.data_ptr(), start_positions.data_ptr(),
        tables.shape[0], Hkv, D, descale_k, descale_v, _address(status), _raw_stream(stream, dev))
    if st:
        _check(st)
    return k_out, v_out


def alloc_kv4_decode_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                               device="cuda") -> torch.Tensor:
    """A zero-filled workspace for kv4_decode (its tickets start at zero)."""
    n = (_lib or lib()).vfa_kv4_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise VfaError(VFA_ERR_UNSUPPORTED, "no 4-bit decode workspace for these sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kv4_decode(q: torch.Tensor, pool: torch.Tensor, tables: torch.Tensor,
               token_counts: torch.Tensor, descale_k: float = 1.0, descale_v: float = 1.0,
               softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream=None):
    """(out bf16 [S, Hq, D], lse f32 [S, Hq]): one query token per sequence over a 4-bit cache
    (vfa_kv4_decode).  Keep a workspace from alloc_kv4_decode_workspace between calls;
    without one, each call allocates and clears its own."""
    dev, D = _kv4_pool(pool, tables, status)
    _dense(q, _BF16, "q", dev)
    _dense(token_counts, _I32, "token_counts", dev)
    if q.dim() != 3 or q.shape[0] != tables.shape[0] or q.shape[2] != D:
        raise ValueError("q must be [num_seqs, num_q_heads, head_dim]")
    S, Hq, _ = q.shape
    blocks, Hkv, _ = pool.shape
    if token_counts.numel() != S:
        raise ValueError("token_counts must be [num_seqs]")
    if out is None:
        out = _empty_rows(q, stream)
    else:
        _dense(out, _BF16, "out", dev)
    if lse is None:
        lse = _empty((S, Hq), torch.float32, q.device, stream)
    else:
        _dense(lse, _F32, "lse", dev)
    if workspace is None:
        with _of(stream):
            workspace = alloc_kv4_decode_workspace(S, Hq, Hkv, D, device=q.device)
    else:
        _dense(workspace, _U8, "workspace", dev)
    if out.shape != q.shape or lse.shape != (S, Hq):
        raise ValueError("out must have q's shape and lse [num_seqs, num_q_heads]")
    st = (_lib or lib()).vfa_kv4_decode(
        q.data_ptr(), pool.data_ptr(), blocks, tables.data_ptr(), tables.shape[1],
        token_counts.data_ptr(), S, Hq, Hkv, D, descale_k, descale_v, softmax_scale, out.data_ptr(),
        lse.data_ptr(), _address(status), workspace.data_ptr(), workspace.numel(),
        _raw_stream(stream, dev))
    if st:
        _check(st)
    return out, lse


# ----------------------------------------------------------------- pages

def alloc_pages_workspace(num_blocks: int, num_seqs: int, num_forks: int = 0,
                          device="cuda") -> torch.Tensor:
    """Scratch of the page operations for at least these sizes."""
    n = (_lib or lib()).vfa_pages_workspace_bytes(num_blocks, num_seqs, num_forks)
    if n == 0:
        raise VfaError(VFA_ERR_INVALID_ARG, "no page workspace for these sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _page_state(refcounts, tables, token_counts, status, block_size):
    """Checks; (device, num_blocks, capacity, num_seqs)."""
    dev = _device(refcounts, "refcounts")
    _dense(refcounts, _I32, "refcounts", dev)
    _dense(tables, _I32, "tables", dev)
    _dense(token_counts, _I32, "token_counts", dev)
    if status is not None:
        _dense(status, _I32, "status", dev)
    if refcounts.dim() != 1 or tables.dim() != 2 or token_counts.dim() != 1 or \
            token_counts.shape[0] != tables.shape[0]:
        raise ValueError("refcounts [num_blocks], tables [num_seqs, capacity] and token_counts "
                         "[num_seqs]")
    S, cap = tables.shape
    blocks = refcounts.shape[0]
    _fits(blocks, cap, S, block_size)
    return dev, blocks, cap, S


def _pool_list(pools, num_blocks, dev):
    """Host arrays of the pools' addresses and page sizes."""
    n = len(pools)
    for i, p in enumerate(pools):
        if p.get_device() != dev or not p.is_contiguous():
            _refuse(p, p.dtype, f"pools[{i}]", dev)
        if p.dim() < 2 or p.size(0) != num_blocks:
            raise ValueError(f"pools[{i}] must hold {num_blocks} pages")
    blocks = max(num_blocks, 1)
    sizes = [p.nbytes // blocks for p in pools]
    _fits(num_blocks, *sizes)
    return (_P * n)(*[p.data_ptr() for p in pools]), (_I * n)(*sizes), n


def pages_extend(refcounts: torch.Tensor, tables: torch.Tensor, token_counts: torch.Tensor,
                 add_tokens: torch.Tensor, block_size: int, workspace: torch.Tensor,
                 status: Optional[torch.Tensor] = None, stream=None):
    """token_counts += add_tokens, with new pages where rows need them (vfa_pages_extend)."""
    dev, blocks, cap, S = _page_state(refcounts, tables, token_counts, status, block_size)
    _dense(workspace, _U8, "workspace", dev)
    _dense(add_tokens, _I32, "add_tokens", dev)
    if add_tokens.shape != token_counts.shape:
        raise ValueError("add_tokens must be [num_seqs]")
    st = (_lib or lib()).vfa_pages_extend(
        refcounts.data_ptr(), blocks, tables.data_ptr(), cap, token_counts.data_ptr(), S,
        add_tokens.data_ptr(), block_size, workspace.data_ptr(), workspace.numel(),
        _address(status), _raw_stream(stream, dev))
    if st:
        _check(st)


def pages_fork(refcounts: torch.Tensor, tables: torch.Tensor, token_counts: torch.Tensor,
               parents: torch.Tensor, children: torch.Tensor, pools, block_size: int,
               workspace: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None):
    """Rows children[i] become copies of rows parents[i]: full pages shared, a partly filled
    last page copied in every pool (vfa_pages_fork).  A negative parent skips the entry."""
    dev, blocks, cap, S = _page_state(refcounts, tables, token_counts, status, block_size)
    _dense(workspace, _U8, "workspace", dev)
    _dense(parents, _I32, "parents", dev)
    _dense(children, _I32, "children", dev)
    if parents.dim() != 1 or parents.shape != children.shape:
        raise ValueError("parents and children must be [num_forks]")
    _fits(parents.shape[0])
    ptrs, sizes, n = _pool_list(pools, blocks, dev)
    if parents.shape[0] == 0:
        return
    st = (_lib or lib()).vfa_pages_fork(
        refcounts.data_ptr(), blocks, tables.data_ptr(), cap, token_counts.data_ptr(), S,
        parents.data_ptr(), children.data_ptr(), parents.shape[0], ptrs, sizes, n, block_size,
        workspace.data_ptr(), workspace.numel(), _address(status), _raw_stream(stream, dev))
    if st:
        _check(st)


def pages_free(refcounts: torch.Tensor, tables: torch.Tensor, token_counts: torch.Tensor,
               seqs: torch.Tensor, block_size: int, status: Optional[torch.Tensor] = None,
               stream=None):
    """Rows seqs[i] give up their pages (vfa_pages_free).  A negative entry is skipped."""
    dev, blocks, cap, S = _page_state(refcounts, tables, token_counts, status, block_size)
    _dense(seqs, _I32, "seqs", dev)
    n = seqs.numel()
    _fits(n)
    if n == 0:
        return
    st = (_lib or lib()).vfa_pages_free(
        refcounts.data_ptr(), blocks, tables.data_ptr(), cap, token_counts.data_ptr(), S,
        seqs.data_ptr(), n, block_size, _address(status), _raw_stream(stream, dev))
    if st:
        _check(st)


def pages_compact(refcounts: torch.Tensor, tables: torch.Tensor, token_counts: torch.Tensor,
                  pools, block_size: int, workspace: torch.Tensor,
                  refcounts_out: Optional[torch.Tensor] = None,
                  tables_out: Optional[torch.Tensor] = None,
                  num_used: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the used pages to the low end of every pool (vfa_pages_compact); refcounts and
    tables are rewritten in place unless outputs are given.  Returns int32 [1]: used pages."""
    dev, blocks, cap, S = _page_state(refcounts, tables, token_counts, status, block_size)
    _dense(workspace, _U8, "workspace", dev)
    refcounts_out = refcounts if refcounts_out is None else refcounts_out
    tables_out = tables if tables_out is None else tables_out
    if num_used is None:
        num_used = _empty(1, torch.int32, refcounts.device, stream)
    for t, x, n in ((refcounts_out, refcounts, "refcounts_out"), (tables_out, tables, "tables_out")):
        _dense(t, _I32, n, dev)
        if t.shape != x.shape:
            raise ValueError(f"{n} must have shape {tuple(x.shape)}")
    _dense(num_used, _I32, "num_used", dev)
    ptrs, sizes, n = _pool_list(pools, blocks, dev)
    st = (_lib or lib()).vfa_pages_compact(
        refcounts.data_ptr(), blocks, tables.data_ptr(), cap, token_counts.data_ptr(), S, ptrs,
        sizes, n, block_size, refcounts_out.data_ptr(), tables_out.data_ptr(), num_used.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _address(status), _raw_stream(stream, dev))
    if st:
        _check(st)
    return num_used


def pages_copy(pools, src: torch.Tensor, dst: torch.Tensor,
               status: Optional[torch.Tensor] = None, stream=None):
    """Page src[i] of every pool over page dst[i] (vfa_pages_copy)."""
    if not pools:
        return
    dev = _device(src, "src")
    _dense(src, _I32, "src", dev)
    _dense(dst, _I32, "dst", dev)
    if status is not None:
        _dense(status, _I32, "status", dev)
    if src.dim() != 1 or src.shape != dst.shape:
        raise ValueError("src and dst must be [n]")
    _fits(src.shape[0])
    blocks = pools[0].shape[0]
    ptrs, sizes, n = _pool_list(pools, blocks, dev)
    if src.shape[0] == 0:
        return
    st = (_lib or lib()).vfa_pages_copy(
        ptrs, sizes, n, src.data_ptr(), dst.data_ptr(), src.shape[0], blocks, _address(status),
        _raw_stream(stream, dev))
    if st:
        _check(st)


def pages_truncate(refcounts: torch.Tensor, tables: torch.Tensor, token_counts: torch.Tensor,
                   new_counts: torch.Tensor, block_size: int,
                   refcounts_out: Optional[torch.Tensor] = None,
                   token_counts_out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None):
    """Rows shrink to new_counts tokens and give up the pages behind them (vfa_pages_truncate);
    refcounts and token_counts are rewritten in place unless outputs are given.  A negative
    new count leaves a row as it is."""
    dev, blocks, cap, S = _page_state(refcounts, tables, token_counts, status, block_size)
    refcounts_out = refcounts if refcounts_out is None else refcounts_out
    token_counts_out = token_counts if token_counts_out is None else token_counts_out
    for t, x, n in ((new_counts, token_counts, "new_counts"),
                    (refcounts_out, refcounts, "refcounts_out"),
                    (token_counts_out, token_counts, "token_counts_out")):
        _dense(t, _I32, n, dev)
        if t.shape != x.shape:
            raise ValueError(f"{n} must have shape {tuple(x.shape)}")
    if workspace is None:
        workspace = _empty(8 * S, torch.uint8, refcounts.device, stream)
    else:
        _dense(workspace, _U8, "workspace", dev)
    st = (_lib or lib()).vfa_pages_truncate(
        refcounts.data_ptr(), blocks, tables.data_ptr(), cap, token_counts.data_ptr(), S,
        new_counts.data_ptr(), block_size, refcounts_out.data_ptr(), token_counts_out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _address(status), _raw_stream(stream, dev))
    if st:
        _check(st)


# ----------------------------------------------------------------- a bounded bf16 cache

def _bf16_cache(k_pool, v_pool, tables, token_counts, status):
    """Checks; (device, num_blocks, num_kv_heads, head_dim, num_seqs, capacity)."""
    dev = _device(k_pool, "k_pool")
    _dense(k_pool, _BF16, "k_pool", dev)
    _dense(v_pool, _BF16, "v_pool", dev)
    _dense(tables, _I32, "tables", dev)
    _dense(token_counts, _I32, "token_counts", dev)
    if status is not None:
        _dense(status, _I32, "status", dev)
    if k_pool.dim() != 4 or k_pool.shape[1] != 16 or v_pool.shape != k_pool.shape:
        raise ValueError("k_pool and v_pool must be [num_blocks, 16, num_kv_heads, head_dim]")
    if tables.dim() != 2 or token_counts.shape != tables.shape[:1]:
        raise ValueError("tables must be [num_seqs, capacity] and token_counts [num_seqs]")
    blocks, _, Hkv, D = k_pool.shape
    S, cap = tables.shape
    _fits(blocks, Hkv, D, S, cap)
    return dev, blocks, Hkv, D, S, cap


def alloc_paged_decode_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                 capacity: int = 0, device="cuda") -> torch.Tensor:
    """A workspace for paged_decode (what starts at zero does); capacity: pages of a row, for
    calls with key_weights."""
    _fits(num_seqs, num_q_heads, num_kv_heads, capacity)
    n = (_lib or lib()).vfa_paged_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                         capacity)
    if n == 0:
        raise VfaError(VFA_ERR_UNSUPPORTED, "no paged decode workspace for these sizes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    # the logits at the end need no value
    ws[:(_lib or lib()).vfa_paged_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads,
                                                         head_dim, 0)].zero_()
    return ws


def paged_decode(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, tables: torch.Tensor,
                 token_counts: torch.Tensor, window_left: int = -1, sink_tokens: int = 0,
                 softmax_scale: float = 0.0, key_weights: Optional[torch.Tensor] = None,
                 key_weights_out: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream=None):
    """(out bf16 [S, Hq, D], lse f32 [S, Hq]): one new token per sequence, the last of its
    token_counts, over a paged bf16 cache with a window and sinks (vfa_paged_decode).

    key_weights f32 [S, Hkv, 16 * capacity]: the weight every visible token gets is added, in
    place unless key_weights_out is given.  Keep a workspace from
    alloc_paged_decode_workspace between calls; without one, each call allocates and clears
    its own."""
    dev, blocks, Hkv, D, S, cap = _bf16_cache(k_pool, v_pool, tables, token_counts, status)
    _dense(q, _BF16, "q", dev)
    if q.dim() != 3 or q.shape[0] != S or q.shape[2] != D:
        raise ValueError("q must be [num_seqs, num_q_heads, head_dim]")
    Hq = q.shape[1]
    _fits(Hq)
    if out is None:
        out = _empty_rows(q, stream)
    else:
        _dense(out, _BF16, "out", dev)
    if lse is None:
        lse = _empty((S, Hq), torch.float32, q.device, stream)
    else:
        _dense(lse, _F32, "lse", dev)
    if out.shape != q.shape or lse.shape != (S, Hq):
        raise ValueError("out must have q's shape and lse [num_seqs, num_q_heads]")
    if key_weights is not None:
        key_weights_out = key_weights if key_weights_out is None else key_weights_out
        for t, n in ((key_weights, "key_weights"), (key_weights_out, "key_weights_out")):
            _dense(t, _F32, n, dev)
            if t.shape != (S, Hkv, 16 * cap):
                raise ValueError(f"{n} must be [num_seqs, num_kv_heads, 16 * capacity]")
    elif key_weights_out is not None:
        raise ValueError("key_weights_out needs key_weights")
    if workspace is None:
        with _of(stream):
            workspace = alloc_paged_decode_workspace(S, Hq, Hkv, D, 0 if key_weights is None else cap,
                                                     device=q.device)
    else:
        _dense(workspace, _U8, "workspace", dev)
    st = (_lib or lib()).vfa_paged_decode(
        q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), blocks, tables.data_ptr(), cap,
        token_counts.data_ptr(), S, Hq, Hkv, D, _int32(window_left, "window_left"),
        _int32(sink_tokens, "sink_tokens"), softmax_scale, out.data_ptr(), lse.data_ptr(),
        _address(key_weights), _address(key_weights_out), _address(status), workspace.data_ptr(),
        workspace.numel(), _raw_stream(stream, dev))
    if st:
        _check(st)
    return out, lse


def alloc_key_weights_workspace(batch: int, total_q: int, total_k: int, max_seqlen_q: int,
                                num_heads: int, device="cuda") -> torch.Tensor:
    """Scratch of varlen_key_weights; its first int32 is the call's status word."""
    _fits(batch, total_q, total_k, max_seqlen_q, num_heads)
    n = (_lib or lib()).vfa_varlen_key_weights_workspace_bytes(batch, total_q, total_k, max_seqlen_q,
                                                               num_heads)
    if n == 0:
        raise VfaError(VFA_ERR_INVALID_ARG, "no key weights workspace for these sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def varlen_key_weights(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor,
                       cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, max_seqlen_q: int,
                       softmax_scale: float, causal, key_weights: torch.Tensor,
                       window_left: int = -1, sink_tokens: int = 0,
                       key_weights_out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """key_weights f32 [batch, Hkv, L] plus the attention weight that every packed key got
    (vfa_varlen_key_weights), in place unless key_weights_out is given; returns the sums.

    q [Tq, H, D], k [Tk, Hkv, D], lse [Tq, H] and the mask as in varlen_fwd, whose lse it is;
    key j of sequence b is entry j of row b.  read_status(workspace) tells of bad lengths."""
    dev = _device(q, "q")
    _dense(q, _BF16, "q", dev)
    _dense(k, _BF16, "k", dev)
    _dense(lse, _F32, "lse", dev)
    _dense(cu_seqlens_q, _I32, "cu_seqlens_q", dev)
    _dense(cu_seqlens_k, _I32, "cu_seqlens_k", dev)
    if q.dim() != 3 or k.dim() != 3 or q.shape[2] != k.shape[2] or lse.shape != q.shape[:2] or \
            k.shape[1] == 0 or q.shape[1] % k.shape[1] != 0:
        raise ValueError("q [Tq, H, D], k [Tk, Hkv, D] and lse [Tq, H] must agree, Hkv dividing H")
    batch = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != batch + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    (Tq, H, D), (Tk, Hkv, _) = q.shape, k.shape
    key_weights_out = key_weights if key_weights_out is None else key_weights_out
    for t, n in ((key_weights, "key_weights"), (key_weights_out, "key_weights_out")):
        _dense(t, _F32, n, dev)
        if t.dim() != 3 or t.shape[:2] != (batch, Hkv) or t.shape != key_weights.shape:
            raise ValueError(f"{n} must be [batch, num_kv_heads, L]")
    _fits(Tq, Tk, H, D, batch)
    max_seqlen_q = _int32(max_seqlen_q, "max_seqlen_q")
    if workspace is None:
        with _of(stream):
            workspace = alloc_key_weights_workspace(batch, Tq, Tk, max_seqlen_q, H, device=q.device)
    else:
        _dense(workspace, _U8, "workspace", dev)
    st = (_lib or lib()).vfa_varlen_key_weights(
        q.data_ptr(), k.data_ptr(), lse.data_ptr(), cu_seqlens_q.data_ptr(),
        cu_seqlens_k.data_ptr(), Tq, Tk, max_seqlen_q, batch, H, Hkv, D, softmax_scale,
        _int32(causal, "causal"), _int32(window_left, "window_left"), _int32(sink_tokens, "sink_tokens"),
        key_weights.data_ptr(), key_weights_out.data_ptr(), key_weights.shape[2],
        workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev))
    if st:
        _check(st)
    return key_weights_out


def alloc_evict_workspace(num_seqs: int, num_kv_heads: int, capacity: int,
                          device="cuda") -> torch.Tensor:
    """Scratch of cache_evict for at least these sizes."""
    _fits(num_seqs, num_kv_heads, capacity)
    n = (_lib or lib()).vfa_cache_evict_workspace_bytes(num_seqs, num_kv_heads, capacity)
    if n == 0:
        raise VfaError(VFA_ERR_INVALID_ARG, "no eviction workspace for these sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def cache_evict(k_pool: torch.Tensor, v_pool: torch.Tensor, refcounts: torch.Tensor,
                tables: torch.Tensor, token_counts: torch.Tensor, budgets: torch.Tensor,
                key_weights: torch.Tensor, positions: torch.Tensor, history: torch.Tensor,
                sink_tokens: int = 0, recent_tokens: int = 0,
                key_weights_out: Optional[torch.Tensor] = None,
                positions_out: Optional[torch.Tensor] = None,
                history_out: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """The tokens of little weight leave one layer's paged bf16 cache (vfa_cache_evict): of every
    row min(token_counts, budgets) tokens stay, each kv head its own.

    key_weights f32 and positions int32 [S, Hkv, 16 * capacity], history int32 [S, 2] (zeros at
    first); rewritten in place unless outputs are given.  Returns kept int32 [S], for
    pages_truncate once every layer has been called."""
    dev, blocks, Hkv, D, S, cap = _bf16_cache(k_pool, v_pool, tables, token_counts, status)
    key_weights_out = key_weights if key_weights_out is None else key_weights_out
    positions_out = positions if positions_out is None else positions_out
    history_out = history if history_out is None else history_out
    if kept is None:
        kept = _empty(S, torch.int32, tables.device, stream)
    rows = (S, Hkv, 16 * cap)
    want = ((refcounts, _I32, (blocks,), "refcounts"), (budgets, _I32, (S,), "budgets"),
            (key_weights, _F32, rows, "key_weights"), (key_weights_out, _F32, rows, "key_weights_out"),
            (positions, _I32, rows, "positions"), (positions_out, _I32, rows, "positions_out"),
            (history, _I32, (S, 2), "history"), (history_out, _I32, (S, 2), "history_out"),
            (kept, _I32, (S,), "kept"))
    for t, dtype, shape, n in want:
        if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            _dense(t, dtype, n, dev)
            raise ValueError(f"{n} must be {list(shape)}, got {list(t.shape)}")
    if workspace is None:
        n = (_lib or lib()).vfa_cache_evict_workspace_bytes(S, Hkv, cap)
        workspace = _empty(n, torch.uint8, tables.device, stream)
    else:
        _dense(workspace, _U8, "workspace", dev)
    st = (_lib or lib()).vfa_cache_evict(
        k_pool.data_ptr(), v_pool.data_ptr(), refcounts.data_ptr(), blocks, tables.data_ptr(), cap,
        token_counts.data_ptr(), budgets.data_ptr(), S, Hkv, D, key_weights.data_ptr(),
        positions.data_ptr(), history.data_ptr(), _int32(sink_tokens, "sink_tokens"),
        _int32(recent_tokens, "recent_tokens"), key_weights_out.data_ptr(),
        positions_out.data_ptr(), history_out.data_ptr(), kept.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _address(status), _raw_stream(stream, dev))
    if st:
        _check(st)
    return kept


def debug_bounded_wait(status: torch.Tensor, stream=None):
    """vfa_debug_bounded_wait: a wait nothing satisfies must end in VFA_ERR_TIMEOUT."""
    _need(status, torch.int32, "status")
    _check(lib().vfa_debug_bounded_wait(_ptr(status), _stream(stream)))


def debug_paged_gather(k_pool: torch.Tensor, v_pool: torch.Tensor, tile_blocks: torch.Tensor,
                       tile_block_counts: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor,
                       status: Optional[torch.Tensor] = None, stream=None):
    nb, bs, Hkv, D = k_pool.shape
    S, cap = tile_blocks.shape
    _check(lib().vfa_debug_paged_gather(_ptr(k_pool), _ptr(v_pool), nb, _ptr(tile_blocks),
                                        _ptr(tile_block_counts), cap, S, Hkv, D, bs,
                                        _ptr(k_out), _ptr(v_out), _ptr(status), _stream(stream)))
