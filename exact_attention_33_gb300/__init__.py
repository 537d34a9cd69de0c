"""Exact attention for GB300 (sm_103a): thin Python binding of libfa.so.

Every function here only marshals torch tensors into the C ABI declared in
``include/fa.h``, ``fa_window.h`` and ``fa_kvcache.h`` (device pointers, sizes, the current CUDA stream) and checks
the returned status; all arithmetic runs in the library's CUDA kernels.  There
is no fallback: if ``libfa.so`` is missing or a call fails, an exception is
raised.

Functions keep the C names (see ``__all__``).  Every tensor a call touches,
inputs, caller-supplied outputs and workspaces alike, is checked for device,
dtype, shape and contiguity before the library is called, since the kernels
trust the sizes they are given.  A call runs on the device of its ``q`` and
on that device's current stream unless ``stream`` is given.
"""

from __future__ import annotations

import ctypes
import math
import os
import threading
import warnings

__all__ = [
    "FaError", "library_path", "load_library", "fa_fwd", "fa_fwd_varlen", "fa_fwd_paged",
    "fa_fwd_splitkv", "fa_fwd_splitkv_workspace_size", "fa_fwd_fp8", "fa_fwd_varlen_fp8",
    "fa_bwd", "fa_bwd_varlen", "fa_bwd_workspace_size",
    "fa_decode_paged", "fa_decode_paged_noalloc", "fa_decode_workspace_size",
    "fa_fwd_window", "fa_fwd_varlen_window", "fa_fwd_paged_window", "fa_decode_paged_window",
    "fa_decode_window_workspace_size", "fa_bwd_window", "fa_bwd_varlen_window",
    "fa_bwd_window_workspace_size", "fa_cache_append_fp8", "fa_decode_paged_fp8",
    "fa_fwd_paged_fp8",
    "fa_status_string", "fa_device_status", "fa_last_device_status", "new_workspace",
    "FA_WORKSPACE_HEADER_BYTES",
    "fa_version", "FA_DEV_TIMEOUT", "FA_DEV_BAD_BLOCK", "FA_DEV_BAD_CTX", "FA_DEV_BAD_SEQLEN",
    "FA_DEV_BAD_INDEX", "FA_DEV_SMEM_ALIGN",
]

FA_OK = 0
FA_DEV_TIMEOUT = 1
FA_DEV_BAD_BLOCK = 2
FA_DEV_BAD_CTX = 4
FA_DEV_BAD_SEQLEN = 8
FA_DEV_BAD_INDEX = 16   # checked build only
FA_DEV_SMEM_ALIGN = 32  # a kernel found its shared memory not 1 KiB aligned
FA_WORKSPACE_HEADER_BYTES = 256   # control block at the start of a decode / split-KV workspace

_PKG = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None
_torch_module = None   # imported by the first call that needs it


class FaError(RuntimeError):
    def __init__(self, func: str, status: int):
        self.status = status
        super().__init__(f"{func} failed: {status} ({fa_status_string(status)})")


def library_path() -> str:
    """libfa.so, or the checked build libfa_checked.so when FA_CHECKED=1."""
    name = "libfa_checked.so" if os.environ.get("FA_CHECKED") == "1" else "libfa.so"
    return os.path.join(_PKG, name)


def load_library() -> ctypes.CDLL:
    """Load libfa.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m exact_attention_33_gb300.build` "
                "(add --checked for the checked build, or call __graft_entry__.build()); "
                "there is no non-CUDA fallback")
        lib = ctypes.CDLL(path)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        lib.fa_fwd.restype = i
        lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
        lib.fa_fwd_varlen.restype = i
        lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, f, f, f, i, vp]
        lib.fa_fwd_fp8.restype = i
        lib.fa_fwd_varlen_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, f, f, f, i, vp]
        lib.fa_fwd_varlen_fp8.restype = i
        lib.fa_bwd_workspace_size.argtypes = [i, i, i]
        lib.fa_bwd_workspace_size.restype = sz
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, sz, vp]
        lib.fa_bwd.restype = i
        lib.fa_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f,
                                      i, vp, sz, vp]
        lib.fa_bwd_varlen.restype = i
        lib.fa_fwd_splitkv_workspace_size.argtypes = [i, i, i, i, i]
        lib.fa_fwd_splitkv_workspace_size.restype = sz
        lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, sz, vp]
        lib.fa_fwd_splitkv.restype = i
        lib.fa_fwd_paged.argtypes = [vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, i, i, i, f, i,
                                     vp, vp, vp]
        lib.fa_fwd_paged.restype = i
        lib.fa_decode_workspace_size.argtypes = [i, i, i, i, i, i]
        lib.fa_decode_workspace_size.restype = sz
        lib.fa_decode_paged.argtypes = [vp, vp, vp, vp, i, vp, i, i, i, i, i, i, i, f, vp, vp,
                                        vp, sz, vp]
        lib.fa_decode_paged.restype = i
        lib.fa_decode_paged_noalloc.argtypes = [vp, vp, vp, vp, i, vp, i, i, i, i, i, i, i, f,
                                                vp, vp, vp]
        lib.fa_decode_paged_noalloc.restype = i
        lib.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
        lib.fa_fwd_window.restype = i
        lib.fa_fwd_varlen_window.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
        lib.fa_fwd_varlen_window.restype = i
        lib.fa_fwd_paged_window.argtypes = [vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, i, i, i,
                                            f, i, i, vp, vp, vp]
        lib.fa_fwd_paged_window.restype = i
        lib.fa_decode_window_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
        lib.fa_decode_window_workspace_size.restype = sz
        lib.fa_decode_paged_window.argtypes = [vp, vp, vp, vp, i, vp, i, i, i, i, i, i, i, f, i, i,
                                               vp, vp, vp, sz, vp]
        lib.fa_decode_paged_window.restype = i
        lib.fa_bwd_window_workspace_size.argtypes = [i, i, i, i, i, i, i]
        lib.fa_bwd_window_workspace_size.restype = sz
        lib.fa_bwd_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i,
                                      vp, sz, vp]
        lib.fa_bwd_window.restype = i
        lib.fa_bwd_varlen_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i,
                                             i, f, i, i, vp, sz, vp]
        lib.fa_bwd_varlen_window.restype = i
        i64 = ctypes.c_int64
        lib.fa_cache_append_fp8.argtypes = [vp, vp, i64, i64, vp, vp, vp, vp, vp, i, vp, vp, i, i,
                                            i, i, i, i, i, vp]
        lib.fa_cache_append_fp8.restype = i
        lib.fa_decode_paged_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, i, i, f,
                                            i, i, vp, vp, vp, sz, vp]
        lib.fa_decode_paged_fp8.restype = i
        lib.fa_fwd_paged_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, i, i,
                                         i, f, i, i, vp, vp, vp]
        lib.fa_fwd_paged_fp8.restype = i
        lib.fa_status_string.argtypes = [i]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), i]
        lib.fa_device_status.restype = i
        lib.fa_last_device_status.argtypes = [vp]
        lib.fa_last_device_status.restype = i
        lib.fa_selftest_wait_timeout.argtypes = [vp, vp]
        lib.fa_selftest_wait_timeout.restype = i
        lib.fa_version.argtypes = []
        lib.fa_version.restype = i
        _lib = lib
        return lib


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(int(status)).decode()


def fa_version() -> int:
    return int(load_library().fa_version())


def fa_selftest_wait_timeout(stream=None) -> int:
    """Run the bounded-wait self-test; returns the wait's result (0 = it gave
    up, as intended).  FA_DEV_TIMEOUT is set in the status word afterwards."""
    torch = _torch()
    res = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    rc = load_library().fa_selftest_wait_timeout(_ptr(res), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError("fa_selftest_wait_timeout", rc)
    torch.cuda.synchronize()
    return int(res.item())


def fa_device_status(clear: bool = True) -> int:
    """Sticky device status word (FA_DEV_* bits); synchronises the device."""
    v = ctypes.c_uint(0)
    rc = load_library().fa_device_status(ctypes.byref(v), 1 if clear else 0)
    if rc != FA_OK:
        raise FaError("fa_device_status", rc)
    return int(v.value)


def fa_last_device_status(workspace) -> int:
    """FA_DEV_* bits of the last call that finished on ``workspace`` (a
    decode or split-KV workspace).  Read it after that call has completed
    (synchronise its stream first); it does not wait for other streams."""
    torch = _torch()
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda \
            or workspace.numel() * workspace.element_size() < FA_WORKSPACE_HEADER_BYTES:
        raise ValueError("workspace must be a CUDA tensor of at least "
                         f"{FA_WORKSPACE_HEADER_BYTES} bytes")
    with torch.cuda.device(workspace.device):
        rc = load_library().fa_last_device_status(_ptr(workspace))
    if rc < 0:
        raise FaError("fa_last_device_status", rc)
    return int(rc)


def new_workspace(nbytes: int, device=None):
    """A decode or split-KV workspace of ``nbytes`` bytes, zero-filled as the
    library requires before its first call."""
    torch = _torch()
    return torch.zeros(max(int(nbytes), FA_WORKSPACE_HEADER_BYTES), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


# ----------------------------------------------------------------- helpers

def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_handle(stream=None, device=None):
    torch = _torch()
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(int(s.cuda_stream))


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else int(t.data_ptr()))


def _check_bf16_cuda(name, t, ndim, device=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor")


def _check_tensor(name, t, shape, dtype, device):
    """A tensor the kernels read or write with exactly this shape and dtype."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")


def _check_int32(name, t, device, ndim=1, numel=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != torch.int32 or t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D int32 tensor")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} values")


def _workspace(t, need, device, minimum=1, zero=False):
    """The caller's workspace (a 1-D uint8 tensor, its length in bytes), or a
    new one of at least ``need`` bytes (zero-filled with ``zero``: decode and
    split-KV workspaces start with a control block that must be zero)."""
    torch = _torch()
    if t is None:
        alloc = torch.zeros if zero else torch.empty
        return alloc(max(need, minimum), dtype=torch.uint8, device=device)
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.uint8 \
            or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous 1-D uint8 tensor on {device}")
    return t


def _outputs(q_like_shape, lse_shape, out, lse, want_lse, device):
    torch = _torch()
    if out is None:
        out = torch.empty(q_like_shape, dtype=torch.bfloat16, device=device)
    else:
        _check_tensor("out", out, q_like_shape, torch.bfloat16, device)
    if lse is None and want_lse:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=device)
    elif lse is not None:
        _check_tensor("lse", lse, lse_shape, torch.float32, device)
    return out, lse


def _scale(scale, d):
    return float(1.0 / math.sqrt(d)) if scale is None else float(scale)


# ----------------------------------------------------------------- calls

def fa_fwd(q, k, v, causal=False, scale=None, out=None, lse=None, want_lse=True, stream=None):
    """Dense prefill.  q [B,N,H,d], k/v [B,N,Hkv,d] bf16 CUDA tensors.

    Returns (out [B,N,H,d] bf16, lse [B,H,N] fp32 or None).
    """
    torch = _torch()
    _check_bf16_cuda("q", q, 4)
    dev = q.device
    for name, t in (("k", k), ("v", v)):
        _check_bf16_cuda(name, t, 4, dev)
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, N, Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, N, Hkv, d] matching q")
    out, lse = _outputs(q.shape, (B, H, N), out, lse, want_lse, dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv,
                                   N, d, _scale(scale, d), 1 if causal else 0,
                                   _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_fwd", rc)
    return out, lse


def fa_bwd_workspace_size(B, H, N) -> int:
    return int(load_library().fa_bwd_workspace_size(B, H, N))


def fa_bwd(q, k, v, out, lse, dout, causal=False, scale=None, dq=None, dk=None, dv=None,
           workspace=None, stream=None):
    """Gradient of dense attention.  q, out, dout [B,N,H,d]; k, v [B,N,Hkv,d]
    bf16 CUDA tensors; lse [B,H,N] fp32 from fa_fwd.  Returns (dq, dk, dv)."""
    torch = _torch()
    _check_bf16_cuda("q", q, 4)
    dev = q.device
    for name, t in (("k", k), ("v", v), ("out", out), ("dout", dout)):
        _check_bf16_cuda(name, t, 4, dev)
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, N, Hkv, d) or v.shape != k.shape or out.shape != q.shape \
            or dout.shape != q.shape:
        raise ValueError("shapes must be q/out/dout [B,N,H,d], k/v [B,N,Hkv,d]")
    _check_tensor("lse", lse, (B, H, N), torch.float32, dev)
    grads = []
    for name, g, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if g is None:
            g = torch.empty_like(like)
        else:
            _check_tensor(name, g, like.shape, torch.bfloat16, dev)
        grads.append(g)
    dq, dk, dv = grads
    workspace = _workspace(workspace, fa_bwd_workspace_size(B, H, N), dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                   _ptr(dq), _ptr(dk), _ptr(dv), B, H, Hkv, N, d,
                                   _scale(scale, d), 1 if causal else 0, _ptr(workspace),
                                   workspace.numel(), _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_bwd", rc)
    return dq, dk, dv


def fa_bwd_varlen(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, causal=False, scale=None,
                  dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradient of a packed varlen batch.  q, out, dout [T,H,d]; k, v [T,Hkv,d]
    bf16 CUDA tensors; lse [H,T] fp32 from fa_fwd_varlen; cu_seqlens int32
    [S+1] on the device.  Returns (dq, dk, dv); rows outside every sequence
    are left as they were."""
    torch = _torch()
    _check_bf16_cuda("q", q, 3)
    dev = q.device
    for name, t in (("k", k), ("v", v), ("out", out), ("dout", dout)):
        _check_bf16_cuda(name, t, 3, dev)
    _check_int32("cu_seqlens", cu_seqlens, dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold num_seqs + 1 offsets")
    T, H, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (T, Hkv, d) or v.shape != k.shape or out.shape != q.shape \
            or dout.shape != q.shape:
        raise ValueError("shapes must be q/out/dout [T,H,d], k/v [T,Hkv,d]")
    _check_tensor("lse", lse, (H, T), torch.float32, dev)
    grads = []
    for name, g, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if g is None:
            g = torch.empty_like(like)
        else:
            _check_tensor(name, g, like.shape, torch.bfloat16, dev)
        grads.append(g)
    dq, dk, dv = grads
    S = cu_seqlens.numel() - 1
    workspace = _workspace(workspace, fa_bwd_workspace_size(S, H, min(int(max_seqlen), T)), dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_bwd_varlen(
            _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
            _ptr(dv), _ptr(cu_seqlens), S, T, int(max_seqlen), H, Hkv, d, _scale(scale, d),
            1 if causal else 0, _ptr(workspace), workspace.numel(), _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_bwd_varlen", rc)
    return dq, dk, dv


def fa_fwd_fp8(q, k, v, q_descale, k_descale, v_descale, causal=False, scale=None, out=None,
               lse=None, want_lse=True, stream=None):
    """Dense prefill on e4m3 codes.  q [B,N,H,d], k/v [B,N,Hkv,d] uint8 CUDA
    tensors holding e4m3 bits; per-tensor descales.  Returns (out bf16, lse)."""
    torch = _torch()
    dev = q.device if isinstance(q, torch.Tensor) else None
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != dev \
                or t.dtype not in (torch.uint8, torch.float8_e4m3fn) or t.dim() != 4 \
                or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D uint8/e4m3 CUDA tensor on the "
                             "device of q")
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, N, Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, N, Hkv, d] matching q")
    out, lse = _outputs((B, N, H, d), (B, H, N), out, lse, want_lse, dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H,
                                       Hkv, N, d, _scale(scale, d), float(q_descale),
                                       float(k_descale), float(v_descale), 1 if causal else 0,
                                       _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_fwd_fp8", rc)
    return out, lse


def _check_fp8(name, t, ndim, dev):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != dev \
            or t.dtype not in (torch.uint8, torch.float8_e4m3fn) or t.dim() != ndim \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D uint8/e4m3 CUDA tensor on the "
                         "device of q")


def fa_fwd_varlen_fp8(q, k, v, cu_seqlens, max_seqlen, q_descale, k_descale, v_descale,
                      causal=False, scale=None, out=None, lse=None, want_lse=True, stream=None):
    """Packed varlen prefill on e4m3 codes.  q [T,H,d], k/v [T,Hkv,d] uint8
    CUDA tensors holding e4m3 bits, cu_seqlens int32 [S+1] on the device;
    per-tensor descales.  Returns (out [T,H,d] bf16, lse [H,T] fp32 or None)."""
    torch = _torch()
    dev = q.device if isinstance(q, torch.Tensor) else None
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_fp8(name, t, 3, dev)
    _check_int32("cu_seqlens", cu_seqlens, dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold num_seqs + 1 offsets")
    T, H, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (T, Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [T, Hkv, d] matching q")
    out, lse = _outputs((T, H, d), (H, T), out, lse, want_lse, dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_fwd_varlen_fp8(
            _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_seqlens),
            cu_seqlens.numel() - 1, T, int(max_seqlen), H, Hkv, d, _scale(scale, d),
            float(q_descale), float(k_descale), float(v_descale), 1 if causal else 0,
            _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_fwd_varlen_fp8", rc)
    return out, lse


def fa_fwd_splitkv_workspace_size(B, H, N, d, num_splits=0) -> int:
    return int(load_library().fa_fwd_splitkv_workspace_size(B, H, N, d, num_splits))


def fa_fwd_splitkv(q, k, v, causal=False, scale=None, num_splits=0, out=None, lse=None,
                   workspace=None, want_lse=True, stream=None):
    """Dense prefill with split-KV partial states and a combine (for small
    B * H).  Same layouts as :func:`fa_fwd`."""
    torch = _torch()
    _check_bf16_cuda("q", q, 4)
    dev = q.device
    for name, t in (("k", k), ("v", v)):
        _check_bf16_cuda(name, t, 4, dev)
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, N, Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, N, Hkv, d] matching q")
    workspace = _workspace(workspace, fa_fwd_splitkv_workspace_size(B, H, N, d, num_splits),
                           dev, 256, zero=True)
    out, lse = _outputs(q.shape, (B, H, N), out, lse, want_lse, dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B,
                                           H, Hkv, N, d, _scale(scale, d), 1 if causal else 0,
                                           int(num_splits), _ptr(workspace), workspace.numel(),
                                           _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_fwd_splitkv", rc)
    return out, lse


def fa_fwd_varlen(q, k, v, cu_seqlens, max_seqlen, causal=False, scale=None, out=None,
                  lse=None, want_lse=True, stream=None):
    """Packed varlen prefill.  q [T,H,d], k/v [T,Hkv,d], cu_seqlens int32 [S+1] on device.

    Returns (out [T,H,d] bf16, lse [H,T] fp32 or None).
    """
    torch = _torch()
    _check_bf16_cuda("q", q, 3)
    dev = q.device
    for name, t in (("k", k), ("v", v)):
        _check_bf16_cuda(name, t, 3, dev)
    _check_int32("cu_seqlens", cu_seqlens, dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold num_seqs + 1 offsets")
    T, H, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (T, Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [T, Hkv, d] matching q")
    out, lse = _outputs(q.shape, (H, T), out, lse, want_lse, dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                          _ptr(cu_seqlens), cu_seqlens.numel() - 1, T,
                                          int(max_seqlen), H, Hkv, d, _scale(scale, d),
                                          1 if causal else 0, _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_fwd_varlen", rc)
    return out, lse


def _check_pools(k_pool, v_pool, dev):
    _check_bf16_cuda("k_pool", k_pool, 4, dev)
    _check_bf16_cuda("v_pool", v_pool, 4, dev)
    if v_pool.shape != k_pool.shape:
        raise ValueError("k_pool and v_pool must have the same shape [num_blocks,16,Hkv,d]")
    return k_pool.shape


def fa_fwd_paged(q, k_pool, v_pool, block_table, ctx_lens, cu_seqlens_q, max_seqlen_q,
                 max_ctx_len, causal=True, scale=None, out=None, lse=None, want_lse=True,
                 stream=None):
    """Query chunks [Tq,H,d] against a paged KV cache (chunked prefill).

    pools [num_blocks,16,Hkv,d] bf16; block_table int32 [batch,max_blocks];
    ctx_lens int32 [batch]; cu_seqlens_q int32 [batch+1]; all on the device.
    Returns (out [Tq,H,d] bf16, lse [H,Tq] fp32 or None).
    """
    torch = _torch()
    _check_bf16_cuda("q", q, 3)
    dev = q.device
    num_blocks, block_size, Hkv, dp = _check_pools(k_pool, v_pool, dev)
    _check_int32("block_table", block_table, dev, ndim=2)
    batch = block_table.shape[0]
    _check_int32("ctx_lens", ctx_lens, dev, numel=batch)
    _check_int32("cu_seqlens_q", cu_seqlens_q, dev, numel=batch + 1)
    Tq, H, d = q.shape
    if dp != d:
        raise ValueError("the pools' head size must match q")
    out, lse = _outputs(q.shape, (H, Tq), out, lse, want_lse, dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_fwd_paged(
            _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), block_table.shape[1],
            _ptr(ctx_lens), _ptr(cu_seqlens_q), batch, Tq, int(max_seqlen_q),
            int(max_ctx_len), H, Hkv, d, block_size, num_blocks, _scale(scale, d),
            1 if causal else 0, _ptr(out), _ptr(lse), _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_fwd_paged", rc)
    return out, lse


def fa_decode_workspace_size(batch, H, Hkv, d, max_ctx_len, block_size=16) -> int:
    return int(load_library().fa_decode_workspace_size(batch, H, Hkv, d, max_ctx_len,
                                                       block_size))


def _decode_args(q, k_pool, v_pool, block_table, ctx_lens):
    _check_bf16_cuda("q", q, 3)
    dev = q.device
    num_blocks, block_size, Hkv, dp = _check_pools(k_pool, v_pool, dev)
    batch, H, d = q.shape
    if dp != d:
        raise ValueError("the pools' head size must match q")
    _check_int32("block_table", block_table, dev, ndim=2)
    if block_table.shape[0] != batch:
        raise ValueError("block_table must have one row per sequence of q")
    _check_int32("ctx_lens", ctx_lens, dev, numel=batch)
    return dev, batch, H, Hkv, d, num_blocks, block_size


def fa_decode_paged(q, k_pool, v_pool, block_table, ctx_lens, max_ctx_len, scale=None,
                    out=None, lse=None, workspace=None, want_lse=True, stream=None):
    """Paged GQA flash-decoding.

    q [batch,H,d]; pools [num_blocks,block_size,Hkv,d] bf16; block_table int32
    [batch, max_blocks]; ctx_lens int32 [batch]; all on the device.
    Returns (out [batch,H,d] bf16, lse [batch,H] fp32 or None).
    """
    torch = _torch()
    dev, batch, H, Hkv, d, num_blocks, block_size = _decode_args(q, k_pool, v_pool,
                                                                 block_table, ctx_lens)
    workspace = _workspace(
        workspace, fa_decode_workspace_size(batch, H, Hkv, d, max_ctx_len, block_size), dev, 256,
        zero=True)
    out, lse = _outputs(q.shape, (batch, H), out, lse, want_lse, dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_decode_paged(
            _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), block_table.shape[1],
            _ptr(ctx_lens), int(max_ctx_len), batch, H, Hkv, d, block_size, num_blocks,
            _scale(scale, d), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
            _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_decode_paged", rc)
    return out, lse


FA_DECODE_NOALLOC_SCRATCH_BYTES = 32 << 20


def fa_decode_paged_noalloc(q, k_pool, v_pool, block_table, ctx_lens, max_ctx_len, *, out,
                            lse=None, scale=None, stream=None):
    """Paged decode that allocates nothing on the device, for callers that
    cannot call cudaMalloc (a plugin whose host framework owns all device
    memory, or a decode loop that must avoid the implicit synchronisation of
    cudaMalloc/cudaFree).  The split partial states live in the library's
    static scratch array of FA_DECODE_NOALLOC_SCRATCH_BYTES; larger requests
    are rejected.  The caller passes ``out`` (and optionally ``lse``); calls
    whose kernels overlap on the GPU race on the shared scratch."""
    torch = _torch()
    dev, batch, H, Hkv, d, num_blocks, block_size = _decode_args(q, k_pool, v_pool,
                                                                 block_table, ctx_lens)
    _check_tensor("out", out, q.shape, torch.bfloat16, dev)
    if lse is not None:
        _check_tensor("lse", lse, (batch, H), torch.float32, dev)
    with torch.cuda.device(dev):
        rc = load_library().fa_decode_paged_noalloc(
            _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), block_table.shape[1],
            _ptr(ctx_lens), int(max_ctx_len), batch, H, Hkv, d, block_size, num_blocks,
            _scale(scale, d), _ptr(out), _ptr(lse), _stream_handle(stream, dev))
    if rc != FA_OK:
        raise FaError("fa_decode_paged_noalloc", rc)
    return out, lse


# ------------------------------------------------------- windowed attention
#
# A query at position p of its sequence sees key j <= p when j > p - window
# or j < sinks (include/fa_window.h).

def _check_window(window, sinks):
    window, sinks = int(window), int(sinks)
    if window < 1 or sinks < 0:
        raise ValueError("window must be at least 1 and sinks at least 0")
    limit = 0x7FFFFFFF   # every sequence is shorter
    return min(window, limit), min(sinks, limit)


class _Launch:
    """``with _Launch(stream, dev) as handle``: the call's device is current,
    and so is ``stream`` where one is given, so that what the call allocates
    (outputs, workspace) belongs to the stream that it runs on.  ``handle`` is
    the stream's address."""

    __slots__ = ("context", "stream", "device")

    def __init__(self, stream, device):
        cuda = _torch().cuda
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream must be a stream of {device}")
            self.context = cuda.stream(stream)
        else:  # entering a device costs more than asking which one is current
            self.context = None if cuda.current_device() == device.index else cuda.device(device)
        self.stream, self.device = stream, device

    def __enter__(self):
        if self.context is not None:
            self.context.__enter__()
        if self.stream is not None:
            return self.stream.cuda_stream
        return _current_stream(self.device)

    def __exit__(self, *exc):
        return self.context.__exit__(*exc) if self.context is not None else None


def _current_stream(device):
    """Address of the device's current stream, without a Stream object where
    torch offers that."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream


def _are(dtype, index, *pairs):
    """Every (tensor, shape) of ``pairs`` is a contiguous tensor of this type
    and shape on CUDA device ``index``.  The calls ask this first; the checks
    that name what is wrong run only when the answer is no."""
    try:
        for t, shape in pairs:
            if t.dtype is not dtype or t.shape != shape or t.get_device() != index \
                    or not t.is_contiguous():
                return False
    except AttributeError:
        return False
    return True


_calls = None   # the extension module, or False where it has not been built

# the library's functions that the extension calls, in its order
_BOUND = ("fa_fwd_window", "fa_fwd_varlen_window", "fa_fwd_paged_window", "fa_decode_paged_window",
          "fa_bwd_window", "fa_bwd_varlen_window", "fa_cache_append_fp8", "fa_decode_paged_fp8",
          "fa_fwd_paged_fp8")


def _short():
    """The extension module (csrc/torch_calls.cpp) whose functions make a call
    on the current stream when all its tensors are as they should be, and
    return None otherwise; the functions here go on from there.  False where it
    has not been built or does not load: the calls are then made from here, which
    takes longer."""
    global _calls
    if _calls is None:
        lib = load_library()
        _torch()   # its libraries first
        path = os.path.join(_PKG, "_torch_calls.so")
        if not os.path.exists(path):
            _calls = False
            return _calls
        import importlib.util
        try:
            spec = importlib.util.spec_from_file_location(__name__ + "._torch_calls", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _BOUND))
            _calls = module
        except Exception as e:  # made for another torch or Python
            _calls = False
            warnings.warn(f"calls on torch tensors take longer: {path} does not load ({e})",
                          RuntimeWarning)
    return _calls


def _addr(t):
    """Device address of a tensor, 0 for None (the C arguments take an int)."""
    return 0 if t is None else t.data_ptr()


def _results(q, lse_shape, out, lse, want_lse):
    """The output tensors: the caller's, checked, or new ones."""
    if out is not None or lse is not None:
        return _outputs(q.shape, lse_shape, out, lse, want_lse, q.device)
    torch = _torch()
    return torch.empty(q.shape, dtype=q.dtype, device=q.device), \
        torch.empty(lse_shape, dtype=torch.float32, device=q.device) if want_lse else None


def _check_table(block_table, ctx_lens, batch, dev):
    i32 = _torch().int32
    if not _are(i32, dev.index, (block_table, (batch, *block_table.shape[1:])), (ctx_lens, (batch,))) \
            or block_table.dim() != 2:
        _check_int32("block_table", block_table, dev, ndim=2)
        _check_int32("ctx_lens", ctx_lens, dev, numel=batch)
        raise ValueError("block_table must have one row per sequence")


def _check_sequences(block_table, ctx_lens, cu_seqlens, cu_name, dev):
    """Checks the int32 arrays of a call on packed rows over a cache; returns
    the number of sequences."""
    shape = getattr(block_table, "shape", ())
    if len(shape) != 2 or not _are(_torch().int32, dev.index, (block_table, shape),
                                   (ctx_lens, shape[:1]), (cu_seqlens, (shape[0] + 1,))):
        _check_int32("block_table", block_table, dev, ndim=2)
        _check_int32("ctx_lens", ctx_lens, dev, numel=block_table.shape[0])
        _check_int32(cu_name, cu_seqlens, dev, numel=block_table.shape[0] + 1)
    return block_table.shape[0]


def fa_fwd_window(q, k, v, window, sinks=0, scale=None, out=None, lse=None, want_lse=True,
                  stream=None):
    """Dense causal prefill over the last ``window`` keys and the first
    ``sinks`` keys.  q [B,N,H,d], k/v [B,N,Hkv,d] bf16 CUDA tensors.

    Returns (out [B,N,H,d] bf16, lse [B,H,N] fp32 or None).
    """
    short = _calls or _short()
    if short and stream is None:
        done = short.fwd_window(q, k, v, window, sinks, scale, want_lse, out, lse)
        if done is not None:
            return done
    _check_bf16_cuda("q", q, 4)
    dev = q.device
    B, N, H, d = q.shape
    if not _are(q.dtype, dev.index, (k, v.shape), (v, k.shape)) or k.dim() != 4 \
            or k.shape[:2] != (B, N) or k.shape[3] != d:
        for name, t in (("k", k), ("v", v)):
            _check_bf16_cuda(name, t, 4, dev)
        raise ValueError("k and v must be [B, N, Hkv, d] matching q")
    Hkv = k.shape[2]
    window, sinks = _check_window(window, sinks)
    with _Launch(stream, dev) as handle:
        out, lse = _results(q, (B, H, N), out, lse, want_lse)
        if not B * N:   # (an empty tensor has no address)
            return out, lse
        rc = load_library().fa_fwd_window(_addr(q), _addr(k), _addr(v), _addr(out), _addr(lse), B, H,
                                          Hkv, N, d, _scale(scale, d), window, sinks,
                                          handle)
    if rc != FA_OK:
        raise FaError("fa_fwd_window", rc)
    return out, lse


def fa_fwd_varlen_window(q, k, v, cu_seqlens, max_seqlen, window, sinks=0, scale=None, out=None,
                         lse=None, want_lse=True, stream=None):
    """Packed causal prefill over each sequence's last ``window`` and first
    ``sinks`` keys.  q [T,H,d], k/v [T,Hkv,d], cu_seqlens int32 [S+1] on device.

    Returns (out [T,H,d] bf16, lse [H,T] fp32 or None).
    """
    short = _calls or _short()
    if short and stream is None:
        done = short.fwd_varlen_window(q, k, v, cu_seqlens, max_seqlen, window, sinks, scale, want_lse,
                                       out, lse)
        if done is not None:
            return done
    _check_bf16_cuda("q", q, 3)
    dev = q.device
    T, H, d = q.shape
    if not _are(q.dtype, dev.index, (k, v.shape), (v, k.shape)) or k.dim() != 3 \
            or k.shape[0] != T or k.shape[2] != d:
        for name, t in (("k", k), ("v", v)):
            _check_bf16_cuda(name, t, 3, dev)
        raise ValueError("k and v must be [T, Hkv, d] matching q")
    Hkv = k.shape[1]
    _check_int32("cu_seqlens", cu_seqlens, dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold num_seqs + 1 offsets")
    window, sinks = _check_window(window, sinks)
    with _Launch(stream, dev) as handle:
        out, lse = _results(q, (H, T), out, lse, want_lse)
        if not T:
            return out, lse
        rc = load_library().fa_fwd_varlen_window(
            _addr(q), _addr(k), _addr(v), _addr(out), _addr(lse), _addr(cu_seqlens),
            cu_seqlens.numel() - 1, T, int(max_seqlen), H, Hkv, d, _scale(scale, d), window, sinks,
            handle)
    if rc != FA_OK:
        raise FaError("fa_fwd_varlen_window", rc)
    return out, lse


def fa_fwd_paged_window(q, k_pool, v_pool, block_table, ctx_lens, cu_seqlens_q, max_seqlen_q,
                        max_ctx_len, window, sinks=0, scale=None, out=None, lse=None,
                        want_lse=True, stream=None):
    """:func:`fa_fwd_paged` (causal) over each query's last ``window`` keys and
    the first ``sinks`` keys.  Blocks behind the window of a chunk's first
    query, but for those of the sinks, are not read and may have been freed."""
    short = _calls or _short()
    if short and stream is None:
        done = short.fwd_paged_window(q, k_pool, v_pool, block_table, ctx_lens, cu_seqlens_q,
                                      max_seqlen_q, max_ctx_len, window, sinks, scale, want_lse, out,
                                      lse)
        if done is not None:
            return done
    _check_bf16_cuda("q", q, 3)
    dev = q.device
    num_blocks, block_size, Hkv, dp = _check_pools(k_pool, v_pool, dev)
    batch = _check_sequences(block_table, ctx_lens, cu_seqlens_q, "cu_seqlens_q", dev)
    window, sinks = _check_window(window, sinks)
    Tq, H, d = q.shape
    if dp != d:
        raise ValueError("the pools' head size must match q")
    with _Launch(stream, dev) as handle:
        out, lse = _results(q, (H, Tq), out, lse, want_lse)
        if not Tq:
            return out, lse
        rc = load_library().fa_fwd_paged_window(
            _addr(q), _addr(k_pool), _addr(v_pool), _addr(block_table), block_table.shape[1],
            _addr(ctx_lens), _addr(cu_seqlens_q), batch, Tq, int(max_seqlen_q), int(max_ctx_len), H,
            Hkv, d, block_size, num_blocks, _scale(scale, d), window, sinks, _addr(out), _addr(lse),
            handle)
    if rc != FA_OK:
        raise FaError("fa_fwd_paged_window", rc)
    return out, lse


def fa_decode_window_workspace_size(batch, H, Hkv, d, max_ctx_len, window, sinks=0,
                                    block_size=16) -> int:
    """Bytes of workspace of a decode call with this window (0: every key)."""
    window, sinks = _check_cache_window(window, sinks)
    return int(load_library().fa_decode_window_workspace_size(batch, H, Hkv, d, max_ctx_len,
                                                              block_size, window, sinks))


def fa_decode_paged_window(q, k_pool, v_pool, block_table, ctx_lens, max_ctx_len, window, sinks=0,
                           scale=None, out=None, lse=None, workspace=None, want_lse=True,
                           stream=None):
    """:func:`fa_decode_paged` over the last ``window`` keys and the first
    ``sinks`` keys of each sequence; other blocks are not read."""
    short = _calls or _short()
    if short and stream is None:
        done = short.decode_paged_window(q, k_pool, v_pool, block_table, ctx_lens, max_ctx_len, window,
                                         sinks, scale, want_lse, out, lse, workspace)
        if done is not None:
            return done
    _check_bf16_cuda("q", q, 3)
    dev = q.device
    batch, H, d = q.shape
    if not _are(q.dtype, dev.index, (k_pool, v_pool.shape), (v_pool, k_pool.shape)) \
            or k_pool.dim() != 4 or k_pool.shape[3] != d:
        _check_pools(k_pool, v_pool, dev)
        raise ValueError("the pools' head size must match q")
    num_blocks, block_size, Hkv, _ = k_pool.shape
    _check_table(block_table, ctx_lens, batch, dev)
    window, sinks = _check_window(window, sinks)
    with _Launch(stream, dev) as handle:
        need = 0 if workspace is not None else fa_decode_window_workspace_size(
            batch, H, Hkv, d, max_ctx_len, window, sinks, block_size)
        workspace = _workspace(workspace, need, dev, 256, zero=True)
        out, lse = _results(q, (batch, H), out, lse, want_lse)
        if not batch:
            return out, lse
        rc = load_library().fa_decode_paged_window(
            _addr(q), _addr(k_pool), _addr(v_pool), _addr(block_table), block_table.shape[1],
            _addr(ctx_lens), int(max_ctx_len), batch, H, Hkv, d, block_size, num_blocks,
            _scale(scale, d), window, sinks, _addr(out), _addr(lse), _addr(workspace),
            workspace.numel(), handle)
    if rc != FA_OK:
        raise FaError("fa_decode_paged_window", rc)
    return out, lse


def fa_bwd_window_workspace_size(B, H, Hkv, N, d, window, sinks=0) -> int:
    """Bytes of workspace of :func:`fa_bwd_window`, or, with B sequences of at
    most N rows, of :func:`fa_bwd_varlen_window`."""
    window, sinks = _check_window(window, sinks)
    return int(load_library().fa_bwd_window_workspace_size(B, H, Hkv, N, d, window, sinks))


def _check_bwd(q, k, v, out, dout, ndim):
    """Checks the inputs of a windowed backward call (out may be None)."""
    _check_bf16_cuda("q", q, ndim)
    out = dout if out is None else out
    for name, t in (("k", k), ("v", v), ("out", out), ("dout", dout)):
        _check_bf16_cuda(name, t, ndim, q.device)
    if k.shape != (*q.shape[:-2], k.shape[-2], q.shape[-1]) or v.shape != k.shape \
            or out.shape != q.shape or dout.shape != q.shape:
        raise ValueError("out and dout must have the shape of q; k and v its shape with Hkv heads")


def _grads(q, k, v, dq, dk, dv):
    """The gradients' tensors: the caller's, checked, or new ones."""
    torch = _torch()
    grads = []
    for name, g, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if g is None:
            g = torch.empty_like(like)
        else:
            _check_tensor(name, g, like.shape, torch.bfloat16, q.device)
        grads.append(g)
    return grads


def fa_bwd_window(q, k, v, out, lse, dout, window, sinks=0, scale=None, dq=None, dk=None, dv=None,
                  workspace=None, stream=None):
    """Gradient of :func:`fa_fwd_window`.  q, out, dout [B,N,H,d]; k, v
    [B,N,Hkv,d] bf16 CUDA tensors; lse [B,H,N] fp32.  out is not read and may
    be None.  Returns (dq, dk, dv)."""
    short = _calls or _short()
    if short and stream is None:
        done = short.bwd_window(q, k, v, out, lse, dout, window, sinks, scale, dq, dk, dv, workspace)
        if done is not None:
            return done
    _check_bwd(q, k, v, out, dout, 4)
    window, sinks = _check_window(window, sinks)
    dev, (B, N, H, d), Hkv = q.device, q.shape, k.shape[2]
    _check_tensor("lse", lse, (B, H, N), _torch().float32, dev)
    with _Launch(stream, dev) as handle:
        dq, dk, dv = _grads(q, k, v, dq, dk, dv)
        if not B * N:
            return dq, dk, dv
        need = 0 if workspace is not None else fa_bwd_window_workspace_size(
            B, H, Hkv, N, d, window, sinks)
        workspace = _workspace(workspace, need, dev)
        rc = load_library().fa_bwd_window(
            _addr(q), _addr(k), _addr(v), _addr(out), _addr(lse), _addr(dout), _addr(dq), _addr(dk),
            _addr(dv), B, H, Hkv, N, d, _scale(scale, d), window, sinks, _addr(workspace),
            workspace.numel(), handle)
    if rc != FA_OK:
        raise FaError("fa_bwd_window", rc)
    return dq, dk, dv


def fa_bwd_varlen_window(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, window, sinks=0,
                         scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradient of :func:`fa_fwd_varlen_window`.  q, out, dout [T,H,d]; k, v
    [T,Hkv,d] bf16 CUDA tensors; lse [H,T] fp32; cu_seqlens int32 [S+1].  out is
    not read and may be None.  Returns (dq, dk, dv); rows outside every sequence
    are left as they were."""
    short = _calls or _short()
    if short and stream is None:
        done = short.bwd_varlen_window(q, k, v, out, lse, dout, cu_seqlens, max_seqlen, window, sinks,
                                       scale, dq, dk, dv, workspace)
        if done is not None:
            return done
    _check_bwd(q, k, v, out, dout, 3)
    window, sinks = _check_window(window, sinks)
    dev, (T, H, d), Hkv = q.device, q.shape, k.shape[1]
    _check_tensor("lse", lse, (H, T), _torch().float32, dev)
    _check_int32("cu_seqlens", cu_seqlens, dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold num_seqs + 1 offsets")
    S = cu_seqlens.numel() - 1
    with _Launch(stream, dev) as handle:
        dq, dk, dv = _grads(q, k, v, dq, dk, dv)
        if not T:
            return dq, dk, dv
        need = 0 if workspace is not None else fa_bwd_window_workspace_size(
            S, H, Hkv, min(int(max_seqlen), T), d, window, sinks)
        workspace = _workspace(workspace, need, dev)
        rc = load_library().fa_bwd_varlen_window(
            _addr(q), _addr(k), _addr(v), _addr(out), _addr(lse), _addr(dout), _addr(dq), _addr(dk),
            _addr(dv), _addr(cu_seqlens), S, T, int(max_seqlen), H, Hkv, d, _scale(scale, d), window,
            sinks, _addr(workspace), workspace.numel(), handle)
    if rc != FA_OK:
        raise FaError("fa_bwd_varlen_window", rc)
    return dq, dk, dv


# ------------------------------------------------------------ 8-bit KV cache
#
# Pools [num_blocks,16,Hkv,d] of e4m3 codes with one fp32 scale per block and
# KV head (include/fa_kvcache.h).

def _check_cache(k_pool, v_pool, k_scale, v_scale, dev):
    torch = _torch()
    shape = getattr(k_pool, "shape", ())
    if len(shape) != 4 or k_pool.dtype not in (torch.uint8, torch.float8_e4m3fn) \
            or not _are(k_pool.dtype, dev.index, (k_pool, shape), (v_pool, shape)) \
            or not _are(torch.float32, dev.index, (k_scale, shape[::2]), (v_scale, shape[::2])):
        _check_fp8("k_pool", k_pool, 4, dev)
        _check_fp8("v_pool", v_pool, 4, dev)
        if v_pool.shape != k_pool.shape:
            raise ValueError("k_pool and v_pool must have the same shape [num_blocks,16,Hkv,d]")
        num_blocks, _, Hkv, _ = k_pool.shape
        _check_tensor("k_scale", k_scale, (num_blocks, Hkv), torch.float32, dev)
        _check_tensor("v_scale", v_scale, (num_blocks, Hkv), torch.float32, dev)
    return k_pool.shape


def _check_cache_window(window, sinks):
    if int(window) == 0 and int(sinks) == 0:
        return 0, 0
    return _check_window(window, sinks)


def _check_token_rows(name, t, Hkv, d):
    """bf16 rows [T, Hkv, d] whose tokens may lie apart (a view of a fused
    projection); returns the token stride in elements."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor")
    if t.dim() != 3 or t.shape[1:] != (Hkv, d) or (t.numel() and t.stride()[1:] != (d, 1)):
        raise ValueError(f"{name} must be [T, {Hkv}, {d}] with the heads of a token dense")
    stride = t.stride(0) if t.shape[0] > 1 else Hkv * d
    if stride < Hkv * d or stride % 8:
        raise ValueError(f"{name}: tokens must lie a multiple of 8 elements apart, not overlapping")
    return stride


def fa_cache_append_fp8(k, v, k_pool, v_pool, k_scale, v_scale, block_table, ctx_lens, cu_seqlens,
                        max_new, stream=None):
    """Quantise new keys and values and write them into an 8-bit cache.

    k, v [T,Hkv,d] bf16 (tokens may lie apart: views of a fused projection);
    pools [num_blocks,16,Hkv,d] uint8/e4m3 and scales [num_blocks,Hkv] fp32,
    written in place; block_table int32 [batch,max_blocks]; ctx_lens int32
    [batch], the new tokens counted; cu_seqlens int32 [batch+1]: sequence b's
    new tokens; max_new bounds their number per sequence.  Returns None.
    """
    short = _calls or _short()
    if short and stream is None:
        done = short.cache_append_fp8(k_pool, v_pool, k_scale, v_scale, k, v, block_table, ctx_lens,
                                      cu_seqlens, max_new)
        if done is not None:
            return
    torch = _torch()
    if not isinstance(k, torch.Tensor) or not k.is_cuda:
        raise ValueError("k must be a CUDA tensor")
    dev = k.device
    num_blocks, block_size, Hkv, d = _check_cache(k_pool, v_pool, k_scale, v_scale, dev)
    k_stride = _check_token_rows("k", k, Hkv, d)
    v_stride = _check_token_rows("v", v, Hkv, d)
    if v.shape[0] != k.shape[0] or v.device != dev:
        raise ValueError("k and v must have the same tokens on one device")
    batch = _check_sequences(block_table, ctx_lens, cu_seqlens, "cu_seqlens", dev)
    if not k.shape[0]:
        return
    with _Launch(stream, dev) as handle:
        rc = load_library().fa_cache_append_fp8(
            _addr(k), _addr(v), k_stride, v_stride, _addr(k_pool), _addr(v_pool), _addr(k_scale),
            _addr(v_scale), _addr(block_table), block_table.shape[1], _addr(ctx_lens),
            _addr(cu_seqlens), batch, k.shape[0], int(max_new), Hkv, d, block_size, num_blocks,
            handle)
    if rc != FA_OK:
        raise FaError("fa_cache_append_fp8", rc)


def fa_decode_paged_fp8(q, k_pool, v_pool, k_scale, v_scale, block_table, ctx_lens, max_ctx_len,
                        window=0, sinks=0, scale=None, out=None, lse=None, workspace=None,
                        want_lse=True, stream=None):
    """Paged GQA flash-decoding over an 8-bit cache, every key (window 0) or
    the last ``window`` and the first ``sinks``.

    q [batch,H,d] bf16; pools and scales as in :func:`fa_cache_append_fp8`.
    Returns (out [batch,H,d] bf16, lse [batch,H] fp32 or None).
    """
    short = _calls or _short()
    if short and stream is None:
        done = short.decode_paged_fp8(k_pool, v_pool, k_scale, v_scale, q, block_table, ctx_lens,
                                      max_ctx_len, window, sinks, scale, want_lse, out, lse, workspace)
        if done is not None:
            return done
    _check_bf16_cuda("q", q, 3)
    dev = q.device
    num_blocks, block_size, Hkv, dp = _check_cache(k_pool, v_pool, k_scale, v_scale, dev)
    batch, H, d = q.shape
    if dp != d:
        raise ValueError("the pools' head size must match q")
    _check_table(block_table, ctx_lens, batch, dev)
    window, sinks = _check_cache_window(window, sinks)
    with _Launch(stream, dev) as handle:
        need = 0
        if workspace is None:
            need = fa_decode_window_workspace_size(batch, H, Hkv, d, max_ctx_len, window, sinks,
                                                   block_size)
        workspace = _workspace(workspace, need, dev, 256, zero=True)
        out, lse = _results(q, (batch, H), out, lse, want_lse)
        if not batch:
            return out, lse
        rc = load_library().fa_decode_paged_fp8(
            _addr(q), _addr(k_pool), _addr(v_pool), _addr(k_scale), _addr(v_scale), _addr(block_table),
            block_table.shape[1], _addr(ctx_lens), int(max_ctx_len), batch, H, Hkv, d, block_size,
            num_blocks, _scale(scale, d), window, sinks, _addr(out), _addr(lse), _addr(workspace),
            workspace.numel(), handle)
    if rc != FA_OK:
        raise FaError("fa_decode_paged_fp8", rc)
    return out, lse


def fa_fwd_paged_fp8(q, k_pool, v_pool, k_scale, v_scale, block_table, ctx_lens, cu_seqlens_q,
                     max_seqlen_q, max_ctx_len, window=0, sinks=0, scale=None, out=None, lse=None,
                     want_lse=True, stream=None):
    """Query chunks [Tq,H,d] (causal) against an 8-bit cache, every key up to
    each query's own (window 0) or the last ``window`` and the first ``sinks``.

    Pools and scales as in :func:`fa_cache_append_fp8`; ctx_lens int32 [batch]
    and cu_seqlens_q int32 [batch+1] as in :func:`fa_fwd_paged`.
    Returns (out [Tq,H,d] bf16, lse [H,Tq] fp32 or None).
    """
    short = _calls or _short()
    if short and stream is None:
        done = short.fwd_paged_fp8(k_pool, v_pool, k_scale, v_scale, q, block_table, ctx_lens,
                                   cu_seqlens_q, max_seqlen_q, max_ctx_len, window, sinks, scale,
                                   want_lse, out, lse)
        if done is not None:
            return done
    _check_bf16_cuda("q", q, 3)
    dev = q.device
    num_blocks, block_size, Hkv, dp = _check_cache(k_pool, v_pool, k_scale, v_scale, dev)
    batch = _check_sequences(block_table, ctx_lens, cu_seqlens_q, "cu_seqlens_q", dev)
    window, sinks = _check_cache_window(window, sinks)
    Tq, H, d = q.shape
    if dp != d:
        raise ValueError("the pools' head size must match q")
    with _Launch(stream, dev) as handle:
        out, lse = _results(q, (H, Tq), out, lse, want_lse)
        if not Tq:
            return out, lse
        rc = load_library().fa_fwd_paged_fp8(
            _addr(q), _addr(k_pool), _addr(v_pool), _addr(k_scale), _addr(v_scale), _addr(block_table),
            block_table.shape[1], _addr(ctx_lens), _addr(cu_seqlens_q), batch, Tq,
            int(max_seqlen_q), int(max_ctx_len), H, Hkv, d, block_size, num_blocks,
            _scale(scale, d), window, sinks, _addr(out), _addr(lse), handle)
    if rc != FA_OK:
        raise FaError("fa_fwd_paged_fp8", rc)
    return out, lse
