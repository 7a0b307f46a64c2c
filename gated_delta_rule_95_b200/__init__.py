"""Gated DeltaNet-2 token mixer for NVIDIA B200 (sm_100a).

Python binding of ``libgdn2.so`` (the C ABI declared in ``include/gdn2.h``).
It only marshals arguments: every step of the computation runs in the
library's CUDA kernels.  PyTorch provides device memory and streams.  There is
no CPU fallback: without the built library every call raises.

    o, S_T = gdn2_chunk_fwd(q, k, v, log_alpha, b, w, S0=None)   # prefill, C = 64
    o      = gdn2_decode_step(q, k, v, log_alpha, b, w, S)       # S updated in place

Shapes: prefill tokens [B, T, H, D], decode tokens [B, H, D], states
[B, H, d_k, d_v] float32; q, k, v, b, w in bfloat16 or float32 (one dtype);
log_alpha float32 (log of the channel-wise decay, <= 0); o is always float32.

Around the mixer: the short convolution and its gradients (gdn2_short_conv, gdn2_short_conv_bwd),
the gated delta rule with scalar gates (gdn2_gdr_chunk_fwd, gdn2_gdr_decode_step; o in the
inputs' dtype) and the layer norm over the residual sum (gdn2_layer_norm_fwd, gdn2_layer_norm_bwd).
Their inputs are contiguous CUDA tensors of one device; outputs and workspaces are allocated
when not given, on the stream that the call runs on (stream: a torch stream or a raw handle).

Sizes are the library's 32-bit ints: rows, tokens or columns past 2^31 - 1 raise ValueError.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = ["gdn2_chunk_fwd", "gdn2_chunk_fwd_csize", "gdn2_chunk_bwd", "gdn2_chunk_fwd_split", "gdn2_chunk_fwd_split_static", "gdn2_chunk_fwd_varlen", "gdn2_chunk_fwd_raw", "gdn2_short_conv", "gdn2_decode_step", "gdn2_decode_step_raw", "gdn2_gdr_chunk_fwd", "gdn2_gdr_decode_step", "gdn2_layer_norm_fwd", "gdn2_layer_norm_bwd", "gdn2_short_conv_bwd", "gdn2_device_status", "GDN2Error", "library_path", "lib"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

GDN2_F32, GDN2_BF16 = 0, 1
_DT = {torch.float32: GDN2_F32, torch.bfloat16: GDN2_BF16}


class GDN2Error(RuntimeError):
    """A gdn2_* call returned a non-zero status."""

    def __init__(self, fn, status):
        msg = lib().gdn2_status_string(status).decode()
        if status == 5:
            msg += " (" + lib().gdn2_last_cuda_error().decode() + ")"
        super().__init__(f"{fn}: status {status}: {msg}")
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, "libgdn2.so")


def lib(path=None):
    """The loaded C library (ctypes).  Raises if it has not been built.  ``path`` loads
    another build of the same library in its place (the instrumented build of the
    profiling driver)."""
    global _LIB
    if path is not None and (_LIB is None or _LIB._name != path):
        _LIB = None
    if _LIB is None:
        path = path or library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m gated_delta_rule_95_b200.build` "
                               "(or __graft_entry__.build()); there is no fallback path")
        L = ctypes.CDLL(path)
        P, I = ctypes.c_void_p, ctypes.c_int
        L.gdn2_chunk_fwd.argtypes = [P] * 9 + [I] * 6 + [P]
        L.gdn2_chunk_fwd.restype = I
        L.gdn2_chunk_bwd.argtypes = [P] * 16 + [I] * 6 + [P, ctypes.c_size_t, P]
        L.gdn2_chunk_bwd.restype = I
        L.gdn2_chunk_bwd_workspace_bytes.argtypes = [I] * 5
        L.gdn2_chunk_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn2_chunk_fwd_split.argtypes = [P] * 9 + [I] * 7 + [P, ctypes.c_size_t, P]
        L.gdn2_chunk_fwd_split.restype = I
        L.gdn2_chunk_fwd_split_static.argtypes = [P] * 9 + [I] * 7 + [P]
        L.gdn2_chunk_fwd_split_static.restype = I
        L.gdn2_chunk_fwd_split_segments.argtypes = [I] * 4
        L.gdn2_chunk_fwd_split_segments.restype = I
        L.gdn2_chunk_fwd_split_workspace_bytes.argtypes = [I] * 5
        L.gdn2_chunk_fwd_split_workspace_bytes.restype = ctypes.c_size_t
        L.gdn2_chunk_fwd_csize.argtypes = [P] * 9 + [I] * 7 + [P]
        L.gdn2_chunk_fwd_csize.restype = I
        L.gdn2_chunk_fwd_csize_smem_bytes.argtypes = [I] * 2
        L.gdn2_chunk_fwd_csize_smem_bytes.restype = ctypes.c_size_t
        L.gdn2_chunk_fwd_varlen.argtypes = [P] * 10 + [I] * 6 + [P]
        L.gdn2_chunk_fwd_varlen.restype = I
        L.gdn2_chunk_fwd_raw.argtypes = [P] * 11 + [I] * 6 + [P]
        L.gdn2_chunk_fwd_raw.restype = I
        L.gdn2_short_conv.argtypes = [P] * 7 + [I] * 4 + [P]
        L.gdn2_short_conv.restype = I
        L.gdn2_decode_step.argtypes = [P] * 8 + [I] * 5 + [P]
        L.gdn2_decode_step.restype = I
        L.gdn2_decode_step_raw.argtypes = [P] * 9 + [I] * 5 + [P]
        L.gdn2_decode_step_raw.restype = I
        L.gdn2_short_conv_bwd.argtypes = [P] * 10 + [I] * 4 + [P, ctypes.c_size_t, P]
        L.gdn2_short_conv_bwd.restype = I
        L.gdn2_short_conv_bwd_workspace_bytes.argtypes = [I] * 2
        L.gdn2_short_conv_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn2_layer_norm_fwd.argtypes = [P] * 8 + [I] * 2 + [ctypes.c_float, I, P]
        L.gdn2_layer_norm_fwd.restype = I
        L.gdn2_layer_norm_bwd.argtypes = [P] * 9 + [I] * 3 + [P, ctypes.c_size_t, P]
        L.gdn2_layer_norm_bwd.restype = I
        L.gdn2_layer_norm_bwd_workspace_bytes.argtypes = [I] * 2
        L.gdn2_layer_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn2_gdr_chunk_fwd.argtypes = [P] * 9 + [I] * 6 + [ctypes.c_float, I, P, ctypes.c_size_t, P]
        L.gdn2_gdr_chunk_fwd_workspace_bytes.argtypes = [I] * 7
        L.gdn2_gdr_chunk_fwd_workspace_bytes.restype = ctypes.c_size_t
        L.gdn2_gdr_chunk_fwd.restype = I
        L.gdn2_gdr_decode_step.argtypes = [P] * 8 + [I] * 5 + [ctypes.c_float, I, P]
        L.gdn2_gdr_decode_step.restype = I
        L.gdn2_device_status.argtypes = []
        L.gdn2_device_status.restype = I
        L.gdn2_status_string.argtypes = [I]
        L.gdn2_status_string.restype = ctypes.c_char_p
        L.gdn2_last_cuda_error.argtypes = []
        L.gdn2_last_cuda_error.restype = ctypes.c_char_p
        L.gdn2_version.argtypes = []
        L.gdn2_version.restype = I
        for name, fn in vars(L).items():  # where an entry point's sizes are: the run of ints after its pointers
            if name.startswith("gdn2_") and P in (fn.argtypes or ()) and I in fn.argtypes:
                at = fn.argtypes.index(I)
                fn.sizes = slice(at, next(i for i in range(at, len(fn.argtypes)) if fn.argtypes[i] is not I))
        _LIB = L
    return _LIB


def _check_sizes(fn, args):
    """Raises for a size that the library's ints do not hold (they would keep its low 32 bits)."""
    if max(args[fn.sizes]) > 0x7FFFFFFF:
        raise ValueError(f"{fn.__name__}: a size of {max(args[fn.sizes])} is past 2^31 - 1")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev, stream):
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on(device, fn, *args):
    """Calls ``fn`` with ``device`` current (the library keys its per-device state, the
    error word, scratch address and kernel attributes, by the current device)."""
    _check_sizes(fn, args)
    with torch.cuda.device(device):
        return fn(*args)


def _check_tokens(name, tensors, dtype, device):
    for n, t in tensors.items():
        if not t.is_cuda or t.device != device:
            raise ValueError(f"{name}: {n} must be a CUDA tensor on {device}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: {n} must be contiguous")
        want = torch.float32 if n in ("log_alpha", "a_raw", "S0", "S", "S_T", "o", "decay_scale", "weight",
                                      "bias") else dtype
        if t.dtype != want:
            raise ValueError(f"{name}: {n} must be {want}, got {t.dtype}")


def gdn2_chunk_fwd(q, k, v, log_alpha, b, w, S0=None, *, o=None, S_T=None, want_state=True, stream=None):
    """Chunkwise prefill forward.  Returns (o [B,T,H,d_v], S_T [B,H,d_k,d_v] or None)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DT:
        raise ValueError(f"gdn2_chunk_fwd: unsupported dtype {q.dtype}")
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ts = dict(q=q, k=k, v=v, log_alpha=log_alpha, b=b, w=w, o=o)
    if S0 is not None:
        ts["S0"] = S0
    if S_T is not None:
        ts["S_T"] = S_T
    _check_tokens("gdn2_chunk_fwd", ts, q.dtype, q.device)
    rc = _on(q.device, lib().gdn2_chunk_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(o),
                              _ptr(S_T), B, T, H, dk, dv, _DT[q.dtype], _stream(q.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_chunk_fwd", rc)
    return o, S_T


def gdn2_chunk_fwd_csize(q, k, v, log_alpha, b, w, S0=None, *, chunk=64, o=None, S_T=None, want_state=True,
                         stream=None):
    """Chunkwise prefill forward at chunk size 32, 64 or 128 (bf16 inputs).  Returns
    (o [B,T,H,d_v], S_T [B,H,d_k,d_v] or None), like gdn2_chunk_fwd."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DT:
        raise ValueError(f"gdn2_chunk_fwd_csize: unsupported dtype {q.dtype}")
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ts = dict(q=q, k=k, v=v, log_alpha=log_alpha, b=b, w=w, o=o)
    if S0 is not None:
        ts["S0"] = S0
    if S_T is not None:
        ts["S_T"] = S_T
    _check_tokens("gdn2_chunk_fwd_csize", ts, q.dtype, q.device)
    rc = _on(q.device, lib().gdn2_chunk_fwd_csize, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0),
                                    _ptr(o), _ptr(S_T), B, T, H, dk, dv, _DT[q.dtype], int(chunk),
                                    _stream(q.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_chunk_fwd_csize", rc)
    return o, S_T


def gdn2_chunk_bwd(q, k, v, log_alpha, b, w, S0, dO, dS_T=None, *, workspace=None, want_dS0=True, out=None,
                   stream=None):
    """Backward of gdn2_chunk_fwd: gradients of L given dO = dL/do [B,T,H,d_v] fp32 and
    dS_T = dL/dS_T (or None).  Returns dict(dq, dk, dv, dlog_alpha, db, dw: fp32 like the
    inputs; dS0 [B,H,d_k,d_v] or None).  workspace (uint8 CUDA tensor of at least
    gdn2_chunk_bwd_workspace_bytes) is allocated when not given."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DT:
        raise ValueError(f"gdn2_chunk_bwd: unsupported dtype {q.dtype}")
    L = lib()
    need = L.gdn2_chunk_bwd_workspace_bytes(B, T, H, dk, dv)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    g = out if out is not None else dict(
        dq=torch.empty((B, T, H, dk), **f32), dk=torch.empty((B, T, H, dk), **f32),
        dv=torch.empty((B, T, H, dv), **f32), dlog_alpha=torch.empty((B, T, H, dk), **f32),
        db=torch.empty((B, T, H, dk), **f32), dw=torch.empty((B, T, H, dv), **f32),
        dS0=torch.empty((B, H, dk, dv), **f32) if want_dS0 else None)
    ts = dict(q=q, k=k, v=v, log_alpha=log_alpha, b=b, w=w, o=dO)
    for n, t in (("S0", S0), ("S_T", dS_T)):
        if t is not None:
            ts[n] = t
    _check_tokens("gdn2_chunk_bwd", ts, q.dtype, q.device)
    for n, t in g.items():
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or t.device != q.device):
            raise ValueError(f"gdn2_chunk_bwd: {n} must be a contiguous fp32 tensor on {q.device}")
    rc = _on(q.device, L.gdn2_chunk_bwd, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(dO),
                          _ptr(dS_T), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_alpha"]),
                          _ptr(g["db"]), _ptr(g["dw"]), _ptr(g["dS0"]), B, T, H, dk, dv, _DT[q.dtype],
                          _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(q.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_chunk_bwd", rc)
    return g


def gdn2_chunk_fwd_split(q, k, v, log_alpha, b, w, S0=None, *, segments=None, workspace=None, o=None, S_T=None,
                         want_state=True, stream=None):
    """Chunkwise prefill forward with each sequence split into ``segments`` parallel segments
    (bf16, d_k = d_v).  segments=None takes the library's choice for this device's SM count;
    workspace (a uint8 CUDA tensor of at least gdn2_chunk_fwd_split_workspace_bytes) is
    allocated when not given.  Returns (o [B,T,H,d_v], S_T [B,H,d_k,d_v] or None)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype != torch.bfloat16:
        raise ValueError("gdn2_chunk_fwd_split: bf16 inputs only")
    L = lib()
    if segments is None:
        sms = torch.cuda.get_device_properties(q.device).multi_processor_count
        segments = L.gdn2_chunk_fwd_split_segments(B, T, H, sms)
    need = L.gdn2_chunk_fwd_split_workspace_bytes(B, H, dk, dv, segments)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ts = dict(q=q, k=k, v=v, log_alpha=log_alpha, b=b, w=w, o=o)
    if S0 is not None:
        ts["S0"] = S0
    if S_T is not None:
        ts["S_T"] = S_T
    _check_tokens("gdn2_chunk_fwd_split", ts, q.dtype, q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _on(q.device, L.gdn2_chunk_fwd_split, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(o),
                                _ptr(S_T), B, T, H, dk, dv, _DT[q.dtype], segments, _ptr(workspace), wbytes,
                                _stream(q.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_chunk_fwd_split", rc)
    return o, S_T


def gdn2_chunk_fwd_split_static(q, k, v, log_alpha, b, w, S0=None, *, segments, o=None, S_T=None, want_state=True,
                                stream=None):
    """gdn2_chunk_fwd_split with the library's fixed 16 MiB device scratch instead of a
    workspace (the call allocates nothing when o and S_T are given)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype != torch.bfloat16:
        raise ValueError("gdn2_chunk_fwd_split_static: bf16 inputs only")
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ts = dict(q=q, k=k, v=v, log_alpha=log_alpha, b=b, w=w, o=o)
    if S0 is not None:
        ts["S0"] = S0
    if S_T is not None:
        ts["S_T"] = S_T
    _check_tokens("gdn2_chunk_fwd_split_static", ts, q.dtype, q.device)
    rc = _on(q.device, lib().gdn2_chunk_fwd_split_static, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0),
                                           _ptr(o), _ptr(S_T), B, T, H, dk, dv, _DT[q.dtype], segments,
                                           _stream(q.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_chunk_fwd_split_static", rc)
    return o, S_T


def gdn2_chunk_fwd_varlen(q, k, v, log_alpha, b, w, cu_seqlens, S0=None, *, o=None, S_T=None, want_state=True,
                          stream=None):
    """Chunkwise prefill forward over packed variable-length sequences.

    q, k, b: [T, H, d_k]; v, w: [T, H, d_v]; log_alpha: [T, H, d_k]; cu_seqlens: int32 [N + 1]
    on the device.  Returns (o [T, H, d_v], S_T [N, H, d_k, d_v] or None)."""
    T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype != torch.bfloat16:
        raise ValueError("gdn2_chunk_fwd_varlen: bf16 inputs only")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
        raise ValueError("gdn2_chunk_fwd_varlen: cu_seqlens must be a contiguous int32 vector")
    if cu_seqlens.device != q.device:
        raise ValueError("gdn2_chunk_fwd_varlen: cu_seqlens must be on the inputs' device")
    N = cu_seqlens.numel() - 1
    if o is None:
        o = torch.empty((T, H, dv), dtype=torch.float32, device=q.device)
    if S_T is None and want_state:
        S_T = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    ts = dict(q=q, k=k, v=v, log_alpha=log_alpha, b=b, w=w, o=o)
    if S0 is not None:
        ts["S0"] = S0
    if S_T is not None:
        ts["S_T"] = S_T
    _check_tokens("gdn2_chunk_fwd_varlen", ts, q.dtype, q.device)
    rc = _on(q.device, lib().gdn2_chunk_fwd_varlen, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(cu_seqlens),
                                     _ptr(S0), _ptr(o), _ptr(S_T), N, T, H, dk, dv, _DT[q.dtype],
                                     _stream(q.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_chunk_fwd_varlen", rc)
    return o, S_T


def gdn2_chunk_fwd_raw(q_raw, k_raw, v, a_raw, b_raw, w_raw, S0=None, *, decay_scale=None, cu_seqlens=None,
                       o=None, S_T=None, want_state=True, stream=None):
    """Chunkwise prefill forward on the raw projections (q, k normalised, sigmoid gates and
    log alpha = -decay_scale[h] * softplus(a_raw) inside the kernel).

    Without cu_seqlens: q_raw, k_raw, b_raw [B, T, H, d_k], v, w_raw [B, T, H, d_v], a_raw fp32
    [B, T, H, d_k]; returns (o [B, T, H, d_v], S_T [B, H, d_k, d_v] or None).  With cu_seqlens
    (int32 [N + 1] on the device) the tensors are packed, [T, H, D], and S0 / S_T are
    [N, H, d_k, d_v].  decay_scale: fp32 [H] on the device, or None for 1."""
    if q_raw.dtype != torch.bfloat16:
        raise ValueError("gdn2_chunk_fwd_raw: bf16 inputs only")
    if cu_seqlens is None:
        B, T, H, dk = q_raw.shape
        o_shape = (B, T, H, v.shape[-1])
    else:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
            raise ValueError("gdn2_chunk_fwd_raw: cu_seqlens must be a contiguous int32 vector")
        if cu_seqlens.device != q_raw.device:
            raise ValueError("gdn2_chunk_fwd_raw: cu_seqlens must be on the inputs' device")
        T, H, dk = q_raw.shape
        B = cu_seqlens.numel() - 1
        o_shape = (T, H, v.shape[-1])
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(o_shape, dtype=torch.float32, device=q_raw.device)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q_raw.device)
    ts = dict(q_raw=q_raw, k_raw=k_raw, v=v, a_raw=a_raw, b_raw=b_raw, w_raw=w_raw, o=o)
    for n, t in (("S0", S0), ("S_T", S_T), ("decay_scale", decay_scale)):
        if t is not None:
            ts[n] = t
    if decay_scale is not None and decay_scale.numel() != H:
        raise ValueError("gdn2_chunk_fwd_raw: decay_scale must hold one value per head")
    _check_tokens("gdn2_chunk_fwd_raw", ts, q_raw.dtype, q_raw.device)
    rc = _on(q_raw.device, lib().gdn2_chunk_fwd_raw, _ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(a_raw), _ptr(b_raw), _ptr(w_raw),
                                  _ptr(decay_scale), _ptr(cu_seqlens), _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, dk,
                                  dv, _DT[q_raw.dtype], _stream(q_raw.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_chunk_fwd_raw", rc)
    return o, S_T


def gdn2_short_conv(x, weight, bias=None, *, cu_seqlens=None, hist=None, y=None, hist_out=None, want_hist=False,
                    stream=None):
    """Short causal depthwise convolution (4 taps) over the token axis.

    x: [B, T, C] (or packed [T, C] with cu_seqlens int32 [N + 1] on the device); weight fp32
    [C, 4] (or [C, 1, 4]); bias fp32 [C] or None; hist: [B, 3, C] carried history or None.
    Returns (y like x, hist_out [B, 3, C] or None); hist_out may be hist (in-place update)."""
    if x.dtype not in _DT:
        raise ValueError(f"gdn2_short_conv: unsupported dtype {x.dtype}")
    if cu_seqlens is None:
        B, T, C = x.shape
    else:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
            raise ValueError("gdn2_short_conv: cu_seqlens must be a contiguous int32 vector")
        if cu_seqlens.device != x.device:
            raise ValueError("gdn2_short_conv: cu_seqlens must be on the inputs' device")
        T, C = x.shape
        B = cu_seqlens.numel() - 1
    if weight.numel() != 4 * C:
        raise ValueError("gdn2_short_conv: weight must hold 4 taps per channel")
    if y is None:
        y = torch.empty_like(x)
    if hist_out is None and want_hist:
        hist_out = torch.empty((B, 3, C), dtype=x.dtype, device=x.device)
    ts = dict(x=x, weight=weight, y=y)
    for n, t in (("bias", bias), ("hist", hist), ("hist_out", hist_out)):
        if t is not None:
            ts[n] = t
    _check_tokens("gdn2_short_conv", ts, x.dtype, x.device)
    rc = _on(x.device, lib().gdn2_short_conv, _ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens), _ptr(hist), _ptr(y),
                               _ptr(hist_out), B, T, C, _DT[x.dtype], _stream(x.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_short_conv", rc)
    return y, hist_out


def gdn2_decode_step(q, k, v, log_alpha, b, w, S, *, o=None, stream=None):
    """One decode step; S [B,H,d_k,d_v] fp32 is updated in place.  Returns o [B,H,d_v]."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DT:
        raise ValueError(f"gdn2_decode_step: unsupported dtype {q.dtype}")
    if o is None:
        o = torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
    _check_tokens("gdn2_decode_step", dict(q=q, k=k, v=v, log_alpha=log_alpha, b=b, w=w, S=S, o=o), q.dtype,
                  q.device)
    rc = _on(q.device, lib().gdn2_decode_step, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S), _ptr(o),
                                B, H, dk, dv, _DT[q.dtype], _stream(q.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_decode_step", rc)
    return o


def gdn2_decode_step_raw(q_raw, k_raw, v, a_raw, b_raw, w_raw, S, *, decay_scale=None, o=None, stream=None):
    """One decode step on the raw projections (q, k normalised, sigmoid gates, log alpha =
    -decay_scale[h] * softplus(a_raw) inside the step); S [B,H,d_k,d_v] fp32 is updated in
    place.  Returns o [B,H,d_v]."""
    B, H, dk = q_raw.shape
    dv = v.shape[-1]
    if q_raw.dtype not in _DT:
        raise ValueError(f"gdn2_decode_step_raw: unsupported dtype {q_raw.dtype}")
    if decay_scale is not None and decay_scale.numel() != H:
        raise ValueError("gdn2_decode_step_raw: decay_scale must hold one value per head")
    if o is None:
        o = torch.empty((B, H, dv), dtype=torch.float32, device=q_raw.device)
    ts = dict(q_raw=q_raw, k_raw=k_raw, v=v, a_raw=a_raw, b_raw=b_raw, w_raw=w_raw, S=S, o=o)
    if decay_scale is not None:
        ts["decay_scale"] = decay_scale
    _check_tokens("gdn2_decode_step_raw", ts, q_raw.dtype, q_raw.device)
    rc = _on(q_raw.device, lib().gdn2_decode_step_raw, _ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(a_raw), _ptr(b_raw), _ptr(w_raw),
                                    _ptr(decay_scale), _ptr(S), _ptr(o), B, H, dk, dv, _DT[q_raw.dtype],
                                    _stream(q_raw.device, stream))
    if rc != 0:
        raise GDN2Error("gdn2_decode_step_raw", rc)
    return o


def _need(fn, name, t, dtype, shape, dev):
    """Raises unless ``t`` is a contiguous tensor on ``dev`` (a CUDA device) of that dtype and shape."""
    if t.dtype is dtype and t.device == dev and t.shape == shape and t.is_contiguous():
        return
    if t.device != dev:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor on {dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} must be of shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{fn}: {name} must be contiguous")


def _adr(t):
    return None if t is None else t.data_ptr()


def _call(fn, dev, *args):
    """Calls the library's ``fn`` with ``args`` and the current stream, the tensors' device current, and
    raises on a status.  (The raw stream handle, and no device switch where none is needed: a
    small kernel's call costs the host more than the GPU.)"""
    f = getattr(lib(), fn)
    _check_sizes(f, args)
    handle = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch._C._cuda_getDevice() == dev.index:
        rc = f(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, handle)
    if rc != 0:
        raise GDN2Error(fn, rc)


def _elsewhere(stream, dev):
    """A given stream as the current one: what a call allocates belongs to the stream that it runs on, and
    is not handed out again before the call is done there."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = getattr(stream, "cuda_stream", stream)  # (0, the default stream, would make a new ExternalStream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"the stream is of {stream.device}, the tensors are on {dev}")
    return torch.cuda.stream(stream)


def _dtype_of(fn, name, t, dims, what):
    """The library's code of t's dtype, its number of axes checked."""
    if t.dim() not in dims:
        raise ValueError(f"{fn}: {name} must be {what}")
    if t.dtype not in _DT:
        raise ValueError(f"{fn}: unsupported dtype {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor")
    return _DT[t.dtype]


def _offsets(fn, cu_seqlens, dev):
    """Number of packed sequences."""
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError(f"{fn}: cu_seqlens must be a vector of N + 1 offsets")
    _need(fn, "cu_seqlens", cu_seqlens, torch.int32, cu_seqlens.shape, dev)
    return cu_seqlens.shape[0] - 1


def _workspace(fn, workspace, need, dev, like):
    """The caller's workspace, checked, or a new one of ``need`` bytes, on the device of ``like`` (fp32)."""
    if workspace is None:
        return like.new_empty((max(need, 16) + 3) // 4)
    if not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be a contiguous CUDA tensor on {dev}")
    return workspace


def gdn2_short_conv_bwd(dy, x, weight, *, cu_seqlens=None, hist=None, dhist_out=None, want_dbias=True, want_dhist=None,
                        workspace=None, out=None, stream=None):
    """Backward of gdn2_short_conv: dy, x [B, T, C] (packed [T, C] with cu_seqlens int32 [N + 1]
    on the device), weight fp32 [C, 4] (or [C, 1, 4]), hist the forward's [B, 3, C] or None,
    dhist_out the gradient of its hist_out or None.  Returns dict(dx like x, dweight like
    weight, dbias [C] fp32 or None, dhist [B, 3, C] or None); want_dhist=None asks for dhist
    when hist is given.  workspace (uint8, gdn2_short_conv_bwd_workspace_bytes) is allocated
    when not given, and so are the gradients (out: such a dict)."""
    if stream is not None:
        with _elsewhere(stream, x.device):
            return gdn2_short_conv_bwd(dy, x, weight, cu_seqlens=cu_seqlens, hist=hist, dhist_out=dhist_out,
                                       want_dbias=want_dbias, want_dhist=want_dhist, workspace=workspace, out=out)
    fn, f32 = "gdn2_short_conv_bwd", torch.float32
    packed = cu_seqlens is not None
    dt = _dtype_of(fn, "x", x, (2,) if packed else (3,), "[B, T, C], or packed [T, C] with cu_seqlens")
    dev, C = x.device, x.shape[-1]
    if packed:
        B, T = _offsets(fn, cu_seqlens, dev), x.shape[0]
        tokens = T
    else:
        B, T, _ = x.shape
        tokens = B * T
    if weight.shape != (C, 4) and weight.shape != (C, 1, 4):
        raise ValueError(f"{fn}: weight must hold 4 taps per channel")
    h = (B, 3, C)
    _need(fn, "x", x, x.dtype, x.shape, dev)
    _need(fn, "dy", dy, x.dtype, x.shape, dev)
    _need(fn, "weight", weight, f32, weight.shape, dev)
    if hist is not None:
        _need(fn, "hist", hist, x.dtype, h, dev)
    if dhist_out is not None:
        _need(fn, "dhist_out", dhist_out, x.dtype, h, dev)
    if out is None:
        if want_dhist is None:
            want_dhist = hist is not None
        out = dict(dx=torch.empty_like(x), dweight=torch.empty_like(weight),
                   dbias=weight.new_empty((C,)) if want_dbias else None,
                   dhist=x.new_empty(h) if want_dhist else None)
    else:
        _need(fn, "dx", out["dx"], x.dtype, x.shape, dev)
        _need(fn, "dweight", out["dweight"], f32, weight.shape, dev)
        if out.get("dbias") is not None:
            _need(fn, "dbias", out["dbias"], f32, (C,), dev)
        if out.get("dhist") is not None:
            _need(fn, "dhist", out["dhist"], x.dtype, h, dev)
    workspace = _workspace(fn, workspace, lib().gdn2_short_conv_bwd_workspace_bytes(tokens, C), dev, weight)
    _call(fn, dev, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), _adr(cu_seqlens), _adr(hist), _adr(dhist_out),
          out["dx"].data_ptr(), out["dweight"].data_ptr(), _adr(out.get("dbias")), _adr(out.get("dhist")), B, T, C, dt,
          workspace.data_ptr(), workspace.nbytes)
    return out


def gdn2_layer_norm_fwd(x, weight, bias=None, residual=None, *, eps=1e-5, y=None, sum_out=None, want_stats=True,
                        stream=None):
    """Layer norm of s = x + residual (rounded to x's dtype; s = x without one) over the last
    axis: x, residual [..., cols], weight, bias fp32 [cols].  Returns (y like x, s or None
    without a residual, mean [...] fp32, rstd [...] fp32); the statistics are None with
    want_stats=False.  sum_out may be x or residual (updated in place)."""
    if stream is not None:
        with _elsewhere(stream, x.device):
            return gdn2_layer_norm_fwd(x, weight, bias, residual, eps=eps, y=y, sum_out=sum_out, want_stats=want_stats)
    fn, f32 = "gdn2_layer_norm_fwd", torch.float32
    dt = _dtype_of(fn, "x", x, range(1, 65), "[..., cols]")
    dev, shape, dtype = x.device, x.shape, x.dtype
    cols = shape[-1]
    if cols == 0:
        raise ValueError(f"{fn}: a row of x has no columns")
    rows = x.numel() // cols
    _need(fn, "x", x, dtype, shape, dev)
    _need(fn, "weight", weight, f32, (cols,), dev)
    if bias is not None:
        _need(fn, "bias", bias, f32, (cols,), dev)
    if residual is not None:
        _need(fn, "residual", residual, dtype, shape, dev)
        if sum_out is None:
            sum_out = torch.empty_like(x)
        else:
            _need(fn, "sum_out", sum_out, dtype, shape, dev)
    elif sum_out is not None:
        raise ValueError(f"{fn}: sum_out needs a residual")
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(fn, "y", y, dtype, shape, dev)
    mean = rstd = None
    if want_stats:
        mean = weight.new_empty(shape[:-1])
        rstd = torch.empty_like(mean)
    _call(fn, dev, x.data_ptr(), _adr(residual), weight.data_ptr(), _adr(bias), y.data_ptr(), _adr(sum_out),
          _adr(mean), _adr(rstd), rows, cols, eps, dt)
    return y, sum_out, mean, rstd


def gdn2_layer_norm_bwd(dy, s, weight, mean, rstd, ds=None, *, want_dbias=True, workspace=None, out=None, stream=None):
    """Backward of gdn2_layer_norm_fwd: dy, s, ds [..., cols] (s the forward's sum, or its x), mean
    and rstd the forward's.  Returns dict(dx like s: the gradient of x and of the residual,
    dweight [cols] fp32, dbias [cols] fp32 or None).  workspace (uint8,
    gdn2_layer_norm_bwd_workspace_bytes) is allocated when not given, and so are the gradients
    (out: such a dict)."""
    if stream is not None:
        with _elsewhere(stream, s.device):
            return gdn2_layer_norm_bwd(dy, s, weight, mean, rstd, ds, want_dbias=want_dbias, workspace=workspace, out=out)
    fn, f32 = "gdn2_layer_norm_bwd", torch.float32
    dt = _dtype_of(fn, "s", s, range(1, 65), "[..., cols]")
    dev, shape, dtype = s.device, s.shape, s.dtype
    cols = shape[-1]
    rows = s.numel() // cols if cols else 0
    _need(fn, "s", s, dtype, shape, dev)
    _need(fn, "dy", dy, dtype, shape, dev)
    _need(fn, "weight", weight, f32, (cols,), dev)
    _need(fn, "mean", mean, f32, shape[:-1], dev)
    _need(fn, "rstd", rstd, f32, shape[:-1], dev)
    if ds is not None:
        _need(fn, "ds", ds, dtype, shape, dev)
    if out is None:
        dw = torch.empty_like(weight)
        out = dict(dx=torch.empty_like(s), dweight=dw, dbias=torch.empty_like(dw) if want_dbias else None)
    else:
        _need(fn, "dx", out["dx"], dtype, shape, dev)
        _need(fn, "dweight", out["dweight"], f32, (cols,), dev)
        if out.get("dbias") is not None:
            _need(fn, "dbias", out["dbias"], f32, (cols,), dev)
    workspace = _workspace(fn, workspace, lib().gdn2_layer_norm_bwd_workspace_bytes(rows, cols), dev, weight)
    _call(fn, dev, dy.data_ptr(), s.data_ptr(), weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _adr(ds),
          out["dx"].data_ptr(), out["dweight"].data_ptr(), _adr(out.get("dbias")), rows, cols, dt,
          workspace.data_ptr(), workspace.nbytes)
    return out


def gdn2_gdr_chunk_fwd(q, k, v, g, beta, S0=None, *, scale=1.0, cu_seqlens=None, o=None, S_T=None, want_state=True,
                       workspace=None, stream=None):
    """Chunkwise prefill forward of the gated delta rule with scalar gates:
    S_t = e^g_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T, o_t = scale S_t^T q_t.

    q, k [B, T, H_k, d_k], v [B, T, H_v, d_v] (H_v a multiple of H_k), g, beta fp32 [B, T, H_v]; with
    cu_seqlens (int32 [N + 1] on the device) packed, without the B axis.  Returns (o like v in
    shape and dtype, S_T [B, H_v, d_k, d_v] fp32 or None); S_T may be S0.  workspace (uint8,
    gdn2_gdr_chunk_fwd_workspace_bytes; none for fp32) is allocated when not given."""
    if stream is not None:
        with _elsewhere(stream, q.device):
            return gdn2_gdr_chunk_fwd(q, k, v, g, beta, S0, scale=scale, cu_seqlens=cu_seqlens, o=o, S_T=S_T,
                                      want_state=want_state, workspace=workspace)
    fn, f32 = "gdn2_gdr_chunk_fwd", torch.float32
    packed = cu_seqlens is not None
    rank = 3 if packed else 4
    dt = _dtype_of(fn, "q", q, (rank,), "[B, T, H_k, d_k], or packed [T, H_k, d_k] with cu_seqlens")
    if v.dim() != rank:
        raise ValueError(f"{fn}: v must be [B, T, H_v, d_v], or packed [T, H_v, d_v] with cu_seqlens")
    dev, dtype = q.device, q.dtype
    if packed:
        T, Hk, dk = q.shape
        B, lead = _offsets(fn, cu_seqlens, dev), (T,)
    else:
        B, T, Hk, dk = q.shape
        lead = (B, T)
    Hv, dv = v.shape[-2:]
    state = (B, Hv, dk, dv)
    _need(fn, "q", q, dtype, q.shape, dev)
    _need(fn, "k", k, dtype, q.shape, dev)
    _need(fn, "v", v, dtype, (*lead, Hv, dv), dev)
    _need(fn, "g", g, f32, (*lead, Hv), dev)
    _need(fn, "beta", beta, f32, (*lead, Hv), dev)
    if S0 is not None:
        _need(fn, "S0", S0, f32, state, dev)
    if o is None:
        o = torch.empty_like(v)
    else:
        _need(fn, "o", o, dtype, v.shape, dev)
    if S_T is not None:
        _need(fn, "S_T", S_T, f32, state, dev)
    elif want_state:
        S_T = g.new_empty(state)
    if dt == GDN2_BF16 or workspace is not None:
        workspace = _workspace(fn, workspace, lib().gdn2_gdr_chunk_fwd_workspace_bytes(B, T, Hv, dk, dv, packed, dt), dev, g)
    _call(fn, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _adr(cu_seqlens),
          _adr(S0), o.data_ptr(), _adr(S_T), B, T, Hk, Hv, dk, dv, scale, dt, _adr(workspace),
          0 if workspace is None else workspace.nbytes)
    return o, S_T


def gdn2_gdr_decode_step(q, k, v, g, beta, S, *, S_out=None, scale=1.0, o=None, stream=None):
    """One step of the gated delta rule with scalar gates: q, k [B, H_k, d_k], v [B, H_v, d_v], g, beta
    fp32 [B, H_v], S fp32 [B, H_v, d_k, d_v].  The new state goes to S_out, or replaces S when
    S_out is None.  Returns o [B, H_v, d_v] in q's dtype."""
    if stream is not None:
        with _elsewhere(stream, q.device):
            return gdn2_gdr_decode_step(q, k, v, g, beta, S, S_out=S_out, scale=scale, o=o)
    fn, f32 = "gdn2_gdr_decode_step", torch.float32
    dt = _dtype_of(fn, "q", q, (3,), "[B, H_k, d_k]")
    if v.dim() != 3:
        raise ValueError(f"{fn}: v must be [B, H_v, d_v]")
    dev, dtype = q.device, q.dtype
    B, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    state = (B, Hv, dk, dv)
    _need(fn, "q", q, dtype, q.shape, dev)
    _need(fn, "k", k, dtype, q.shape, dev)
    _need(fn, "v", v, dtype, (B, Hv, dv), dev)
    _need(fn, "g", g, f32, (B, Hv), dev)
    _need(fn, "beta", beta, f32, (B, Hv), dev)
    _need(fn, "S", S, f32, state, dev)
    if S_out is None:
        S_out = S
    else:
        _need(fn, "S_out", S_out, f32, state, dev)
    if o is None:
        o = torch.empty_like(v)
    else:
        _need(fn, "o", o, dtype, v.shape, dev)
    _call(fn, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), S.data_ptr(),
          S_out.data_ptr(), o.data_ptr(), B, Hk, Hv, dk, dv, scale, dt)
    return o


def gdn2_device_status() -> int:
    """Synchronises the device and returns (then clears) the library's device status."""
    return lib().gdn2_device_status()
