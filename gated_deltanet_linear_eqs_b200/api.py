"""Python binding of libgdn.so with the C ABI's names.

Argument marshalling only: every function checks that the torch tensors are CUDA,
contiguous and of the expected dtype, allocates the outputs (and workspace) it is not
given, and calls the C entry point on the current CUDA stream.  Every arithmetic step
runs in the library's kernels; a non-OK status raises ``GdnError``.

``stream`` (every call's last argument) runs the call on that stream instead, and takes what
the call allocates from it.  As with torch's own operators, the caller orders the streams: the
tensors given must be ready on that stream, and must be kept until it has used them.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _abi
from ._abi import GdnError

_DT = {torch.bfloat16: _abi.GDN_BF16, torch.float32: _abi.GDN_FP32}


def _lib():
    return _abi.load()


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _on(stream, f, args):
    """f(**args) with `stream` the current one.  The workspace and the outputs then come from that stream's
    memory: a block of the caller's current stream could still be in use by its earlier work, and
    the workspace, dropped when the call returns, could be handed to its next allocation while the
    kernels run.  Outputs may be used on the caller's current stream, too (after waiting for `stream`)."""
    t = next((a for a in args.values() if isinstance(a, torch.Tensor) and a.is_cuda), None)
    if not isinstance(stream, torch.cuda.Stream):  # another library's stream object
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=None if t is None else t.device)
    if t is not None and stream.device != t.device:
        raise ValueError(f"stream is of {stream.device}, the first tensor on {t.device}")
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = f(**{**args, "stream": None})
    if stream != here:
        for o in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
            if isinstance(o, torch.Tensor):
                o.record_stream(here)
    return out


def _p(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t, name, dtype=None, shape=None, optional=False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check(rc, what):
    if rc != _abi.GDN_OK:
        raise GdnError(rc, what)


def gdn_workspace_bytes(op, B, T, H, dk, dv, num_seqs=0):
    n = ctypes.c_size_t(0)
    _check(_lib().gdn_workspace_bytes(int(op), B, T, H, dk, dv, num_seqs, ctypes.byref(n)),
           "gdn_workspace_bytes")
    return int(n.value)


def _workspace(op, device, B, T, H, dk, dv, num_seqs=0, ws=None):
    n = gdn_workspace_bytes(op, B, T, H, dk, dv, num_seqs)
    if n == 0:
        return None, 0
    if ws is None:
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def gdn_prefill(q, k, v, alpha, beta, s0=None, scale=1.0, l2norm_qk=True, y=None,
                s_final=None, want_final=True, ws=None, stream=None):
    """q,k [B,T,H,dk], v [B,T,H,dv] (bf16 or fp32), alpha,beta [B,T,H] fp32,
    s0 [B,H,dk,dv] fp32 or None.  Returns (y, s_final)."""
    if stream is not None:
        return _on(stream, gdn_prefill, locals())
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (B, T, H, dv))
    _need(alpha, "alpha", torch.float32, (B, T, H))
    _need(beta, "beta", torch.float32, (B, T, H))
    _need(s0, "s0", torch.float32, (B, H, dk, dv), optional=True)
    if y is None:
        y = torch.empty((B, T, H, dv), dtype=dt, device=q.device)
    _need(y, "y", dt, (B, T, H, dv))
    if s_final is None and want_final:
        s_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _need(s_final, "s_final", torch.float32, (B, H, dk, dv), optional=True)
    ws, wsb = _workspace(_abi.GDN_OP_PREFILL, q.device, B, T, H, dk, dv, ws=ws)
    rc = _lib().gdn_prefill(_p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(s0), _p(y),
                            _p(s_final), B, T, H, dk, dv, _DT[dt], float(scale),
                            int(bool(l2norm_qk)), _p(ws), wsb, _stream())
    _check(rc, "gdn_prefill")
    return y, s_final


def gdn_prefill_segmented(q, k, v, alpha, beta, s0=None, num_segments=1, scale=1.0,
                          l2norm_qk=True, y=None, s_final=None, want_final=True, ws=None,
                          stream=None):
    """gdn_prefill with every sequence cut into ``num_segments`` segments that run side by side
    (affine state maps, a scan, and a pass from every segment's start state).  Same tensors as
    gdn_prefill.  Returns (y, s_final)."""
    if stream is not None:
        return _on(stream, gdn_prefill_segmented, locals())
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (B, T, H, dv))
    _need(alpha, "alpha", torch.float32, (B, T, H))
    _need(beta, "beta", torch.float32, (B, T, H))
    _need(s0, "s0", torch.float32, (B, H, dk, dv), optional=True)
    if y is None:
        y = torch.empty((B, T, H, dv), dtype=dt, device=q.device)
    _need(y, "y", dt, (B, T, H, dv))
    if s_final is None and want_final:
        s_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _need(s_final, "s_final", torch.float32, (B, H, dk, dv), optional=True)
    ws, wsb = _workspace(_abi.GDN_OP_PREFILL_SEGMENTED, q.device, B, T, H, dk, dv,
                         int(num_segments), ws=ws)
    rc = _lib().gdn_prefill_segmented(_p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(s0), _p(y),
                                      _p(s_final), B, T, H, dk, dv, _DT[dt], float(scale),
                                      int(bool(l2norm_qk)), int(num_segments), _p(ws), wsb,
                                      _stream())
    _check(rc, "gdn_prefill_segmented")
    return y, s_final


def gdn_prefill_varlen(q, k, v, alpha, beta, cu_seqlens, s0=None, scale=1.0, l2norm_qk=True,
                       y=None, s_final=None, ws=None, stream=None):
    """Packed documents: q,k [1,T,H,dk] (or [T,H,dk]), v likewise, alpha,beta [1,T,H],
    cu_seqlens int32 [N+1] on the device, s0 [N,H,dk,dv] or None.  Returns (y, s_final)."""
    if stream is not None:
        return _on(stream, gdn_prefill_varlen, locals())
    if q.dim() == 3:
        q, k, v, alpha, beta = (x.unsqueeze(0) for x in (q, k, v, alpha, beta))
    _, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    N = cu_seqlens.numel() - 1
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (1, T, H, dv))
    _need(alpha, "alpha", torch.float32, (1, T, H))
    _need(beta, "beta", torch.float32, (1, T, H))
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    _need(s0, "s0", torch.float32, (N, H, dk, dv), optional=True)
    if y is None:
        y = torch.empty((1, T, H, dv), dtype=dt, device=q.device)
    _need(y, "y", dt, (1, T, H, dv))
    if s_final is None:
        s_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    _need(s_final, "s_final", torch.float32, (N, H, dk, dv))
    ws, wsb = _workspace(_abi.GDN_OP_PREFILL_VARLEN, q.device, 1, T, H, dk, dv, N, ws=ws)
    rc = _lib().gdn_prefill_varlen(_p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(cu_seqlens), N,
                                   _p(s0), _p(y), _p(s_final), T, H, dk, dv, _DT[dt],
                                   float(scale), int(bool(l2norm_qk)), _p(ws), wsb,
                                   _stream())
    _check(rc, "gdn_prefill_varlen")
    return y, s_final


def gdn_prefill_varlen_prepare(q, k, v, alpha, beta, cu_seqlens, ws, scale=1.0,
                               l2norm_qk=True, stream=None):
    """First phase of gdn_prefill_varlen (bf16): the state-independent chunk work, into ``ws``
    (a uint8 device tensor of gdn_workspace_bytes(GDN_OP_PREFILL_VARLEN, ...) bytes)."""
    if stream is not None:
        return _on(stream, gdn_prefill_varlen_prepare, locals())
    if q.dim() == 3:
        q, k, v, alpha, beta = (x.unsqueeze(0) for x in (q, k, v, alpha, beta))
    _, T, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16, q.shape)
    _need(v, "v", torch.bfloat16, (1, T, H, dv))
    _need(alpha, "alpha", torch.float32, (1, T, H))
    _need(beta, "beta", torch.float32, (1, T, H))
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    rc = _lib().gdn_prefill_varlen_prepare(_p(q), _p(k), _p(v), _p(alpha), _p(beta),
                                           _p(cu_seqlens), N, T, H, dk, dv, _DT[torch.bfloat16],
                                           float(scale), int(bool(l2norm_qk)), _p(ws),
                                           ws.numel() * ws.element_size(), _stream())
    _check(rc, "gdn_prefill_varlen_prepare")


def gdn_prefill_varlen_finish(q, k, cu_seqlens, ws, s0=None, y=None, s_final=None, dv=None,
                              stream=None):
    """Second phase of gdn_prefill_varlen (bf16): the sequential chunk pass from s0 over the
    records gdn_prefill_varlen_prepare wrote into ``ws``.  Returns (y, s_final)."""
    if stream is not None:
        return _on(stream, gdn_prefill_varlen_finish, locals())
    if q.dim() == 3:
        q, k = q.unsqueeze(0), k.unsqueeze(0)
    _, T, H, dk = q.shape
    dv = dk if dv is None else dv
    N = cu_seqlens.numel() - 1
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16, q.shape)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    _need(s0, "s0", torch.float32, (N, H, dk, dv), optional=True)
    if y is None:
        y = torch.empty((1, T, H, dv), dtype=torch.bfloat16, device=q.device)
    _need(y, "y", torch.bfloat16, (1, T, H, dv))
    if s_final is None:
        s_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    _need(s_final, "s_final", torch.float32, (N, H, dk, dv))
    rc = _lib().gdn_prefill_varlen_finish(_p(q), _p(k), _p(cu_seqlens), N, _p(s0), _p(y),
                                          _p(s_final), T, H, dk, dv, _DT[torch.bfloat16], _p(ws),
                                          ws.numel() * ws.element_size(), _stream())
    _check(rc, "gdn_prefill_varlen_finish")
    return y, s_final


def gdn_decode_step(q, k, v, alpha, beta, state, scale=1.0, l2norm_qk=True, y=None,
                    stream=None):
    """q,k [N,H,dk], v [N,H,dv], alpha,beta [N,H], state [N,H,dk,dv] fp32 (updated in
    place).  Returns y [N,H,dv]."""
    if stream is not None:
        return _on(stream, gdn_decode_step, locals())
    N, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (N, H, dv))
    _need(alpha, "alpha", torch.float32, (N, H))
    _need(beta, "beta", torch.float32, (N, H))
    _need(state, "state", torch.float32, (N, H, dk, dv))
    if y is None:
        y = torch.empty((N, H, dv), dtype=dt, device=q.device)
    _need(y, "y", dt, (N, H, dv))
    rc = _lib().gdn_decode_step(_p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(state), _p(y), N, H,
                                dk, dv, _DT[dt], float(scale), int(bool(l2norm_qk)),
                                _stream())
    _check(rc, "gdn_decode_step")
    return y


def gdn_backward(q, k, v, alpha, beta, dy, s0=None, ds_final=None, scale=1.0, l2norm_qk=True,
                 want_ds0=True, ws=None, stream=None):
    """Gradients of (y, s_final) w.r.t. (q, k, v, alpha, beta, s0) given dy and ds_final.
    Returns dict dq, dk, dv, dalpha, dbeta, ds0."""
    if stream is not None:
        return _on(stream, gdn_backward, locals())
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (B, T, H, dv))
    _need(alpha, "alpha", torch.float32, (B, T, H))
    _need(beta, "beta", torch.float32, (B, T, H))
    _need(dy, "dy", dt, (B, T, H, dv))
    _need(s0, "s0", torch.float32, (B, H, dk, dv), optional=True)
    _need(ds_final, "ds_final", torch.float32, (B, H, dk, dv), optional=True)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dalpha=torch.empty_like(alpha), dbeta=torch.empty_like(beta),
               ds0=torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
               if want_ds0 else None)
    ws, wsb = _workspace(_abi.GDN_OP_BACKWARD, q.device, B, T, H, dk, dv, ws=ws)
    rc = _lib().gdn_backward(_p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(s0), _p(dy),
                             _p(ds_final), _p(out["dq"]), _p(out["dk"]), _p(out["dv"]),
                             _p(out["dalpha"]), _p(out["dbeta"]), _p(out["ds0"]), B, T, H, dk,
                             dv, _DT[dt], float(scale), int(bool(l2norm_qk)), _p(ws), wsb,
                             _stream())
    _check(rc, "gdn_backward")
    return out


def gdn_backward_noalloc(q, k, v, alpha, beta, dy, s0=None, ds_final=None, scale=1.0,
                         l2norm_qk=True, want_ds0=True, out=None, stream=None):
    """gdn_backward on the library's fixed device scratch: no workspace is passed and the
    library allocates nothing.  ``out`` may supply preallocated gradient tensors (a dict with
    the keys of gdn_backward's result), so that a caller without an allocator can pass its
    own buffers.  Returns the gradient dict."""
    if stream is not None:
        return _on(stream, gdn_backward_noalloc, locals())
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (B, T, H, dv))
    _need(alpha, "alpha", torch.float32, (B, T, H))
    _need(beta, "beta", torch.float32, (B, T, H))
    _need(dy, "dy", dt, (B, T, H, dv))
    _need(s0, "s0", torch.float32, (B, H, dk, dv), optional=True)
    _need(ds_final, "ds_final", torch.float32, (B, H, dk, dv), optional=True)
    if out is None:
        out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                   dalpha=torch.empty_like(alpha), dbeta=torch.empty_like(beta),
                   ds0=torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
                   if want_ds0 else None)
    rc = _lib().gdn_backward_noalloc(_p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(s0), _p(dy),
                                     _p(ds_final), _p(out["dq"]), _p(out["dk"]), _p(out["dv"]),
                                     _p(out["dalpha"]), _p(out["dbeta"]), _p(out.get("ds0")), B,
                                     T, H, dk, dv, _DT[dt], float(scale), int(bool(l2norm_qk)),
                                     _stream())
    _check(rc, "gdn_backward_noalloc")
    return out


def gdn_backward_noalloc_max_workspace():
    return int(_lib().gdn_backward_noalloc_max_workspace())


def _need_gate(a, b, A_log, b_alpha, shape, H):
    _need(a, "a", torch.float32, shape)
    _need(b, "b", torch.float32, shape)
    _need(A_log, "A_log", torch.float32, (H,))
    _need(b_alpha, "b_alpha", torch.float32, (H,))


def gdn_prefill_gated(q, k, v, a, b, A_log, b_alpha, s0=None, scale=1.0, l2norm_qk=True,
                      y=None, s_final=None, want_final=True, ws=None, stream=None):
    """gdn_prefill with alpha and beta given by eqs. (9)-(10): a = W_alpha x, b = W_beta x
    [B,T,H] fp32, A_log and b_alpha [H] fp32.  Returns (y, s_final)."""
    if stream is not None:
        return _on(stream, gdn_prefill_gated, locals())
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (B, T, H, dv))
    _need_gate(a, b, A_log, b_alpha, (B, T, H), H)
    _need(s0, "s0", torch.float32, (B, H, dk, dv), optional=True)
    if y is None:
        y = torch.empty((B, T, H, dv), dtype=dt, device=q.device)
    _need(y, "y", dt, (B, T, H, dv))
    if s_final is None and want_final:
        s_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _need(s_final, "s_final", torch.float32, (B, H, dk, dv), optional=True)
    ws, wsb = _workspace(_abi.GDN_OP_PREFILL, q.device, B, T, H, dk, dv, ws=ws)
    rc = _lib().gdn_prefill_gated(_p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log), _p(b_alpha),
                                  _p(s0), _p(y), _p(s_final), B, T, H, dk, dv, _DT[dt],
                                  float(scale), int(bool(l2norm_qk)), _p(ws), wsb,
                                  _stream())
    _check(rc, "gdn_prefill_gated")
    return y, s_final


def gdn_prefill_varlen_gated(q, k, v, a, b, A_log, b_alpha, cu_seqlens, s0=None, scale=1.0,
                             l2norm_qk=True, y=None, s_final=None, ws=None, stream=None):
    """gdn_prefill_varlen with alpha and beta given by eqs. (9)-(10) (a, b [1,T,H] or [T,H]
    fp32; A_log, b_alpha [H]).  Returns (y, s_final)."""
    if stream is not None:
        return _on(stream, gdn_prefill_varlen_gated, locals())
    if q.dim() == 3:
        q, k, v, a, b = (x.unsqueeze(0) for x in (q, k, v, a, b))
    _, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    N = cu_seqlens.numel() - 1
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (1, T, H, dv))
    _need_gate(a, b, A_log, b_alpha, (1, T, H), H)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,))
    _need(s0, "s0", torch.float32, (N, H, dk, dv), optional=True)
    if y is None:
        y = torch.empty((1, T, H, dv), dtype=dt, device=q.device)
    _need(y, "y", dt, (1, T, H, dv))
    if s_final is None:
        s_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    _need(s_final, "s_final", torch.float32, (N, H, dk, dv))
    ws, wsb = _workspace(_abi.GDN_OP_PREFILL_VARLEN, q.device, 1, T, H, dk, dv, N, ws=ws)
    rc = _lib().gdn_prefill_varlen_gated(_p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log),
                                         _p(b_alpha), _p(cu_seqlens), N, _p(s0), _p(y),
                                         _p(s_final), T, H, dk, dv, _DT[dt], float(scale),
                                         int(bool(l2norm_qk)), _p(ws), wsb, _stream())
    _check(rc, "gdn_prefill_varlen_gated")
    return y, s_final


def gdn_decode_step_gated(q, k, v, a, b, A_log, b_alpha, state, scale=1.0, l2norm_qk=True,
                          y=None, stream=None):
    """gdn_decode_step with alpha and beta given by eqs. (9)-(10) (a, b [N,H] fp32; A_log,
    b_alpha [H]).  The state is updated in place.  Returns y [N,H,dv]."""
    if stream is not None:
        return _on(stream, gdn_decode_step_gated, locals())
    N, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (N, H, dv))
    _need_gate(a, b, A_log, b_alpha, (N, H), H)
    _need(state, "state", torch.float32, (N, H, dk, dv))
    if y is None:
        y = torch.empty((N, H, dv), dtype=dt, device=q.device)
    _need(y, "y", dt, (N, H, dv))
    rc = _lib().gdn_decode_step_gated(_p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log), _p(b_alpha),
                                      _p(state), _p(y), N, H, dk, dv, _DT[dt], float(scale),
                                      int(bool(l2norm_qk)), _stream())
    _check(rc, "gdn_decode_step_gated")
    return y


def gdn_backward_gated(q, k, v, a, b, A_log, b_alpha, dy, s0=None, ds_final=None, scale=1.0,
                       l2norm_qk=True, want_ds0=True, ws=None, stream=None):
    """Gradients of (y, s_final) for the gated form.  Returns dict dq, dk, dv, da, db,
    dA_log, db_alpha, ds0."""
    if stream is not None:
        return _on(stream, gdn_backward_gated, locals())
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DT:
        raise ValueError("q/k/v must be bf16 or fp32")
    _need(q, "q", dt)
    _need(k, "k", dt, q.shape)
    _need(v, "v", dt, (B, T, H, dv))
    _need_gate(a, b, A_log, b_alpha, (B, T, H), H)
    _need(dy, "dy", dt, (B, T, H, dv))
    _need(s0, "s0", torch.float32, (B, H, dk, dv), optional=True)
    _need(ds_final, "ds_final", torch.float32, (B, H, dk, dv), optional=True)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               da=torch.empty_like(a), db=torch.empty_like(b), dA_log=torch.empty_like(A_log),
               db_alpha=torch.empty_like(b_alpha),
               ds0=torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
               if want_ds0 else None)
    ws, wsb = _workspace(_abi.GDN_OP_BACKWARD, q.device, B, T, H, dk, dv, ws=ws)
    rc = _lib().gdn_backward_gated(_p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log), _p(b_alpha),
                                   _p(s0), _p(dy), _p(ds_final), _p(out["dq"]), _p(out["dk"]),
                                   _p(out["dv"]), _p(out["da"]), _p(out["db"]),
                                   _p(out["dA_log"]), _p(out["db_alpha"]), _p(out["ds0"]), B, T,
                                   H, dk, dv, _DT[dt], float(scale), int(bool(l2norm_qk)), _p(ws),
                                   wsb, _stream())
    _check(rc, "gdn_backward_gated")
    return out


def gdn_gated_rmsnorm(y, z, w, eps=1e-6, o=None, stream=None):
    """The bracket of eq. (11): sigmoid(z) * (1 + w) * y / sqrt(mean(y^2) + eps) over the last
    axis.  y, z [..., dv] (bf16 or fp32, same dtype), w [dv] fp32.  Returns o like y."""
    if stream is not None:
        return _on(stream, gdn_gated_rmsnorm, locals())
    dt = y.dtype
    if dt not in _DT:
        raise ValueError("y/z must be bf16 or fp32")
    dv = y.shape[-1]
    _need(y, "y", dt)
    _need(z, "z", dt, y.shape)
    _need(w, "w", torch.float32, (dv,))
    if o is None:
        o = torch.empty_like(y)
    _need(o, "o", dt, y.shape)
    rows = y.numel() // dv if dv else 0
    rc = _lib().gdn_gated_rmsnorm(_p(y), _p(z), _p(w), _p(o), rows, dv, _DT[dt], float(eps),
                                  _stream())
    _check(rc, "gdn_gated_rmsnorm")
    return o


def gdn_gated_rmsnorm_backward(y, z, w, d_o, eps=1e-6, stream=None):
    """Gradients of gdn_gated_rmsnorm given d_o.  Returns dict dy, dz (like y) and dw [dv]."""
    if stream is not None:
        return _on(stream, gdn_gated_rmsnorm_backward, locals())
    dt = y.dtype
    if dt not in _DT:
        raise ValueError("y/z must be bf16 or fp32")
    dv = y.shape[-1]
    _need(y, "y", dt)
    _need(z, "z", dt, y.shape)
    _need(w, "w", torch.float32, (dv,))
    _need(d_o, "d_o", dt, y.shape)
    out = dict(dy=torch.empty_like(y), dz=torch.empty_like(z), dw=torch.empty_like(w))
    rows = y.numel() // dv if dv else 0
    rc = _lib().gdn_gated_rmsnorm_backward(_p(y), _p(z), _p(w), _p(d_o), _p(out["dy"]),
                                           _p(out["dz"]), _p(out["dw"]), rows, dv, _DT[dt],
                                           float(eps), _stream())
    _check(rc, "gdn_gated_rmsnorm_backward")
    return out


def gdn_read_device_status(reset=True):
    st = ctypes.c_int(0)
    _check(_lib().gdn_read_device_status(int(bool(reset)), ctypes.byref(st)),
           "gdn_read_device_status")
    return int(st.value)


def gdn_selftest_wait_timeout(limit_ns=1_000_000, stream=None):
    """Launch the kernel whose bounded wait runs out (see include/gdn.h); afterwards
    gdn_read_device_status() reports GDN_ERR_TIMEOUT."""
    if stream is not None:
        return _on(stream, gdn_selftest_wait_timeout, locals())
    _check(_lib().gdn_selftest_wait_timeout(int(limit_ns), _stream()),
           "gdn_selftest_wait_timeout")


_ACT = {"none": 0, "silu": 1}


def gdn_short_conv_varlen(x, w, cu_seqlens, conv_state=None, activation="none",
                          return_state=True, y=None, stream=None):
    """Short causal convolution of packed documents: x [T, C] (bf16 or fp32, C % 8 == 0),
    w [C, W] fp32, cu_seqlens [N+1] int32 (CUDA), conv_state [N, W-1, C] like x or None (zero).
    Returns (y [T, C], final conv state [N, W-1, C] or None)."""
    if stream is not None:
        return _on(stream, gdn_short_conv_varlen, locals())
    dt = x.dtype
    if dt not in _DT:
        raise ValueError("x must be bf16 or fp32")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [T, C] and w [C, W]")
    T, C = x.shape
    W = w.shape[1]
    _need(x, "x", dt)
    _need(w, "w", torch.float32, (C, W))
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    N = cu_seqlens.numel() - 1
    _need(conv_state, "conv_state", dt, (N, W - 1, C), optional=True)
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", dt, (T, C))
    sf = torch.empty((N, W - 1, C), dtype=dt, device=x.device) if return_state else None
    rc = _lib().gdn_short_conv_varlen(_p(x), _p(w), _p(cu_seqlens), N, _p(conv_state), _p(sf),
                                      _p(y), T, C, W, _DT[dt], _ACT[activation], _stream())
    _check(rc, "gdn_short_conv_varlen")
    return y, sf


def gdn_short_conv_step(x, w, conv_state, activation="none", y=None, stream=None):
    """One decode token per sequence: x [N, C], w [C, W] fp32, conv_state [N, W-1, C] like x,
    updated in place.  Returns y [N, C]."""
    if stream is not None:
        return _on(stream, gdn_short_conv_step, locals())
    dt = x.dtype
    if dt not in _DT:
        raise ValueError("x must be bf16 or fp32")
    N, C = x.shape
    W = w.shape[1]
    _need(x, "x", dt)
    _need(w, "w", torch.float32, (C, W))
    _need(conv_state, "conv_state", dt, (N, W - 1, C))
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", dt, (N, C))
    rc = _lib().gdn_short_conv_step(_p(x), _p(w), _p(conv_state), _p(y), N, C, W, _DT[dt],
                                    _ACT[activation], _stream())
    _check(rc, "gdn_short_conv_step")
    return y


def _qsa_ld(max_doc_len):
    return ((max_doc_len // 4) + 3) // 4 * 4


def gdn_qsa_block_scores(q, k, g, cu_seqlens, max_doc_len, stream=None):
    """QSA indexer, pooled keys and block scores: q [T, 4, 128] bf16, k [T, 128] bf16, g [128]
    fp32, cu_seqlens [N+1] int32 (CUDA), every document at most max_doc_len tokens.  Returns
    (k_hat [T//4, 128] bf16, block_base [N+1] int32, scores [T, ld] fp32); row t of scores holds
    its visible blocks' scores (document-local block order), the rest is not written."""
    if stream is not None:
        return _on(stream, gdn_qsa_block_scores, locals())
    T = q.shape[0]
    _need(q, "q", torch.bfloat16, (T, 4, 128))
    _need(k, "k", torch.bfloat16, (T, 128))
    _need(g, "g", torch.float32, (128,))
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    N = cu_seqlens.numel() - 1
    ld = _qsa_ld(max_doc_len)
    dev = q.device
    k_hat = torch.empty((T // 4, 128), dtype=torch.bfloat16, device=dev)
    base = torch.empty(N + 1, dtype=torch.int32, device=dev)
    scores = torch.empty((T, ld), dtype=torch.float32, device=dev)
    ws = torch.empty(gdn_workspace_bytes(_abi.GDN_OP_QSA_SCORES, 1, max(T, 1), 1, 128, 128, N),
                     dtype=torch.uint8, device=dev)
    rc = _lib().gdn_qsa_block_scores(_p(q), _p(k), _p(g), _p(cu_seqlens), N, T, int(max_doc_len),
                                     _p(k_hat), _p(base), _p(scores), ld, _p(ws), ws.numel(),
                                     _stream())
    _check(rc, "gdn_qsa_block_scores")
    return k_hat, base, scores


def gdn_qsa_select_blocks(scores, cu_seqlens, budget=512, sel=None, stream=None):
    """Top-budget block selection from gdn_qsa_block_scores' scores: sel [T, budget] int32."""
    if stream is not None:
        return _on(stream, gdn_qsa_select_blocks, locals())
    _need(scores, "scores", torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    T, ld = scores.shape
    if sel is None:
        sel = torch.empty((T, budget), dtype=torch.int32, device=scores.device)
    _need(sel, "sel", torch.int32, (T, budget))
    rc = _lib().gdn_qsa_select_blocks(_p(scores), ld, _p(cu_seqlens), cu_seqlens.numel() - 1, T,
                                      int(budget), _p(sel), _stream())
    _check(rc, "gdn_qsa_select_blocks")
    return sel


def gdn_qsa_indexer(q, k, g, cu_seqlens, max_doc_len, budget=512, stream=None):
    """Both steps: returns (sel [T, budget] int32, k_hat, block_base, scores)."""
    if stream is not None:
        return _on(stream, gdn_qsa_indexer, locals())
    k_hat, base, scores = gdn_qsa_block_scores(q, k, g, cu_seqlens, max_doc_len)
    return gdn_qsa_select_blocks(scores, cu_seqlens, budget), k_hat, base, scores


# The calls below serve decode steps of a few microseconds on the GPU, so their checks are kept short: one
# comparison a tensor, the reasons looked for only when it fails (_refuse), the stream taken as a raw handle.

_current_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda dev: torch.cuda.current_stream(dev).cuda_stream
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _launch(dev, f, a):
    """f(*a) with device dev current: a launch goes to the current device, whatever device its pointers are on."""
    with torch.cuda.device(dev):
        return f(*a)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _refuse(t, name, dtype, shape, dev):
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} is on device {t.get_device()}, the first tensor on {dev}")


def _want(t, name, dtype, shape, dev):
    """A contiguous tensor of the given type and shape on device dev."""
    if t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != dev or \
            not t.is_contiguous() or dev < 0:
        _refuse(t, name, dtype, shape, dev)


_INT_MAX = 2 ** 31 - 1  # of the sizes that the library takes as ints: a larger one would arrive as its low 32 bits


def _too_large(what, n):
    raise ValueError(f"{what} must be below 2^31, got {n}")


def _dtype(t, name):
    dt = t.dtype
    if dt not in _DT:
        raise ValueError(f"{name} must be bf16 or fp32")
    return dt


@functools.lru_cache(maxsize=1024)
def _attn_ws_bytes(backward, B, T, H, Hk, dk, dv, num_seqs):
    n = ctypes.c_size_t(0)
    _check(_lib().gdn_linear_attn_workspace_bytes(backward, B, T, H, Hk, dk, dv, num_seqs, ctypes.byref(n)),
           "gdn_linear_attn_workspace_bytes")
    return int(n.value)


def gdn_linear_attn_workspace_bytes(B, T, H, Hk, dk, dv, num_seqs=0, backward=False):
    """Bytes of device scratch of gdn_linear_attn (num_seqs = 0) and gdn_linear_attn_varlen
    (num_seqs documents, B = 1), or of their backward calls."""
    return _attn_ws_bytes(int(bool(backward)), B, T, H, Hk, dk, dv, num_seqs)


def _scratch(n, ws, dev):
    """(the tensor, its pointer, its bytes): ws if given (any contiguous tensor), else n bytes."""
    if ws is None:
        if n == 0:
            return None, None, 0
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be contiguous and on the other tensors' device")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _attn_shapes(q, k, v, log_decay):
    """Checks q [B,T,H,d], k and v [B,T,Hk,d], log_decay [H]; returns (dtype, device, B, T, H, Hk, d)."""
    dt = _dtype(q, "q/k/v")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must be [B, T, heads, d] (packed: [1, T, heads, d] or "
                         "[T, heads, d])")
    B, T, H, d = q.shape
    Hk = k.shape[2]
    if Hk < 1 or H % Hk:
        raise ValueError(f"{Hk} heads of k and v cannot be shared by {H} heads of q")
    dev = q.get_device()
    _want(q, "q", dt, (B, T, H, d), dev)
    _want(k, "k", dt, (B, T, Hk, d), dev)
    _want(v, "v", dt, (B, T, Hk, d), dev)
    _want(log_decay, "log_decay", torch.float32, (H,), dev)
    return dt, dev, B, T, H, Hk, d


def _states(t, name, shape, dev, make=False):
    """An optional fp32 state tensor: checked, or made where it is wanted."""
    if t is None:
        return torch.empty(shape, dtype=torch.float32, device=dev) if make else None
    _want(t, name, torch.float32, shape, dev)
    return t


def gdn_linear_attn(q, k, v, log_decay, s0=None, scale=1.0, y=None, s_final=None, want_final=True,
                    ws=None, stream=None):
    """Decayed linear attention S_t = e^g S_{t-1} + k_t v_t^T, y_t = scale S_t^T q_t of dense
    sequences: q [B,T,H,d], k and v [B,T,Hk,d] (bf16 or fp32; Hk divides H), log_decay [H] fp32
    (g <= 0, a constant), s0 [B,H,d,d] fp32 or None.  Returns (y, s_final)."""
    if stream is not None:
        return _on(stream, gdn_linear_attn, locals())
    dt, dev, B, T, H, Hk, d = _attn_shapes(q, k, v, log_decay)
    s0 = _states(s0, "s0", (B, H, d, d), dev)
    if y is None:
        y = torch.empty_like(q)
    else:
        _want(y, "y", dt, q.shape, dev)
    s_final = _states(s_final, "s_final", (B, H, d, d), dev, want_final)
    ws, wsp, wsb = _scratch(_attn_ws_bytes(0, B, T, H, Hk, d, d, 0), ws, dev)
    f = _lib().gdn_linear_attn
    a = (q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(s0), y.data_ptr(), _ptr(s_final),
         B, T, H, Hk, d, d, _DT[dt], scale, wsp, wsb, _current_stream(dev))
    rc = f(*a) if dev == _current_device() else _launch(dev, f, a)
    if rc:
        _check(rc, "gdn_linear_attn")
    return y, s_final


def _packed(q, *more):
    return tuple(x.unsqueeze(0) for x in (q, *more)) if q.dim() == 3 else (q, *more)


def _documents(B, cu_seqlens, dev):
    if B != 1:
        raise ValueError("packed documents are one stream: q must be [1, T, H, d] or [T, H, d]")
    n = cu_seqlens.numel()
    if n > _INT_MAX:
        _too_large("cu_seqlens' length", n)
    _want(cu_seqlens, "cu_seqlens", torch.int32, (n,), dev)
    return n - 1


def gdn_linear_attn_varlen(q, k, v, log_decay, cu_seqlens, s0=None, scale=1.0, y=None,
                           s_final=None, want_final=True, ws=None, stream=None):
    """gdn_linear_attn of packed documents: q [1,T,H,d] or [T,H,d] (k, v likewise), cu_seqlens
    int32 [N+1] on the device, s0 [N,H,d,d] fp32 or None.  Rows outside the documents are not written.
    Returns (y like q, s_final)."""
    if stream is not None:
        return _on(stream, gdn_linear_attn_varlen, locals())
    if y is None:
        y = torch.empty_like(q)
    else:
        _want(y, "y", q.dtype, q.shape, q.get_device())
    q, k, v = _packed(q, k, v)
    dt, dev, B, T, H, Hk, d = _attn_shapes(q, k, v, log_decay)
    N = _documents(B, cu_seqlens, dev)
    s0 = _states(s0, "s0", (N, H, d, d), dev)
    s_final = _states(s_final, "s_final", (N, H, d, d), dev, want_final)
    ws, wsp, wsb = _scratch(_attn_ws_bytes(0, 1, T, H, Hk, d, d, N), ws, dev)
    f = _lib().gdn_linear_attn_varlen
    a = (q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), cu_seqlens.data_ptr(), N, _ptr(s0),
         y.data_ptr(), _ptr(s_final), T, H, Hk, d, d, _DT[dt], scale, wsp, wsb, _current_stream(dev))
    rc = f(*a) if dev == _current_device() else _launch(dev, f, a)
    if rc:
        _check(rc, "gdn_linear_attn_varlen")
    return y, s_final


def gdn_linear_attn_decode_step(q, k, v, log_decay, state, scale=1.0, y=None, stream=None):
    """One token of N sequences: q [N,H,d], k and v [N,Hk,d], state [N,H,d,d] fp32 (updated in
    place).  Returns y [N,H,d]."""
    if stream is not None:
        return _on(stream, gdn_linear_attn_decode_step, locals())
    dt = _dtype(q, "q/k/v")
    N, H, d = q.shape
    Hk = k.shape[1]
    dev = q.get_device()
    _want(q, "q", dt, (N, H, d), dev)
    _want(k, "k", dt, (N, Hk, d), dev)
    _want(v, "v", dt, (N, Hk, d), dev)
    _want(log_decay, "log_decay", torch.float32, (H,), dev)
    _want(state, "state", torch.float32, (N, H, d, d), dev)
    if y is None:
        y = torch.empty_like(q)
    else:
        _want(y, "y", dt, q.shape, dev)
    f = _lib().gdn_linear_attn_decode_step
    a = (q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state.data_ptr(), y.data_ptr(), N, H,
         Hk, d, d, _DT[dt], scale, _current_stream(dev))
    rc = f(*a) if dev == _current_device() else _launch(dev, f, a)
    if rc:
        _check(rc, "gdn_linear_attn_decode_step")
    return y


def gdn_linear_attn_backward(q, k, v, log_decay, dy, s0=None, ds_final=None, scale=1.0,
                             want_ds0=True, ws=None, stream=None):
    """Gradients of gdn_linear_attn's (y, s_final) given dy [B,T,H,d] and ds_final.  Returns dict
    dq, dk, dv (like q, k, v) and ds0 [B,H,d,d] (None unless want_ds0)."""
    if stream is not None:
        return _on(stream, gdn_linear_attn_backward, locals())
    dt, dev, B, T, H, Hk, d = _attn_shapes(q, k, v, log_decay)
    _want(dy, "dy", dt, q.shape, dev)
    s0 = _states(s0, "s0", (B, H, d, d), dev)
    ds_final = _states(ds_final, "ds_final", (B, H, d, d), dev)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ds0 = _states(None, "ds0", (B, H, d, d), dev, want_ds0)
    ws, wsp, wsb = _scratch(_attn_ws_bytes(1, B, T, H, Hk, d, d, 0), ws, dev)
    f = _lib().gdn_linear_attn_backward
    a = (q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(s0), dy.data_ptr(), _ptr(ds_final),
         dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(ds0), B, T, H, Hk, d, d, _DT[dt], scale, wsp, wsb,
         _current_stream(dev))
    rc = f(*a) if dev == _current_device() else _launch(dev, f, a)
    if rc:
        _check(rc, "gdn_linear_attn_backward")
    return dict(dq=dq, dk=dk, dv=dv, ds0=ds0)


def gdn_linear_attn_backward_varlen(q, k, v, log_decay, cu_seqlens, dy, s0=None, ds_final=None,
                                    scale=1.0, want_ds0=True, ws=None, stream=None):
    """Gradients of gdn_linear_attn_varlen given dy (like q) and ds_final [N,H,d,d].  Returns
    dict dq, dk, dv (like q, k, v; rows outside the documents are not written) and ds0 [N,H,d,d]
    (None unless want_ds0)."""
    if stream is not None:
        return _on(stream, gdn_linear_attn_backward_varlen, locals())
    _want(dy, "dy", q.dtype, q.shape, q.get_device())
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    q, k, v = _packed(q, k, v)
    dt, dev, B, T, H, Hk, d = _attn_shapes(q, k, v, log_decay)
    N = _documents(B, cu_seqlens, dev)
    s0 = _states(s0, "s0", (N, H, d, d), dev)
    ds_final = _states(ds_final, "ds_final", (N, H, d, d), dev)
    ds0 = _states(None, "ds0", (N, H, d, d), dev, want_ds0)
    ws, wsp, wsb = _scratch(_attn_ws_bytes(1, 1, T, H, Hk, d, d, N), ws, dev)
    f = _lib().gdn_linear_attn_backward_varlen
    a = (q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), cu_seqlens.data_ptr(), N, _ptr(s0),
         dy.data_ptr(), _ptr(ds_final), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(ds0), T, H, Hk, d, d,
         _DT[dt], scale, wsp, wsb, _current_stream(dev))
    rc = f(*a) if dev == _current_device() else _launch(dev, f, a)
    if rc:
        _check(rc, "gdn_linear_attn_backward_varlen")
    return dict(dq=dq, dk=dk, dv=dv, ds0=ds0)


def _heads(t, name, dtype, dev, tokens, heads, d):
    """The token distance of a [T, heads, d] or [B, T, heads, d] tensor whose heads are contiguous and whose
    tokens are evenly spaced (tokens, heads, d: what it must have; heads None: any)."""
    shape = t.shape
    if t.dtype is not dtype or t.get_device() != dev or dev < 0:
        _need(t, name, dtype)
        raise ValueError(f"{name} is on device {t.get_device()}, the first tensor on {dev}")
    nd = len(shape)
    if nd == 3 and t.is_contiguous() and shape[0] == tokens and shape[2] == d and (heads is None or shape[1] == heads):
        return shape[1] * d
    st = t.stride()
    if nd != 3 and nd != 4:
        raise ValueError(f"{name} must be [T, heads, d] or [B, T, heads, d]")
    h, hd = shape[-2], shape[-1]
    row = h * hd
    n = shape[0] if nd == 3 else shape[0] * shape[1]
    if n != tokens or hd != d or (heads is not None and h != heads):
        raise ValueError(f"{name} has {n} tokens of {h} heads of {hd}; expected {tokens} of "
                         f"{'any' if heads is None else heads} heads of {d}")
    if n <= 1:
        ld = row
    else:
        ld = st[-3] if shape[-3] > 1 else st[0]
    if n and ((hd > 1 and st[-1] != 1) or (h > 1 and st[-2] != hd) or
              (nd == 4 and shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * ld)):
        raise ValueError(f"{name}: a token's heads must be contiguous and its tokens evenly spaced")
    return ld


def gdn_rotary(q, k, positions, inv_freq, interleaved=False, inverse=False, scale=1.0, q_out=None,
               k_out=None, stream=None):
    """Rotary positions of q [T,Hq,d] and k [T,Hk,d] (or [B,T,..]; k may be None): the first
    2 * len(inv_freq) values of each head, in pairs (i, i + r/2) or, interleaved, (2i, 2i+1), turn
    by positions[t] * inv_freq[i] and are scaled; inverse turns back (the gradient).  q and k may be
    views into one projection (contiguous heads, evenly spaced tokens).  positions int32 (one
    per token), inv_freq fp32 on the device.  q_out / k_out may be q / k.  Returns (q_out, k_out)."""
    if stream is not None:
        return _on(stream, gdn_rotary, locals())
    dt = _dtype(q, "q/k")
    dev = q.get_device()
    if q.dim() < 3:
        raise ValueError("q must be [T, heads, d] or [B, T, heads, d]")
    Hq, d = q.shape[-2:]
    T = q.shape[0] if q.dim() == 3 else q.shape[0] * q.shape[1]
    if T > _INT_MAX or Hq * d > _INT_MAX:
        _too_large("q's tokens, and a token's row,", (T, Hq * d))
    ldq = _heads(q, "q", dt, dev, T, None, d)
    _want(positions, "positions", torch.int32, positions.shape, dev)
    half = inv_freq.numel()
    _want(inv_freq, "inv_freq", torch.float32, (half,), dev)
    if positions.numel() != T:
        raise ValueError(f"positions must have {T} entries, got {positions.numel()}")
    if k is None:
        Hk = ldk = ldko = 0
        kp = kop = k_out = None
    else:
        Hk = k.shape[-2]
        if Hk * d > _INT_MAX:
            _too_large("a token's row of k", Hk * d)
        ldk = _heads(k, "k", dt, dev, T, None, d)
        if k_out is None:
            k_out, ldko = torch.empty_like(k, memory_format=torch.contiguous_format), Hk * d
        else:
            ldko = _heads(k_out, "k_out", dt, dev, T, Hk, d)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    if q_out is None:
        q_out, ldqo = torch.empty_like(q, memory_format=torch.contiguous_format), Hq * d
    else:
        ldqo = _heads(q_out, "q_out", dt, dev, T, Hq, d)
    f = _lib().gdn_rotary
    a = (q.data_ptr(), kp, q_out.data_ptr(), kop, positions.data_ptr(), inv_freq.data_ptr(), T, Hq, Hk, d,
         2 * half, ldq, ldk, ldqo, ldko, 1 if interleaved else 0, 1 if inverse else 0, scale, _DT[dt],
         _current_stream(dev))
    rc = f(*a) if dev == _current_device() else _launch(dev, f, a)
    if rc:
        _check(rc, "gdn_rotary")
    return q_out, k_out


_ROTARY = {"plain": _abi.GDN_ROTARY_PLAIN, "linear": _abi.GDN_ROTARY_LINEAR,
           "ntk": _abi.GDN_ROTARY_NTK, "yarn": _abi.GDN_ROTARY_YARN}


def gdn_rotary_inv_freq(rotary_dim, base=10000.0, scaling="plain", factor=1.0, original_context=0,
                        beta_fast=32.0, beta_slow=1.0):
    """The frequencies of gdn_rotary, [rotary_dim / 2] fp32 on the host, and its scale; scaling is
    "plain", "linear", "ntk" or "yarn" (see include/gdn.h)."""
    f = torch.empty(max(0, rotary_dim // 2), dtype=torch.float32)
    s = ctypes.c_float(0)
    if scaling not in _ROTARY:
        raise ValueError(f"scaling must be one of {sorted(_ROTARY)}")
    _check(_lib().gdn_rotary_inv_freq(int(rotary_dim), float(base), _ROTARY[scaling], float(factor),
                                      int(original_context), float(beta_fast), float(beta_slow),
                                      ctypes.cast(f.data_ptr(), ctypes.POINTER(ctypes.c_float)),
                                      ctypes.byref(s)), "gdn_rotary_inv_freq")
    return f, float(s.value)


def _rows(x, w, name):
    """Checks x [..., C] and w [C]; returns (dtype, device, shape, C, rows)."""
    dt = _dtype(x, name)
    dev, shape = x.get_device(), x.shape
    C = shape[-1]
    if C > _INT_MAX:
        _too_large("the last axis", C)
    _want(x, name, dt, shape, dev)
    _want(w, "w", torch.float32, (C,), dev)
    return dt, dev, shape, C, x.numel() // C if C else 0


def _like(t, name, x, make):
    """An optional output like x: checked, or made where it is wanted."""
    if t is not None:
        _want(t, name, x.dtype, x.shape, x.get_device())
    elif make:
        t = torch.empty_like(x)
    return t


def gdn_add_rmsnorm(x, residual, w, eps=1e-6, o=None, h=None, stream=None):
    """h = x + residual, o = (1 + w) h / sqrt(mean(h^2) + eps) over the last axis: x, residual
    [..., C] (bf16 or fp32; residual None: h = x and is not written), w [C] fp32.  h may be x or
    residual, o may be x.  Returns (o, h), and h = None where o is x and nothing else holds h."""
    if stream is not None:
        return _on(stream, gdn_add_rmsnorm, locals())
    dt, dev, shape, C, rows = _rows(x, w, "x")
    if residual is not None:
        _want(residual, "residual", dt, shape, dev)
    o = _like(o, "o", x, True)
    h = _like(h, "h", x, residual is not None)
    f = _lib().gdn_add_rmsnorm
    a = (x.data_ptr(), _ptr(residual), w.data_ptr(), o.data_ptr(), _ptr(h), rows, C, _DT[dt], eps,
         _current_stream(dev))
    rc = f(*a) if dev == _current_device() else _launch(dev, f, a)
    if rc:
        _check(rc, "gdn_add_rmsnorm")
    if h is None and (o.data_ptr() != x.data_ptr() or rows == 0):
        h = x
    return o, h


def gdn_add_rmsnorm_fp8(x, residual, w, eps=1e-6, group=0, o=None, scales=None, h=None,
                        stream=None):
    """gdn_add_rmsnorm with an 8-bit o (float8_e4m3fn) and fp32 scales [..., C / group]: scale =
    max|o| / 448 over each group of columns, group 0 (a whole row) or 128.  Returns (o, scales, h)."""
    if stream is not None:
        return _on(stream, gdn_add_rmsnorm_fp8, locals())
    dt, dev, shape, C, rows = _rows(x, w, "x")
    if residual is not None:
        _want(residual, "residual", dt, shape, dev)
    group = C if group == 0 else group
    if group < 1 or C % group:
        raise ValueError(f"group {group} does not divide {C} columns")
    if o is None:
        o = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    else:
        _want(o, "o", torch.float8_e4m3fn, shape, dev)
    scales = _states(scales, "scales", (*shape[:-1], C // group), dev, True)
    h = _like(h, "h", x, residual is not None)
    f = _lib().gdn_add_rmsnorm_fp8
    a = (x.data_ptr(), _ptr(residual), w.data_ptr(), o.data_ptr(), scales.data_ptr(), _ptr(h), rows, C, group,
         _DT[dt], eps, _current_stream(dev))
    rc = f(*a) if dev == _current_device() else _launch(dev, f, a)
    if rc:
        _check(rc, "gdn_add_rmsnorm_fp8")
    return o, scales, x if h is None else h


@functools.lru_cache(maxsize=1024)
def _norm_ws_bytes(rows, C):
    return gdn_workspace_bytes(_abi.GDN_OP_ADD_RMSNORM_BACKWARD, 1, rows, 1, C, C) if rows else 0


def gdn_add_rmsnorm_backward(h, w, d_o, d_h=None, eps=1e-6, ws=None, stream=None):
    """Gradients of gdn_add_rmsnorm from the stored h, given d_o and d_h (the gradient of h itself;
    None = 0).  Returns dict dx (like h: the gradient of x and of residual) and dw [C]."""
    if stream is not None:
        return _on(stream, gdn_add_rmsnorm_backward, locals())
    dt, dev, shape, C, rows = _rows(h, w, "h")
    _want(d_o, "d_o", dt, shape, dev)
    if d_h is not None:
        _want(d_h, "d_h", dt, shape, dev)
    dx, dw = torch.empty_like(h), torch.empty_like(w)
    ws, wsp, wsb = _scratch(_norm_ws_bytes(rows, C), ws, dev)
    f = _lib().gdn_add_rmsnorm_backward
    a = (h.data_ptr(), w.data_ptr(), d_o.data_ptr(), _ptr(d_h), dx.data_ptr(), dw.data_ptr(), rows, C, _DT[dt],
         eps, wsp, wsb, _current_stream(dev))
    rc = f(*a) if dev == _current_device() else _launch(dev, f, a)
    if rc:
        _check(rc, "gdn_add_rmsnorm_backward")
    return dict(dx=dx, dw=dw)
