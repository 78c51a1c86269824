"""Python binding of the KLA C ABI (include/kla.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libkla.so.  Tensors must live on the current CUDA device; outputs
are allocated here with torch (the library itself never allocates).
"""
from __future__ import annotations

import contextlib
from typing import Optional, Tuple

import torch

from . import _native

KLA_BF16, KLA_FP32 = 0, 1
CHUNK = 64
_DT = {torch.bfloat16: KLA_BF16, torch.float32: KLA_FP32}


class KLAError(RuntimeError):
    """A non-OK kla_status returned by the library."""

    def __init__(self, status: int, where: str):
        msg = _native.lib().kla_status_string(status).decode()
        super().__init__("%s: %s (status %d)" % (where, msg, status))
        self.status = status


def _check(status: int, where: str):
    if status != 0:
        raise KLAError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype=None, shape=None, dev=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dev is not None and t.device != dev:
        raise ValueError("%s is on %s, the call's other tensors on %s" % (name, t.device, dev))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


@contextlib.contextmanager
def _on(ref, stream):
    """Device and stream of one call: ``ref``'s device is made current (the
    library sizes its TMA maps and error word for the current device) and
    ``stream`` (default: that device's current stream) becomes torch's
    current stream, so every temporary allocated inside (outputs,
    workspaces) belongs to the stream the kernels run on.  The caching
    allocator then only reuses a freed temporary for work ordered after
    those kernels.  Yields the raw stream handle for the C call."""
    _need(ref, "q")
    dev = ref.device
    with torch.cuda.device(dev):
        s = torch.cuda.current_stream(dev) if stream is None else stream
        if s.device != dev:
            raise ValueError("stream is on %s, the tensors on %s" % (s.device, dev))
        with torch.cuda.stream(s):
            yield s.cuda_stream


def chunk_fwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int,
                             dtype: torch.dtype = torch.bfloat16) -> int:
    return int(_native.lib().kla_chunk_fwd_workspace_size(B, T, H, dk, dv, _DT[dtype]))


def chunk_fwd_segments(B: int, T: int, H: int, dk: int, dv: int,
                       dtype: torch.dtype = torch.bfloat16, ws_bytes: Optional[int] = None) -> int:
    """Segments the bf16 state chain runs in (1 = uncut, 0 = not the chunk
    path); ws_bytes defaults to the full workspace size."""
    if ws_bytes is None:
        ws_bytes = chunk_fwd_workspace_size(B, T, H, dk, dv, dtype)
    return int(_native.lib().kla_chunk_fwd_segments(B, T, H, dk, dv, _DT[dtype], ws_bytes))


def chunk_fwd_single_launch(B: int, T: int, H: int, dk: int, dv: int,
                            dtype: torch.dtype = torch.bfloat16,
                            ws_bytes: Optional[int] = None) -> bool:
    """Whether the bf16 prefill of this shape runs as one kernel launch
    (kla_chunk_fwd_single_launch); ws_bytes defaults to the full workspace
    size.  False for every shape at present: the single launch is built but
    not taken."""
    if ws_bytes is None:
        ws_bytes = chunk_fwd_workspace_size(B, T, H, dk, dv, dtype)
    return bool(_native.lib().kla_chunk_fwd_single_launch(B, T, H, dk, dv, _DT[dtype],
                                                          ws_bytes))


def _prefill_args(q, k, v, g, eta, h0, o, hT, return_state):
    _need(q, "q")
    if q.dtype not in _DT:
        raise ValueError("q, k, v must be bfloat16 or float32")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    d = q.device
    _need(k, "k", q.dtype, (B, T, H, dk), d)
    _need(v, "v", q.dtype, (B, T, H, dv), d)
    _need(g, "g", torch.float32, (B, T, H), d)
    _need(eta, "eta", torch.float32, (B, T, H), d)
    _need(h0, "h0", torch.float32, (B, H, dk, dv), d)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=d)
    _need(o, "o", q.dtype, (B, T, H, dv), d)
    if hT is None and return_state:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=d)
    _need(hT, "hT", torch.float32, (B, H, dk, dv), d)
    return B, T, H, dk, dv, o, hT


def chunk_fwd(q, k, v, g, eta, eps: float = 1e-6, h0=None, *, o=None, hT=None,
              return_state: bool = True, workspace=None,
              stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunkwise KLA prefill (kla_chunk_fwd).  Returns (o, hT)."""
    with _on(q, stream) as s:
        B, T, H, dk, dv, o, hT = _prefill_args(q, k, v, g, eta, h0, o, hT, return_state)
        need = chunk_fwd_workspace_size(B, T, H, dk, dv, q.dtype)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        _need(workspace, "workspace", torch.uint8, dev=q.device)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        st = _native.lib().kla_chunk_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(eta), float(eps), _ptr(h0),
            _ptr(o), _ptr(hT), B, T, H, dk, dv, CHUNK, _DT[q.dtype], _ptr(workspace),
            ws_bytes, s)
    _check(st, "kla_chunk_fwd")
    return o, hT


def chunk_fwd_states(q, k, v, g, eta, eps: float = 1e-6, h0=None, *, outputs: bool = True,
                     workspace=None, stream=None):
    """bf16 chunk prefill that also returns the state at the start of every
    chunk (kla_chunk_fwd_states).  Returns (o, hT, hs) with hs
    [B, H, ceil(T / 64), dk, dv] fp32; o and hT are None if not outputs."""
    with _on(q, stream) as s:
        B, T, H, dk, dv, o, hT = _prefill_args(q, k, v, g, eta, h0, None, None, outputs)
        if not outputs:
            o = None
        hs = torch.empty((B, H, (T + CHUNK - 1) // CHUNK, dk, dv), dtype=torch.float32,
                         device=q.device)
        need = chunk_fwd_workspace_size(B, T, H, dk, dv, q.dtype)
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
        _need(workspace, "workspace", torch.uint8, dev=q.device)
        ws_bytes = workspace.numel() * workspace.element_size()
        st = _native.lib().kla_chunk_fwd_states(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(eta), float(eps), _ptr(h0), _ptr(o),
            _ptr(hT), _ptr(hs), B, T, H, dk, dv, _DT[q.dtype], _ptr(workspace), ws_bytes, s)
    _check(st, "kla_chunk_fwd_states")
    return o, hT, hs


def _workspace(workspace, B, T, H, dk, dv, dtype, device):
    need = chunk_fwd_workspace_size(B, T, H, dk, dv, dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    _need(workspace, "workspace", torch.uint8, dev=device)
    return workspace, workspace.numel() * workspace.element_size()


def chunk_ut_transform(k, g, eta, eps: float = 1e-6, *, workspace=None, stream=None):
    """First stage of the bf16 chunk prefill (kla_chunk_ut_transform): the
    per-chunk factors T diag(beta), T diag(beta e^G) into the workspace,
    which is returned."""
    _need(k, "k", torch.bfloat16)
    B, T, H, dk = k.shape
    _need(g, "g", torch.float32, (B, T, H), k.device)
    _need(eta, "eta", torch.float32, (B, T, H), k.device)
    with _on(k, stream) as s:
        workspace, ws_bytes = _workspace(workspace, B, T, H, dk, dk, k.dtype, k.device)
        st = _native.lib().kla_chunk_ut_transform(
            _ptr(k), _ptr(g), _ptr(eta), float(eps), B, T, H, dk, KLA_BF16, _ptr(workspace),
            ws_bytes, s)
    _check(st, "kla_chunk_ut_transform")
    return workspace


def chunk_ut_bound_check(k, g, eta, eps: float = 1e-6, *, workspace=None, stream=None):
    """kla_chunk_ut_transform with the debug check of its factors
    (kla_chunk_ut_bound_check).  Returns (workspace, ratio_max) with
    ratio_max a one-element fp32 CUDA tensor: the largest ratio of
    |T_rs| ||k_r|| / ||k_s|| to eta'_r e^{G_r - G_s} over the factors'
    entries.  A ratio above 1.25 also sets the device error word
    (check_device_error then raises KLAError with KLA_ERR_BOUND)."""
    _need(k, "k", torch.bfloat16)
    B, T, H, dk = k.shape
    _need(g, "g", torch.float32, (B, T, H), k.device)
    _need(eta, "eta", torch.float32, (B, T, H), k.device)
    with _on(k, stream) as s:
        workspace, ws_bytes = _workspace(workspace, B, T, H, dk, dk, k.dtype, k.device)
        ratio = torch.empty(4, dtype=torch.float32, device=k.device)  # 16-byte aligned
        st = _native.lib().kla_chunk_ut_bound_check(
            _ptr(k), _ptr(g), _ptr(eta), float(eps), B, T, H, dk, KLA_BF16, _ptr(workspace),
            ws_bytes, _ptr(ratio), s)
    _check(st, "kla_chunk_ut_bound_check")
    return workspace, ratio[:1]


def chunk_state_fwd(q, k, v, g, workspace, h0=None, *, o=None, hT=None,
                    return_state: bool = True, stream=None):
    """Second stage of the bf16 chunk prefill (kla_chunk_state_fwd): the
    state recurrence and outputs from a workspace made by chunk_ut_transform
    of the same k and g.  Returns (o, hT)."""
    with _on(q, stream) as s:
        B, T, H, dk, dv, o, hT = _prefill_args(q, k, v, g, g, h0, o, hT, return_state)
        if workspace is None:
            raise ValueError("workspace must be a CUDA tensor")
        _need(workspace, "workspace", torch.uint8, dev=q.device)
        ws_bytes = workspace.numel() * workspace.element_size()
        st = _native.lib().kla_chunk_state_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(h0), _ptr(o), _ptr(hT), B, T, H, dk, dv,
            _DT[q.dtype], _ptr(workspace), ws_bytes, s)
    _check(st, "kla_chunk_state_fwd")
    return o, hT


def recurrent_fwd(q, k, v, g, eta, eps: float = 1e-6, h0=None, *, o=None, hT=None,
                  return_state: bool = True, stream=None):
    """Token-serial KLA prefill on CUDA cores (kla_recurrent_fwd)."""
    with _on(q, stream) as s:
        B, T, H, dk, dv, o, hT = _prefill_args(q, k, v, g, eta, h0, o, hT, return_state)
        st = _native.lib().kla_recurrent_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(eta), float(eps), _ptr(h0),
            _ptr(o), _ptr(hT), B, T, H, dk, dv, _DT[q.dtype], s)
    _check(st, "kla_recurrent_fwd")
    return o, hT


def recurrent_bwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int) -> int:
    return int(_native.lib().kla_recurrent_bwd_workspace_size(B, T, H, dk, dv))


def kda_recurrent_bwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int) -> int:
    return int(_native.lib().kla_kda_recurrent_bwd_workspace_size(B, T, H, dk, dv))


def chunk_bwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int,
                             dtype: torch.dtype = torch.bfloat16) -> int:
    return int(_native.lib().kla_chunk_bwd_workspace_size(B, T, H, dk, dv, _DT[dtype]))


def _bwd(fn, name, q, k, v, g, step, eps, h0, grad_o, grad_hT, need_h0, workspace, stream,
         vector_gate=False, chunked=False):
    _need(q, "q")
    if q.dtype not in _DT:
        raise ValueError("q, k, v must be bfloat16 or float32")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    d = q.device
    _need(k, "k", q.dtype, (B, T, H, dk), d)
    _need(v, "v", q.dtype, (B, T, H, dv), d)
    gshape = (B, T, H, dk) if vector_gate else (B, T, H)
    _need(g, "g", torch.float32, gshape, d)
    _need(step, "eta/beta", torch.float32, (B, T, H), d)
    _need(h0, "h0", torch.float32, (B, H, dk, dv), d)
    _need(grad_o, "grad_o", q.dtype, (B, T, H, dv), d)
    _need(grad_hT, "grad_hT", torch.float32, (B, H, dk, dv), d)
    with _on(q, stream) as s:
        return _bwd_launch(fn, name, q, k, v, g, step, eps, h0, grad_o, grad_hT, need_h0,
                           workspace, s, gshape, vector_gate, chunked)


def _bwd_launch(fn, name, q, k, v, g, step, eps, h0, grad_o, grad_hT, need_h0, workspace, s,
                gshape, vector_gate, chunked):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    f32 = dict(dtype=torch.float32, device=q.device)
    out = dict(dq=torch.empty((B, T, H, dk), **f32), dk=torch.empty((B, T, H, dk), **f32),
               dv=torch.empty((B, T, H, dv), **f32), dg=torch.empty(gshape, **f32),
               dstep=torch.empty((B, T, H), **f32),
               dh0=torch.empty((B, H, dk, dv), **f32) if need_h0 else None)
    if chunked:
        need = chunk_bwd_workspace_size(B, T, H, dk, dv, q.dtype)
    else:
        need = (kda_recurrent_bwd_workspace_size if vector_gate
                else recurrent_bwd_workspace_size)(B, T, H, dk, dv)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _need(workspace, "workspace", torch.uint8, dev=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(step)]
    if eps is not None:
        args.append(float(eps))
    args += [_ptr(h0), _ptr(grad_o), _ptr(grad_hT), _ptr(out["dq"]), _ptr(out["dk"]),
             _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dstep"]), _ptr(out["dh0"]),
             B, T, H, dk, dv, _DT[q.dtype], _ptr(workspace), ws_bytes, s]
    _check(fn(*args), name)
    return out


def recurrent_bwd(q, k, v, g, eta, grad_o, eps: float = 1e-6, h0=None, grad_hT=None, *,
                  need_h0: bool = True, workspace=None, stream=None):
    """Gradients of the KLA prefill for dL/do = grad_o and dL/dh_T = grad_hT
    (None = 0), token-serial fp32 (kla_recurrent_bwd).  Returns a dict of
    fp32 tensors dq, dk, dv, dg, deta, dh0 (None unless need_h0)."""
    out = _bwd(_native.lib().kla_recurrent_bwd, "kla_recurrent_bwd", q, k, v, g, eta, eps, h0,
               grad_o, grad_hT, need_h0, workspace, stream)
    out["deta"] = out.pop("dstep")
    return out


def chunk_bwd(q, k, v, g, eta, grad_o, eps: float = 1e-6, h0=None, grad_hT=None, *,
              need_h0: bool = True, workspace=None, stream=None):
    """Gradients of the KLA prefill from the chunk form (kla_chunk_bwd):
    dq, dk, dv, dg, deta, dh0 (fp32).  bf16 with d = 128 runs the chunkwise
    tensor-core kernels, everything else the token-serial ones."""
    out = _bwd(_native.lib().kla_chunk_bwd, "kla_chunk_bwd", q, k, v, g, eta, eps, h0, grad_o,
               grad_hT, need_h0, workspace, stream, chunked=True)
    out["deta"] = out.pop("dstep")
    return out


def gdn_chunk_bwd(q, k, v, g, beta, grad_o, h0=None, grad_hT=None, *, need_h0: bool = True,
                  workspace=None, stream=None):
    """The same with beta given per token (kla_gdn_chunk_bwd)."""
    out = _bwd(_native.lib().kla_gdn_chunk_bwd, "kla_gdn_chunk_bwd", q, k, v, g, beta, None, h0,
               grad_o, grad_hT, need_h0, workspace, stream, chunked=True)
    out["dbeta"] = out.pop("dstep")
    return out


def kda_recurrent_bwd(q, k, v, g, eta, grad_o, eps: float = 1e-6, h0=None, grad_hT=None, *,
                      need_h0: bool = True, workspace=None, stream=None):
    """Gradients of the per-channel-gate prefill (g [B,T,H,dk]), KLA step
    size (kla_kda_recurrent_bwd): dq, dk, dv, dg [B,T,H,dk], deta, dh0."""
    out = _bwd(_native.lib().kla_kda_recurrent_bwd, "kla_kda_recurrent_bwd", q, k, v, g, eta,
               eps, h0, grad_o, grad_hT, need_h0, workspace, stream, vector_gate=True)
    out["deta"] = out.pop("dstep")
    return out


def kda_recurrent_bwd_beta(q, k, v, g, beta, grad_o, h0=None, grad_hT=None, *,
                           need_h0: bool = True, workspace=None, stream=None):
    """The same with beta given per token (kla_kda_recurrent_bwd_beta):
    dq, dk, dv, dg, dbeta, dh0."""
    out = _bwd(_native.lib().kla_kda_recurrent_bwd_beta, "kla_kda_recurrent_bwd_beta", q, k, v,
               g, beta, None, h0, grad_o, grad_hT, need_h0, workspace, stream, vector_gate=True)
    out["dbeta"] = out.pop("dstep")
    return out


def gdn_recurrent_bwd(q, k, v, g, beta, grad_o, h0=None, grad_hT=None, *, need_h0: bool = True,
                      workspace=None, stream=None):
    """Gradients of the gated delta rule prefill (beta given per token):
    dq, dk, dv, dg, dbeta, dh0 (kla_gdn_recurrent_bwd)."""
    out = _bwd(_native.lib().kla_gdn_recurrent_bwd, "kla_gdn_recurrent_bwd", q, k, v, g, beta,
               None, h0, grad_o, grad_hT, need_h0, workspace, stream)
    out["dbeta"] = out.pop("dstep")
    return out


def decode_step(q, k, v, g, eta, S, eps: float = 1e-6, *, o=None, stream=None):
    """One decode token per sequence; S [B,H,dk,dv] fp32 is updated in place.
    Returns o [B,H,dv]."""
    _need(q, "q")
    if q.dtype not in _DT:
        raise ValueError("q, k, v must be bfloat16 or float32")
    B, H, dk = q.shape
    dv = v.shape[-1]
    d = q.device
    _need(k, "k", q.dtype, (B, H, dk), d)
    _need(v, "v", q.dtype, (B, H, dv), d)
    _need(g, "g", torch.float32, (B, H), d)
    _need(eta, "eta", torch.float32, (B, H), d)
    _need(S, "S", torch.float32, (B, H, dk, dv), d)
    with _on(q, stream) as s:
        if o is None:
            o = torch.empty((B, H, dv), dtype=q.dtype, device=d)
        _need(o, "o", q.dtype, (B, H, dv), d)
        st = _native.lib().kla_decode_step(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(eta), float(eps), _ptr(S), _ptr(o),
            B, H, dk, dv, _DT[q.dtype], s)
    _check(st, "kla_decode_step")
    return o


def gdn_chunk_fwd(q, k, v, g, beta, h0=None, *, o=None, hT=None, return_state: bool = True,
                  workspace=None, stream=None):
    """Gated DeltaNet prefill (kla_gdn_chunk_fwd): beta [B,T,H] fp32 is the
    step size itself.  Returns (o, hT)."""
    with _on(q, stream) as s:
        B, T, H, dk, dv, o, hT = _prefill_args(q, k, v, g, beta, h0, o, hT, return_state)
        need = chunk_fwd_workspace_size(B, T, H, dk, dv, q.dtype)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        _need(workspace, "workspace", torch.uint8, dev=q.device)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        st = _native.lib().kla_gdn_chunk_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT),
            B, T, H, dk, dv, CHUNK, _DT[q.dtype], _ptr(workspace), ws_bytes, s)
    _check(st, "kla_gdn_chunk_fwd")
    return o, hT


def gdn_decode_step(q, k, v, g, beta, S, *, o=None, stream=None):
    """One Gated DeltaNet decode token per sequence (kla_gdn_decode_step);
    S is updated in place.  Returns o [B,H,dv]."""
    _need(q, "q")
    if q.dtype not in _DT:
        raise ValueError("q, k, v must be bfloat16 or float32")
    B, H, dk = q.shape
    dv = v.shape[-1]
    d = q.device
    _need(k, "k", q.dtype, (B, H, dk), d)
    _need(v, "v", q.dtype, (B, H, dv), d)
    _need(g, "g", torch.float32, (B, H), d)
    _need(beta, "beta", torch.float32, (B, H), d)
    _need(S, "S", torch.float32, (B, H, dk, dv), d)
    with _on(q, stream) as s:
        if o is None:
            o = torch.empty((B, H, dv), dtype=q.dtype, device=d)
        _need(o, "o", q.dtype, (B, H, dv), d)
        st = _native.lib().kla_gdn_decode_step(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(o), B, H, dk, dv,
            _DT[q.dtype], s)
    _check(st, "kla_gdn_decode_step")
    return o


def _need_host(t, name, dtype, shape):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise ValueError("%s must be a host (CPU) tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be %s of shape %s" % (name, dtype, tuple(shape)))


def chunk_fwd_host_staging_size(B: int, T: int, H: int, dk: int, dv: int,
                                dtype: torch.dtype = torch.bfloat16) -> int:
    return int(_native.lib().kla_chunk_fwd_host_staging_size(B, T, H, dk, dv, _DT[dtype]))


def chunk_fwd_host(q, k, v, g, eta, eps: float = 1e-6, h0=None, *, o=None, hT=None,
                   return_state: bool = True, staging=None, device=None, stream=None):
    """Prefill from host tensors (kla_chunk_fwd_host): the copies to and
    from the device are pipelined against the kernels.  Inputs and outputs
    are CPU tensors (pin them for the copies to overlap; outputs allocated
    here are pinned).  Only enqueues work: synchronise ``stream`` before
    reading o, hT.  Returns (o, hT)."""
    if q.dtype not in _DT:
        raise ValueError("q, k, v must be bfloat16 or float32")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    for t, n, dt, sh in ((q, "q", q.dtype, (B, T, H, dk)), (k, "k", q.dtype, (B, T, H, dk)),
                         (v, "v", q.dtype, (B, T, H, dv)), (g, "g", torch.float32, (B, T, H)),
                         (eta, "eta", torch.float32, (B, T, H)),
                         (h0, "h0", torch.float32, (B, H, dk, dv))):
        _need_host(t, n, dt, sh)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, pin_memory=True)
    _need_host(o, "o", q.dtype, (B, T, H, dv))
    if hT is None and return_state:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, pin_memory=True)
    _need_host(hT, "hT", torch.float32, (B, H, dk, dv))
    if device is None:
        device = staging.device if staging is not None else (
            stream.device if stream is not None else
            torch.device("cuda", torch.cuda.current_device()))
    dev = torch.device(device)
    need = chunk_fwd_host_staging_size(B, T, H, dk, dv, q.dtype)
    with torch.cuda.device(dev):
        s = torch.cuda.current_stream(dev) if stream is None else stream
        if s.device != dev:
            raise ValueError("stream is on %s, the staging buffer on %s" % (s.device, dev))
        with torch.cuda.stream(s):
            if staging is None:
                staging = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
            _need(staging, "staging", torch.uint8, dev=dev)
            st = _native.lib().kla_chunk_fwd_host(
                _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(eta), float(eps), _ptr(h0), _ptr(o),
                _ptr(hT), B, T, H, dk, dv, _DT[q.dtype], _ptr(staging),
                staging.numel() * staging.element_size(), s.cuda_stream)
    _check(st, "kla_chunk_fwd_host")
    return o, hT


def _kda_prefill(fn, name, q, k, v, g, step, eps, h0, o, hT, return_state, stream):
    # the per-token arguments as for chunk_fwd; g is checked on its own
    with _on(q, stream) as s:
        B, T, H, dk, dv, o, hT = _prefill_args(q, k, v, None, step, h0, o, hT, return_state)
        if g is None:
            raise ValueError("g must be a CUDA tensor")
        _need(g, "g", torch.float32, (B, T, H, dk), q.device)
        args = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(step)]
        if eps is not None:
            args.append(float(eps))
        st = fn(*args, _ptr(h0), _ptr(o), _ptr(hT), B, T, H, dk, dv, _DT[q.dtype], s)
    _check(st, name)
    return o, hT


def kda_fwd(q, k, v, g, eta, eps: float = 1e-6, h0=None, *, o=None, hT=None,
            return_state: bool = True, stream=None):
    """KLA prefill with a per-channel gate (kla_kda_fwd): g [B,T,H,dk] fp32,
    one log-gate per key channel.  Returns (o, hT)."""
    return _kda_prefill(_native.lib().kla_kda_fwd, "kla_kda_fwd", q, k, v, g, eta, eps, h0,
                        o, hT, return_state, stream)


def kda_fwd_beta(q, k, v, g, beta, h0=None, *, o=None, hT=None, return_state: bool = True,
                 stream=None):
    """Per-channel-gated prefill with beta given per token (kla_kda_fwd_beta)."""
    return _kda_prefill(_native.lib().kla_kda_fwd_beta, "kla_kda_fwd_beta", q, k, v, g, beta,
                        None, h0, o, hT, return_state, stream)


def kda_chunk_fwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int,
                                 dtype: torch.dtype = torch.bfloat16) -> int:
    return int(_native.lib().kla_kda_chunk_fwd_workspace_size(B, T, H, dk, dv, _DT[dtype]))


def _kda_chunk(fn, name, q, k, v, g, step, eps, h0, o, hT, return_state, workspace, stream):
    with _on(q, stream) as s:
        B, T, H, dk, dv, o, hT = _prefill_args(q, k, v, None, step, h0, o, hT, return_state)
        if g is None:
            raise ValueError("g must be a CUDA tensor")
        _need(g, "g", torch.float32, (B, T, H, dk), q.device)
        need = kda_chunk_fwd_workspace_size(B, T, H, dk, dv, q.dtype)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        _need(workspace, "workspace", torch.uint8, dev=q.device)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        args = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(step)]
        if eps is not None:
            args.append(float(eps))
        st = fn(*args, _ptr(h0), _ptr(o), _ptr(hT), B, T, H, dk, dv, CHUNK, _DT[q.dtype],
                _ptr(workspace), ws_bytes, s)
    _check(st, name)
    return o, hT


def kda_chunk_fwd(q, k, v, g, eta, eps: float = 1e-6, h0=None, *, o=None, hT=None,
                  return_state: bool = True, workspace=None, stream=None):
    """Per-channel-gate prefill as chunks (kla_kda_chunk_fwd): g [B,T,H,dk]
    fp32.  bf16 runs the tensor-core chunk path.  Returns (o, hT)."""
    return _kda_chunk(_native.lib().kla_kda_chunk_fwd, "kla_kda_chunk_fwd", q, k, v, g, eta,
                      eps, h0, o, hT, return_state, workspace, stream)


def kda_chunk_fwd_beta(q, k, v, g, beta, h0=None, *, o=None, hT=None, return_state: bool = True,
                       workspace=None, stream=None):
    """kda_chunk_fwd with beta given per token (kla_kda_chunk_fwd_beta)."""
    return _kda_chunk(_native.lib().kla_kda_chunk_fwd_beta, "kla_kda_chunk_fwd_beta", q, k, v,
                      g, beta, None, h0, o, hT, return_state, workspace, stream)


def _kda_decode(fn, name, q, k, v, g, step, eps, S, o, stream):
    _need(q, "q")
    if q.dtype not in _DT:
        raise ValueError("q, k, v must be bfloat16 or float32")
    B, H, dk = q.shape
    dv = v.shape[-1]
    d = q.device
    _need(k, "k", q.dtype, (B, H, dk), d)
    _need(v, "v", q.dtype, (B, H, dv), d)
    _need(g, "g", torch.float32, (B, H, dk), d)
    _need(step, "eta" if eps is not None else "beta", torch.float32, (B, H), d)
    _need(S, "S", torch.float32, (B, H, dk, dv), d)
    with _on(q, stream) as s:
        if o is None:
            o = torch.empty((B, H, dv), dtype=q.dtype, device=d)
        _need(o, "o", q.dtype, (B, H, dv), d)
        args = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(step)]
        if eps is not None:
            args.append(float(eps))
        st = fn(*args, _ptr(S), _ptr(o), B, H, dk, dv, _DT[q.dtype], s)
    _check(st, name)
    return o


def kda_decode_step(q, k, v, g, eta, S, eps: float = 1e-6, *, o=None, stream=None):
    """One per-channel-gated decode token (kla_kda_decode_step): g [B,H,dk];
    S is updated in place.  Returns o [B,H,dv]."""
    return _kda_decode(_native.lib().kla_kda_decode_step, "kla_kda_decode_step", q, k, v, g,
                       eta, eps, S, o, stream)


def kda_decode_step_beta(q, k, v, g, beta, S, *, o=None, stream=None):
    """Per-channel-gated decode token with beta given (kla_kda_decode_step_beta)."""
    return _kda_decode(_native.lib().kla_kda_decode_step_beta, "kla_kda_decode_step_beta",
                       q, k, v, g, beta, None, S, o, stream)


# ---------------------------------------------------------------------------
# Layer operators around the recurrences: short causal convolution, selective
# state space scan, norm and rotation of queries and keys.

# The current device, and the handle of a device's current stream without the
# Stream object around it.  (Both are asked for after a CUDA tensor was seen, so
# CUDA is initialised.)
_this_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """_on for calls of a few microseconds: no context is entered when the
    tensors' device and its current stream are the ones to use anyway."""

    __slots__ = ("dev", "stream", "ctx")

    def __init__(self, ref, stream):
        self.dev, self.stream, self.ctx = ref.device, stream, None

    def __enter__(self):
        if self.stream is None and _this_device() == self.dev.index:
            return _raw_stream(self.dev.index)
        with contextlib.ExitStack() as stack:
            stack.enter_context(torch.cuda.device(self.dev))
            s = torch.cuda.current_stream(self.dev) if self.stream is None else self.stream
            if s.device != self.dev:
                raise ValueError("stream is on %s, the tensors on %s" % (s.device, self.dev))
            stack.enter_context(torch.cuda.stream(s))
            self.ctx = stack.pop_all()
        return s.cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.close()


def _like(t):
    """A new contiguous tensor of t's shape and type."""
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _p(t, name, dtype, shape, dev):
    """Address of a contiguous argument (None stays None); _need's checks, and
    its words where one fails."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == dev.index and t.shape == shape \
                and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # not a tensor
        pass
    _need(t, name, dtype, shape, dev)
    return t.data_ptr()


def _rows(t, name, dtype, lead, inner, dev):
    """Elements between the rows of an input that may be rows of a wider
    matrix: shape lead + inner, inner contiguous, rows evenly spaced."""
    shape = lead + inner
    try:
        good = t.dtype is dtype and t.get_device() == dev.index and t.shape == shape
    except AttributeError:  # not a tensor
        good = False
    if not good:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        if t.device != dev:
            raise ValueError("%s is on %s, the call's other tensors on %s"
                             % (name, t.device, dev))
        if t.dtype is not dtype:
            raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    n = inner[0] if len(inner) == 1 else inner[0] * inner[1]
    if t.is_contiguous() or t.numel() == 0:
        return n
    st = t.stride()
    if (st[-1] != 1 and inner[-1] != 1) or \
            (len(inner) == 2 and st[-2] != inner[1] and inner[0] != 1):
        raise ValueError("%s: the elements of a row must be contiguous" % name)
    if len(lead) == 1:
        ld = st[0] if lead[0] != 1 else n
    else:
        B, T = lead
        ld = st[1] if T != 1 else st[0] if B != 1 else n
        if T != 1 and B != 1 and st[0] != T * ld and ld >= n:
            raise ValueError("%s: rows must be evenly spaced" % name)
    if ld < n:
        raise ValueError("%s: rows must not overlap" % name)
    return ld


_MOST = (1 << 31) - 1


def _head(t, name, dims):
    """Type, device and shape of a call's first tensor."""
    try:
        dt, dev, shape = t.dtype, t.device, tuple(t.shape)
        good = dt in _DT and t.is_cuda
    except AttributeError:  # not a tensor
        good = False
    if not good:
        raise ValueError("%s must be a CUDA tensor of dtype bfloat16 or float32" % name)
    if len(shape) != dims or max(shape) > _MOST:
        raise ValueError("%s must have %d dimensions below 2^31, got %s" % (name, dims, shape))
    return dt, dev, shape


def _scratch(workspace, need, dev):
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev=dev)
    return workspace, workspace.numel()


def conv_bwd_workspace_size(B: int, T: int, D: int, W: int) -> int:
    return int(_native.lib().kla_conv_bwd_workspace_size(B, T, D, W))


def _conv_args(x, w, bias, s0, lengths, lead, D, dt, dev):
    """The width, and the arguments x .. lengths of the C calls."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[0] != D or w.shape[1] < 1:
        raise ValueError("w must be a [D, W] CUDA tensor with D = %d" % D)
    W = w.shape[1]
    ldx = _rows(x, "x", dt, lead, (D,), dev)
    return W, (x.data_ptr(), ldx, _p(w, "w", torch.float32, (D, W), dev),
               _p(bias, "bias", torch.float32, (D,), dev),
               _p(s0, "s0", dt, (lead[0], W - 1, D), dev),
               _p(lengths, "lengths", torch.int32, (lead[0],), dev))


def conv_fwd(x, w, bias=None, s0=None, *, silu: bool = True, lengths=None, y=None, sT=None,
             return_state: bool = True, stream=None):
    """Short causal depthwise convolution of a prompt (kla_conv_fwd): x
    [B,T,D] bf16 or fp32 (rows may be part of a wider matrix), w [D,W] fp32
    with W in {2, 3, 4}, bias [D] fp32, s0 [B,W-1,D] the inputs before x,
    lengths [B] int32.  Returns (y, sT), sT the last W-1 inputs."""
    dt, dev, (B, T, D) = _head(x, "x", 3)
    with _On(x, stream) as s:
        W, args = _conv_args(x, w, bias, s0, lengths, (B, T), D, dt, dev)
        if y is None:
            y = _like(x)
        if sT is None and return_state:
            sT = torch.empty((B, W - 1, D), dtype=dt, device=dev)
        st = _native.lib().kla_conv_fwd(
            *args, _p(y, "y", dt, (B, T, D), dev), _p(sT, "sT", dt, (B, W - 1, D), dev),
            B, T, D, W, bool(silu), _DT[dt], s)
    _check(st, "kla_conv_fwd")
    return y, sT


def conv_bwd(x, w, grad_y, bias=None, s0=None, grad_sT=None, *, silu: bool = True,
             lengths=None, need_s0: bool = True, workspace=None, stream=None):
    """Gradients of conv_fwd for dL/dy = grad_y and dL/dsT = grad_sT (None =
    0) (kla_conv_bwd).  Returns a dict: dx and ds0 in x's type (ds0 None
    unless need_s0), dw and dbias fp32 (dbias None without a bias)."""
    dt, dev, (B, T, D) = _head(x, "x", 3)
    _need_all(grad_y, "grad_y")
    with _On(x, stream) as s:
        W, args = _conv_args(x, w, bias, s0, lengths, (B, T), D, dt, dev)
        pg = _p(grad_y, "grad_y", dt, (B, T, D), dev)
        ps = _p(grad_sT, "grad_sT", dt, (B, W - 1, D), dev)
        f32 = dict(dtype=torch.float32, device=dev)
        out = dict(dx=_like(x),
                   dw=torch.empty((D, W), **f32),
                   dbias=None if bias is None else torch.empty((D,), **f32),
                   ds0=torch.empty((B, W - 1, D), dtype=dt, device=dev) if need_s0 else None)
        workspace, nws = _scratch(workspace, conv_bwd_workspace_size(B, T, D, W), dev)
        st = _native.lib().kla_conv_bwd(
            *args, pg, ps, _ptr(out["dx"]), _ptr(out["dw"]), _ptr(out["dbias"]),
            _ptr(out["ds0"]), B, T, D, W, bool(silu), _DT[dt], _ptr(workspace), nws, s)
    _check(st, "kla_conv_bwd")
    return out


def conv_step(x, w, state, bias=None, *, silu: bool = True, y=None, stream=None):
    """One token of the convolution for each sequence (kla_conv_step): x
    [B,D]; state [B,W-1,D] (conv_fwd's sT) is moved on in place.  Returns y
    [B,D]."""
    dt, dev, (B, D) = _head(x, "x", 2)
    _need_all(state, "state")
    with _On(x, stream) as s:
        W, args = _conv_args(x, w, bias, state, None, (B,), D, dt, dev)
        if y is None:
            y = _like(x)
            py = y.data_ptr()
        else:
            py = _p(y, "y", dt, (B, D), dev)
        st = _native.lib().kla_conv_step(*args[:5], py, B, D, W, bool(silu), _DT[dt], s)
    _check(st, "kla_conv_step")
    return y


def _need_all(t, name):
    if t is None:
        raise ValueError("%s must be a CUDA tensor" % name)


def ssm_fwd_workspace_size(B: int, T: int, D: int, G: int, N: int) -> int:
    return int(_native.lib().kla_ssm_fwd_workspace_size(B, T, D, G, N))


def ssm_bwd_workspace_size(B: int, T: int, D: int, G: int, N: int) -> int:
    return int(_native.lib().kla_ssm_bwd_workspace_size(B, T, D, G, N))


def _ssm_args(u, dt, A, Bm, Cm, D, z, dt_bias, lead, Dn, ty, dev):
    """Groups and states, the row pitches of u, dt, Bm, Cm and z, and the
    addresses of u .. dt_bias, for prompts and single tokens."""
    if not isinstance(A, torch.Tensor) or A.dim() != 2 or A.shape[0] != Dn:
        raise ValueError("A must be a [D, N] CUDA tensor with D = %d" % Dn)
    N = A.shape[1]
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != len(lead) + 2:
        raise ValueError("Bm must be a CUDA tensor of shape [..., G, N]")
    G = Bm.shape[-2]
    ch, gn = (Dn,), (G, N)
    lds = (_rows(u, "u", ty, lead, ch, dev), _rows(dt, "dt", ty, lead, ch, dev),
           _rows(Bm, "Bm", ty, lead, gn, dev), _rows(Cm, "Cm", ty, lead, gn, dev),
           0 if z is None else _rows(z, "z", ty, lead, ch, dev))
    f32 = torch.float32
    return G, N, lds, (
        u.data_ptr(), dt.data_ptr(), _p(A, "A", f32, (Dn, N), dev), Bm.data_ptr(),
        Cm.data_ptr(), _p(D, "D", f32, ch, dev), None if z is None else z.data_ptr(),
        _p(dt_bias, "dt_bias", f32, ch, dev))


def ssm_fwd(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, *, softplus: bool = True,
            lengths=None, y=None, hT=None, return_state: bool = True, workspace=None,
            stream=None):
    """Selective state space scan of a prompt (kla_ssm_fwd): u, dt, z
    [B,T,D], Bm, Cm [B,T,G,N] bf16 or fp32 (rows may be parts of wider
    matrices), A [D,N], D, dt_bias [D], h0 [B,D,N] fp32, lengths [B] int32;
    N in {8, 16, 32, 64}.  Returns (y, hT)."""
    ty, dev, (B, T, Dn) = _head(u, "u", 3)
    f32 = torch.float32
    with _On(u, stream) as s:
        G, N, lds, args = _ssm_args(u, dt, A, Bm, Cm, D, z, dt_bias, (B, T), Dn, ty, dev)
        if y is None:
            y = _like(u)
        if hT is None and return_state:
            hT = torch.empty((B, Dn, N), dtype=f32, device=dev)
        workspace, nws = _scratch(workspace, ssm_fwd_workspace_size(B, T, Dn, G, N), dev)
        st = _native.lib().kla_ssm_fwd(
            *args, _p(h0, "h0", f32, (B, Dn, N), dev),
            _p(lengths, "lengths", torch.int32, (B,), dev), _p(y, "y", ty, (B, T, Dn), dev),
            _p(hT, "hT", f32, (B, Dn, N), dev), B, T, Dn, G, N, *lds, bool(softplus), _DT[ty],
            _ptr(workspace), nws, s)
    _check(st, "kla_ssm_fwd")
    return y, hT


def ssm_bwd(u, dt, A, Bm, Cm, grad_y, D=None, z=None, dt_bias=None, h0=None, grad_hT=None, *,
            softplus: bool = True, lengths=None, need_h0: bool = True, workspace=None,
            stream=None):
    """Gradients of ssm_fwd for dL/dy = grad_y and dL/dhT = grad_hT (None =
    0) (kla_ssm_bwd).  Returns a dict: du, ddt, dB, dC, dz in u's type, dA,
    dD, ddt_bias, dh0 fp32 (None for inputs that are None; dh0 None unless
    need_h0)."""
    ty, dev, (B, T, Dn) = _head(u, "u", 3)
    _need_all(grad_y, "grad_y")
    with _On(u, stream) as s:
        G, N, lds, args = _ssm_args(u, dt, A, Bm, Cm, D, z, dt_bias, (B, T), Dn, ty, dev)
        more = (_p(h0, "h0", torch.float32, (B, Dn, N), dev),
                _p(lengths, "lengths", torch.int32, (B,), dev),
                _p(grad_y, "grad_y", ty, (B, T, Dn), dev),
                _p(grad_hT, "grad_hT", torch.float32, (B, Dn, N), dev))
        f32 = dict(dtype=torch.float32, device=dev)
        out = dict(du=_like(u), ddt=_like(u), dA=_like(A), dB=_like(Bm), dC=_like(Bm),
                   dD=None if D is None else _like(D), dz=None if z is None else _like(u),
                   ddt_bias=None if dt_bias is None else _like(dt_bias),
                   dh0=torch.empty((B, Dn, N), **f32) if need_h0 else None)
        workspace, nws = _scratch(workspace, ssm_bwd_workspace_size(B, T, Dn, G, N), dev)
        st = _native.lib().kla_ssm_bwd(
            *args, *more, *(_ptr(out[k]) for k in ("du", "ddt", "dA", "dB", "dC", "dD", "dz",
                                                   "ddt_bias", "dh0")),
            B, T, Dn, G, N, *lds, bool(softplus), _DT[ty], _ptr(workspace), nws, s)
    _check(st, "kla_ssm_bwd")
    return out


def ssm_step(u, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, *, softplus: bool = True,
             y=None, stream=None):
    """One token of the scan for each sequence (kla_ssm_step): u, dt, z
    [B,D], Bm, Cm [B,G,N]; state [B,D,N] fp32 (ssm_fwd's hT) is moved on in
    place.  Returns y [B,D]."""
    ty, dev, (B, Dn) = _head(u, "u", 2)
    _need_all(state, "state")
    with _On(u, stream) as s:
        G, N, lds, args = _ssm_args(u, dt, A, Bm, Cm, D, z, dt_bias, (B,), Dn, ty, dev)
        if y is None:
            y = _like(u)
            py = y.data_ptr()
        else:
            py = _p(y, "y", ty, (B, Dn), dev)
        st = _native.lib().kla_ssm_step(
            *args, _p(state, "state", torch.float32, (B, Dn, N), dev), py, B, Dn, G, N, *lds, bool(softplus), _DT[ty], s)
    _check(st, "kla_ssm_step")
    return y


_NORMS = {None: 0, "l2": 1, "rms": 2}


def _qk_args(q, k, wq, wk, positions, inv_freq, norm, pos0):
    """Type, device, sizes (B, T, Hq, Hk, d, rot), and the arguments q .. rot of
    the C calls but for pos0, in two parts around it."""
    one = isinstance(q, torch.Tensor) and q.dim() == 3  # a token each: [B, H, d]
    ty, dev, shape = _head(q, "q", 3 if one else 4)
    lead, Hq, d = shape[:-2], shape[-2], shape[-1]
    if not isinstance(k, torch.Tensor) or k.dim() != len(shape):
        raise ValueError("q and k must be CUDA tensors [B, T, H, d] or [B, H, d]")
    Hk = k.shape[-2]
    B, T = lead[0], 1 if one else lead[1]
    ldq, ldk = _rows(q, "q", ty, lead, (Hq, d), dev), _rows(k, "k", ty, lead, (Hk, d), dev)
    if norm not in _NORMS:
        raise ValueError("norm must be None, 'l2' or 'rms', got %r" % (norm,))
    f32 = torch.float32
    stride = rot = 0
    pp = pf = None
    if positions is not None:
        if not isinstance(positions, torch.Tensor):
            raise ValueError("positions must be a CUDA tensor")
        have = tuple(positions.shape)
        if have == lead:
            stride = T
        elif one or have != (T,):
            raise ValueError("positions must have shape %s, got %s"
                             % (lead if one else "%s or %s" % (lead, (T,)), have))
        pp = _p(positions, "positions", torch.int32, have, dev)
    elif not -(1 << 31) <= pos0 <= (1 << 31) - max(T, 1):
        raise ValueError("positions from pos0 = %d on pass 32 bits" % pos0)
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor):
            raise ValueError("inv_freq must be a CUDA tensor")
        rot = 2 * inv_freq.numel()
        pf = _p(inv_freq, "inv_freq", f32, inv_freq.shape, dev)
    return ty, dev, (B, T, Hq, Hk, d, rot), (
        q.data_ptr(), k.data_ptr(), ldq, ldk, _p(wq, "wq", f32, (d,), dev),
        _p(wk, "wk", f32, (d,), dev), pp, stride), (pf, rot)


def qk_norm_bwd_workspace_size(B: int, T: int, Hq: int, Hk: int, d: int, rot: int) -> int:
    return int(_native.lib().kla_qk_norm_bwd_workspace_size(B, T, Hq, Hk, d, rot))


def qk_norm_fwd(q, k, *, wq=None, wk=None, positions=None, inv_freq=None, pos0: int = 0,
                norm: Optional[str] = "l2", eps: float = 1e-6, interleaved: bool = False,
                scale: float = 1.0, oq=None, ok=None, stream=None):
    """Norm of every head of q [B,T,Hq,d] and k [B,T,Hk,d] (or [B,H,d], one
    token of each sequence) and rotation of its first 2 * len(inv_freq)
    channels by position, in one pass (kla_qk_norm_fwd).  norm: "l2", "rms"
    or None; wq, wk [d] fp32; positions int32 [B,T], [T] or (one token) [B],
    None = pos0 + t; inv_freq fp32, None = no rotation.  Returns (oq, ok)."""
    ty, dev, (B, T, Hq, Hk, d, _), head, freq = _qk_args(q, k, wq, wk, positions, inv_freq,
                                                         norm, pos0)
    with _On(q, stream) as s:
        pq, pk = _p(oq, "oq", ty, q.shape, dev), _p(ok, "ok", ty, k.shape, dev)
        if oq is None:
            oq = _like(q)
            pq = oq.data_ptr()
        if ok is None:
            ok = _like(k)
            pk = ok.data_ptr()
        st = _native.lib().kla_qk_norm_fwd(
            *head, pos0, *freq, bool(interleaved), scale, _NORMS[norm], eps,
            pq, pk, B, T, Hq, Hk, d, _DT[ty], s)
    _check(st, "kla_qk_norm_fwd")
    return oq, ok


def qk_norm_bwd(q, k, grad_oq, grad_ok, *, wq=None, wk=None, positions=None, inv_freq=None,
                pos0: int = 0, norm: Optional[str] = "l2", eps: float = 1e-6,
                interleaved: bool = False, scale: float = 1.0, workspace=None, stream=None):
    """Gradients of qk_norm_fwd (kla_qk_norm_bwd).  Returns a dict: dq, dk in
    q's type, dwq, dwk fp32 (None for weights that are None)."""
    ty, dev, (B, T, Hq, Hk, d, rot), head, freq = _qk_args(q, k, wq, wk, positions, inv_freq,
                                                           norm, pos0)
    with _On(q, stream) as s:
        _need_all(grad_oq, "grad_oq")
        _need_all(grad_ok, "grad_ok")
        gq, gk = _p(grad_oq, "grad_oq", ty, q.shape, dev), _p(grad_ok, "grad_ok", ty, k.shape,
                                                              dev)
        out = dict(dq=_like(q), dk=_like(k), dwq=None if wq is None else _like(wq),
                   dwk=None if wk is None else _like(wk))
        need = 0
        if wq is not None or wk is not None:
            need = qk_norm_bwd_workspace_size(B, T, Hq, Hk, d, rot)
        workspace, nws = _scratch(workspace, need, dev)
        st = _native.lib().kla_qk_norm_bwd(
            *head, pos0, *freq, bool(interleaved), scale, _NORMS[norm], eps, gq, gk,
            _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dwq"]), _ptr(out["dwk"]), B, T, Hq, Hk, d, _DT[ty], _ptr(workspace), nws, s)
    _check(st, "kla_qk_norm_bwd")
    return out


def check_device_error(stream=None):
    """Synchronise and raise KLAError if a kernel reported a timed-out wait
    (on the device of ``stream``; default: the current device's current
    stream)."""
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        _check(_native.lib().kla_check_device_error(s.cuda_stream), "kla_check_device_error")
