"""torch.autograd binding of the prefill: forward through kla_chunk_fwd,
backward through kla_chunk_bwd (argument marshalling only; every step of
both runs in the CUDA kernels of libkla.so).

    o, hT = kla_prefill(q, k, v, g, eta, eps=1e-6, h0=None)

q, k, v [B,T,H,d] bf16 or fp32 CUDA tensors, g, eta [B,T,H] fp32, h0
[B,H,dk,dv] fp32 or None.  Gradients flow to q, k, v, g, eta and h0; the
library returns them in fp32 and they are handed to autograd in each
input's dtype.

The layer operators around the recurrence have their differentiable forms
here too: kla_conv (short causal convolution), kla_ssm (selective scan) and
kla_qk_norm (norm and rotation of queries and keys), with gradients to every
tensor input that the formulas depend on smoothly.

A backward pass can be captured into a CUDA graph.  Autograd ties a leaf to
the stream of the first live graph that uses it, so while an eager graph of the
same leaves is alive, capture with leaves of their own (p.detach()
.requires_grad_(), which share the parameters' memory).
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import api


def _given(g, dtype):
    """A gradient as the library takes it (None stays None): of this type,
    contiguous and 16-byte aligned.  Autograd's may be a view that starts at
    any element of another tensor."""
    if g is None:
        return None
    g = g.to(dtype).contiguous()
    return g.clone() if g.data_ptr() % 16 else g


def _or_zeros(g, like):
    return like.new_zeros(like.shape) if g is None else _given(g, like.dtype)


class _KLAPrefill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, eta, h0, eps):
        o, hT = api.chunk_fwd(q, k, v, g, eta, eps, h0)
        ctx.save_for_backward(q, k, v, g, eta, h0)
        ctx.eps = eps
        return o, hT

    @staticmethod
    def backward(ctx, grad_o, grad_hT):
        q, k, v, g, eta, h0 = ctx.saved_tensors
        if grad_o is None:
            grad_o = torch.zeros_like(q[..., :v.shape[-1]])
        r = api.chunk_bwd(q, k, v, g, eta, _given(grad_o, q.dtype), ctx.eps, h0,
                          _given(grad_hT, torch.float32),
                          need_h0=h0 is not None and ctx.needs_input_grad[5])
        dh0 = r["dh0"] if h0 is not None else None
        return (r["dq"].to(q.dtype), r["dk"].to(k.dtype), r["dv"].to(v.dtype), r["dg"],
                r["deta"], dh0, None)


def kla_prefill(q, k, v, g, eta, eps: float = 1e-6, h0=None):
    """Differentiable KLA prefill: returns (o, hT)."""
    return _KLAPrefill.apply(q, k, v, g, eta, h0, eps)


class _KLAConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, s0, lengths, silu):
        y, sT = api.conv_fwd(x, w, bias, s0, silu=silu, lengths=lengths)
        ctx.save_for_backward(x, w, bias, s0, lengths)
        ctx.silu = silu
        ctx.set_materialize_grads(False)
        return y, sT

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_sT):
        x, w, bias, s0, lengths = ctx.saved_tensors
        r = api.conv_bwd(x, w, _or_zeros(grad_y, x), bias, s0, _given(grad_sT, x.dtype),
                         silu=ctx.silu, lengths=lengths,
                         need_s0=s0 is not None and ctx.needs_input_grad[3])
        return r["dx"], r["dw"], r["dbias"], r["ds0"], None, None


def kla_conv(x, w, bias=None, s0=None, *, silu: bool = True, lengths=None):
    """Differentiable short causal convolution (api.conv_fwd): returns
    (y, sT)."""
    return _KLAConv.apply(x, w, bias, s0, lengths, silu)


class _KLASSM(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths, softplus):
        y, hT = api.ssm_fwd(u, dt, A, Bm, Cm, D, z, dt_bias, h0, softplus=softplus,
                            lengths=lengths)
        ctx.save_for_backward(u, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths)
        ctx.softplus = softplus
        ctx.set_materialize_grads(False)
        return y, hT

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_hT):
        u, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths = ctx.saved_tensors
        r = api.ssm_bwd(u, dt, A, Bm, Cm, _or_zeros(grad_y, u), D, z, dt_bias, h0,
                        _given(grad_hT, torch.float32), softplus=ctx.softplus, lengths=lengths,
                        need_h0=h0 is not None and ctx.needs_input_grad[8])
        return (r["du"], r["ddt"], r["dA"], r["dB"], r["dC"], r["dD"], r["dz"], r["ddt_bias"],
                r["dh0"], None, None)


def kla_ssm(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, *, softplus: bool = True,
            lengths=None):
    """Differentiable selective state space scan (api.ssm_fwd): returns
    (y, hT)."""
    return _KLASSM.apply(u, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths, softplus)


class _KLAQKNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, positions, inv_freq, kw):
        oq, ok = api.qk_norm_fwd(q, k, wq=wq, wk=wk, positions=positions, inv_freq=inv_freq,
                                 **kw)
        ctx.save_for_backward(q, k, wq, wk, positions, inv_freq)
        ctx.kw = kw
        ctx.set_materialize_grads(False)
        return oq, ok

    @staticmethod
    @once_differentiable
    def backward(ctx, gq, gk):
        q, k, wq, wk, positions, inv_freq = ctx.saved_tensors
        r = api.qk_norm_bwd(q, k, _or_zeros(gq, q), _or_zeros(gk, k), wq=wq, wk=wk,
                            positions=positions, inv_freq=inv_freq, **ctx.kw)
        return r["dq"], r["dk"], r["dwq"], r["dwk"], None, None, None


def kla_qk_norm(q, k, *, wq=None, wk=None, positions=None, inv_freq=None, pos0: int = 0,
                norm="l2", eps: float = 1e-6, interleaved: bool = False, scale: float = 1.0):
    """Differentiable norm and rotation of queries and keys
    (api.qk_norm_fwd): returns (oq, ok).  inv_freq and positions get no
    gradient."""
    kw = dict(pos0=pos0, norm=norm, eps=eps, interleaved=interleaved, scale=scale)
    return _KLAQKNorm.apply(q, k, wq, wk, positions, inv_freq, kw)
