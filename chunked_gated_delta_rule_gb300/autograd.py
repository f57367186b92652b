"""Differentiable entry points: forward passes and their gradients, both on the
CUDA library (``gdr_chunk_fwd`` and ``gdr_chunk_bwd``, and likewise the short
convolution, the selective scan and the norm).

The first call follows the public shape of the chunked gated-delta-rule operator
(q, k, v, g, beta, scale, initial state, whether to return the final state,
packed-sequence offsets), so code written against that interface can call
this one.  Layouts are those of ``include/gdr.h``: q, k [B, T, H, K];
v [B, T, H, V]; g (per-token log gate) and beta [B, T, H] float32; states
[N, H, K, V] float32 (h = S^T).  ``beta=None`` selects the beta-free mode.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import api, layer


class _ChunkGatedDeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, scale, initial_state, output_final_state, cu_seqlens):
        o, ht = api.gdr_chunk_fwd(q, k, v, g, beta, cu_seqlens=cu_seqlens, h0=initial_state,
                                  output_final_state=output_final_state, scale=scale)
        ctx.save_for_backward(q, k, v, g, beta, initial_state, cu_seqlens)
        ctx.scale = scale
        return o, ht

    @staticmethod
    def backward(ctx, do, dht):
        q, k, v, g, beta, h0, cu = ctx.saved_tensors
        want_dh0 = h0 is not None and ctx.needs_input_grad[6]
        dq, dk, dv, dg, dbeta, dh0 = api.gdr_chunk_bwd(
            q, k, v, g, beta, do.contiguous(), cu_seqlens=cu, h0=h0,
            dht=None if dht is None else dht.contiguous(), scale=ctx.scale, want_dh0=want_dh0)
        return dq, dk, dv, dg, dbeta, None, dh0, None, None


def chunk_gated_delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                           beta: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                           initial_state: Optional[torch.Tensor] = None,
                           output_final_state: bool = False,
                           cu_seqlens: Optional[torch.Tensor] = None
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """o, final_state of the chunked gated delta rule, differentiable with
    respect to q, k, v, g, beta and initial_state.  ``scale`` defaults to
    1/sqrt(K).  ``final_state`` is None unless ``output_final_state``.  q, k
    and v may be views with token and head strides (e.g. slices of one fused
    projection); the library reads them in place."""
    return _ChunkGatedDeltaRule.apply(q, k, v, g.contiguous(),
                                      None if beta is None else beta.contiguous(),
                                      0.0 if scale is None else float(scale),
                                      None if initial_state is None else initial_state.contiguous(),
                                      bool(output_final_state), cu_seqlens)


def _cast(grad, like):
    return None if grad is None or like is None else grad.to(like.dtype)


def _dense(t):
    return None if t is None else t.contiguous()


def _some(grad, like):
    """The gradient of an output, zeros where nothing depends on it."""
    return torch.zeros_like(like) if grad is None else grad.contiguous()


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, activation, h0, output_final_state, cu_seqlens, max_seqlen):
        y, ht = layer.gdr_short_conv_fwd(x, weight, bias, cu_seqlens, h0, activation=activation,
                                         output_final_state=output_final_state,
                                         max_seqlen=max_seqlen)
        ctx.save_for_backward(x, weight, bias, h0, cu_seqlens)
        ctx.args = activation, max_seqlen
        ctx.set_materialize_grads(False)
        return y, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dht):
        x, weight, bias, h0, cu = ctx.saved_tensors
        activation, max_seqlen = ctx.args
        dx, dw, db, dh0 = layer.gdr_short_conv_bwd(
            x, weight, _some(dy, x), bias, cu, h0, _dense(dht),
            activation=activation, want_dh0=h0 is not None and ctx.needs_input_grad[4],
            max_seqlen=max_seqlen)
        return dx, _cast(dw, weight), _cast(db, bias), None, dh0, None, None, None


def short_conv(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               activation: Optional[str] = "silu", initial_state: Optional[torch.Tensor] = None,
               output_final_state: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
               max_seqlen: Optional[int] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """y, final_state of the short causal convolution (``gdr_short_conv_fwd``), differentiable
    with respect to x, weight, bias and initial_state."""
    return _ShortConv.apply(x, weight.contiguous(), _dense(bias), activation, _dense(initial_state),
                            bool(output_final_state), cu_seqlens, max_seqlen)


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, softplus, h0, output_final_state, cu_seqlens,
                max_seqlen):
        y, ht = layer.gdr_selective_scan_fwd(x, dt, A, B, C, D, z, dt_bias, cu_seqlens, h0,
                                             softplus=softplus,
                                             output_final_state=output_final_state,
                                             max_seqlen=max_seqlen)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens)
        ctx.args = softplus, max_seqlen
        ctx.set_materialize_grads(False)
        return y, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dht):
        x, dt, A, B, C, D, z, dt_bias, h0, cu = ctx.saved_tensors
        softplus, max_seqlen = ctx.args
        dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0 = layer.gdr_selective_scan_bwd(
            x, dt, A, B, C, _some(dy, x), D, z, dt_bias, cu, h0, _dense(dht), softplus=softplus,
            want_dh0=h0 is not None and ctx.needs_input_grad[9], max_seqlen=max_seqlen)
        return dx, ddt, dA, dB, dC, dD, dz, ddt_bias, None, dh0, None, None, None


def selective_scan(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                   C: torch.Tensor, D: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                   softplus: bool = True, initial_state: Optional[torch.Tensor] = None,
                   output_final_state: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
                   max_seqlen: Optional[int] = None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """y, final_state of the selective scan (``gdr_selective_scan_fwd``), differentiable with
    respect to x, dt, A, B, C, D, z, dt_bias and initial_state."""
    return _SelectiveScan.apply(x, dt, A.contiguous(), B, C, _dense(D), z, _dense(dt_bias),
                                bool(softplus), _dense(initial_state), bool(output_final_state),
                                cu_seqlens, max_seqlen)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, r, _ = layer.gdr_rms_norm_fwd(x, weight, residual, eps=eps)
        ctx.save_for_backward(x if r is None else r, weight)
        ctx.eps, ctx.residual = eps, residual is not None
        ctx.set_materialize_grads(False)
        return y, r

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr):
        r, weight = ctx.saved_tensors
        dx, dw = layer.gdr_rms_norm_bwd(_some(dy, r), r, weight, _dense(dr), eps=ctx.eps)
        return dx, _cast(dw, weight), dx if ctx.residual else None, None


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
             residual: Optional[torch.Tensor] = None, eps: float = 1e-6
             ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """y, r of the root-mean-square norm of r = x + residual (``gdr_rms_norm_fwd``), differentiable
    with respect to x, weight and residual; r is None without a residual."""
    return _RmsNorm.apply(x, _dense(weight), residual, float(eps))
