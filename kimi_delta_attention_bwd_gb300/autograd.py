"""torch.autograd integration of the KDA operations: the same library calls
as kda_forward / kda_backward (and the convolution and gated-norm entry
points), wrapped so that a model can use them like any differentiable op.

  o = kda_attention(q, k, v, f, b, A_log, dt_bias)                    # o
  o, h_final = kda_attention(..., h0=h0, output_final_state=True)     # and the final states
  x = short_conv(x_raw, conv_w, cu_seqlens)                           # causal conv (k=4) + silu
  y = gated_norm(o, gate, weight)                                     # gated RMSNorm epilogue
  o = linear_attention(q, k, v, A_log)                                # linear attention, one decay per head
  y = layer_norm(x, weight, bias)                                     # layer norm over the last axis

Gradients flow to q, k, v, f, b, A_log, dt_bias and h0 (and to the
convolution's input and taps, the norms' input, gate, weight and bias).  Each
backward runs the library's backward kernels once; a second derivative is
not provided.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (LinearContext, kda_backward, kda_forward, kda_layer_norm, kda_layer_norm_backward, kda_linear_backward,
               kda_linear_forward, kda_norm_gate, kda_norm_gate_backward, kda_short_conv, kda_short_conv_backward)

__all__ = ["kda_attention", "short_conv", "gated_norm", "linear_attention", "layer_norm"]


class _KdaAttention(torch.autograd.Function):
    @staticmethod
    def forward(fctx, q, k, v, f, b, A_log, dt_bias, h0, scale, cu_seqlens, cu_seqlens_host, want_final):
        o, hf, kctx = kda_forward(q, k, v, f, b, A_log, dt_bias, scale=scale, h0=h0, cu_seqlens=cu_seqlens,
                                  cu_seqlens_host=cu_seqlens_host, save_for_backward=True,
                                  want_final_state=want_final)
        fctx.kctx = kctx
        fctx.has_h0 = h0 is not None
        if want_final:
            return o, hf
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(fctx, dO, dhf=None):
        kctx = fctx.kctx
        if dO is None:
            dO = torch.zeros(*kctx.q.shape[:3], kctx.v.shape[-1], dtype=kctx.q.dtype, device=kctx.q.device)
        g = kda_backward(kctx, dO.contiguous(), None if dhf is None else dhf.contiguous(),
                         want_dh0=fctx.has_h0 and fctx.needs_input_grad[7])
        return (g["dq"], g["dk"], g["dv"], g["df"], g["db"], g["dA_log"], g["ddt_bias"],
                g["dh0"] if fctx.has_h0 else None, None, None, None, None)


def kda_attention(q, k, v, f, b, A_log, dt_bias, scale: Optional[float] = None, h0=None, cu_seqlens=None,
                  cu_seqlens_host=None, output_final_state: bool = False):
    """Differentiable KDA: o (and h_final when output_final_state) from the
    layouts of kda_forward; backward through kda_backward."""
    return _KdaAttention.apply(q, k, v, f, b, A_log, dt_bias, h0, scale, cu_seqlens, cu_seqlens_host,
                               output_final_state)


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(fctx, x, w, cu_seqlens, activation):
        fctx.save_for_backward(x, w)
        fctx.cu_seqlens, fctx.activation = cu_seqlens, activation
        return kda_short_conv(x, w, cu_seqlens, activation)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(fctx, dy):
        x, w = fctx.saved_tensors
        dx, dw = kda_short_conv_backward(x, w, dy.contiguous(), fctx.cu_seqlens, fctx.activation)
        return dx, dw, None, None


def short_conv(x, w, cu_seqlens=None, activation: str = "silu"):
    """Differentiable short causal depthwise convolution (kda_short_conv)."""
    return _ShortConv.apply(x, w, cu_seqlens, activation)


class _GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(fctx, x, g, w, eps):
        fctx.save_for_backward(x, g, w)
        fctx.eps = eps
        return kda_norm_gate(x, g, w, eps)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(fctx, dy):
        x, g, w = fctx.saved_tensors
        dx, dg, dw = kda_norm_gate_backward(x, g, w, dy.contiguous(), fctx.eps)
        return dx, dg, dw, None


def gated_norm(x, g, w, eps: Optional[float] = None):
    """Differentiable gated RMSNorm epilogue (kda_norm_gate)."""
    return _GatedNorm.apply(x, g, w, eps)


def _given(g):
    """An incoming gradient as the library takes it: contiguous, and 16-byte
    aligned, which a slice of a larger tensor's gradient need not be."""
    g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(fctx, q, k, v, A_log, h0, scale, cu_seqlens, cu_seqlens_host, want_final, recorded):
        fctx.set_materialize_grads(False)
        o, hf, lctx = kda_linear_forward(q, k, v, A_log, scale=scale, h0=h0, cu_seqlens=cu_seqlens,
                                         cu_seqlens_host=cu_seqlens_host,
                                         save_for_backward=recorded and any(fctx.needs_input_grad),
                                         want_final_state=want_final)
        # (the workspace, which holds every chunk's states, among them: freed by the backward, seen by hooks)
        fctx.save_for_backward(q, k, v, A_log, h0, cu_seqlens, lctx.workspace)
        fctx.rest = (lctx.problem, lctx.cu_seqlens_host, lctx.n_docs, lctx.saved)
        return (o, hf) if want_final else o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(fctx, dO, dhf=None):
        q, k, v, A_log, h0, cu_seqlens, workspace = fctx.saved_tensors
        problem, cu_host, n_docs, saved = fctx.rest
        lctx = LinearContext(problem, q, k, v, A_log, h0, cu_seqlens, cu_host, workspace, n_docs, saved)
        dO = torch.zeros_like(v) if dO is None else _given(dO)
        g = kda_linear_backward(lctx, dO, None if dhf is None else _given(dhf),
                                want_dA_log=fctx.needs_input_grad[3],
                                want_dh0=h0 is not None and fctx.needs_input_grad[4])
        return g["dq"], g["dk"], g["dv"], g["dA_log"], g["dh0"], None, None, None, None, None


def linear_attention(q, k, v, A_log, scale: Optional[float] = None, h0=None, cu_seqlens=None, cu_seqlens_host=None,
                     output_final_state: bool = False):
    """Differentiable linear attention: o (and h_final when
    output_final_state) from the layouts of kda_linear_forward; gradients to q,
    k, v, A_log and h0 through kda_linear_backward."""
    return _LinearAttention.apply(q, k, v, A_log, h0, scale, cu_seqlens, cu_seqlens_host, output_final_state,
                                  torch.is_grad_enabled())


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(fctx, x, w, bias, eps, recorded):
        if not (recorded and any(fctx.needs_input_grad)):
            return kda_layer_norm(x, w, bias, eps)
        y, mean, rstd = kda_layer_norm(x, w, bias, eps, return_stats=True)
        fctx.save_for_backward(x, w, mean, rstd)
        fctx.has_bias = bias is not None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(fctx, dy):
        x, w, mean, rstd = fctx.saved_tensors
        dx, dw, db = kda_layer_norm_backward(x, w, _given(dy), mean, rstd, want_dbias=fctx.has_bias)
        return dx, dw, db, None, None


def layer_norm(x, w, bias=None, eps: Optional[float] = None):
    """Differentiable layer norm over the last axis (kda_layer_norm)."""
    return _LayerNorm.apply(x, w, bias, eps, torch.is_grad_enabled())
