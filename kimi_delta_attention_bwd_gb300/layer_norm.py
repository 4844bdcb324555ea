"""Layer norm over the last axis (kda_layer_norm and its backward):

  y_j = (x_j - mean x) / sqrt(mean (x - mean x)^2 + eps) w_j + bias_j

x [..., D] (bf16 or fp32, any D >= 1), w and bias [D] fp32; e.g. the hidden
states in front of a layer, or each head's output [B, T, H, dv].
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _check, _lib, _same_device, _shape


def _args(x, w, bias=None):
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError(f"x must have a last axis of at least one value, got shape {tuple(x.shape)}")
    D = x.shape[-1]
    _check(x, "x")
    _shape(w, "w", (D,))
    _check(w, "w", torch.float32)
    if bias is not None:
        _shape(bias, "bias", (D,))
        _check(bias, "bias", torch.float32)
    return x.numel() // D, D


def kda_layer_norm(x, w, bias=None, eps: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   return_stats: bool = False):
    """Layer norm of x [..., D]; eps 1e-6 unless given (> 0).  With
    return_stats returns (y, mean, rstd), the rows' statistics [...] in fp32
    that the backward takes."""
    n, D = _args(x, w, bias)
    if out is not None:
        _shape(out, "out", x.shape)
        _check(out, "out", x.dtype)
    _same_device(x, w=w, bias=bias, out=out)
    y = out if out is not None else torch.empty_like(x)
    mean = rstd = None
    if return_stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    _lib.kda_layer_norm_fwd(n, D, x.dtype, eps, x, w, bias, y, mean, rstd)
    return (y, mean, rstd) if return_stats else y


def kda_layer_norm_backward(x, w, dy, mean, rstd, want_dbias: bool = True, workspace: Optional[torch.Tensor] = None):
    """Backward of kda_layer_norm from its inputs and statistics: returns
    (dx, dw, dbias); dbias is None unless wanted."""
    n, D = _args(x, w)
    _shape(dy, "dy", x.shape)
    _check(dy, "dy", x.dtype)
    for t, nm in ((mean, "mean"), (rstd, "rstd")):
        _shape(t, nm, x.shape[:-1])
        _check(t, nm, torch.float32)
    _same_device(x, w=w, dy=dy, mean=mean, rstd=rstd, workspace=workspace)
    if workspace is None:
        workspace = torch.empty(max(1, _lib.kda_layer_norm_workspace_size(n, D, x.dtype)), dtype=torch.uint8,
                                device=x.device)
    else:
        _check(workspace, "workspace", torch.uint8)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db = torch.empty_like(w) if want_dbias else None
    _lib.kda_layer_norm_bwd(n, D, x.dtype, x, w, dy, mean, rstd, dx, dw, db, workspace)
    return dx, dw, db


__all__ = ["kda_layer_norm", "kda_layer_norm_backward"]
