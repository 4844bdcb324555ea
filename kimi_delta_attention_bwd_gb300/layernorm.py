"""Layer norm over the last axis (kda_layer_norm and its backward):

  y_j = (x_j - mean x) / sqrt(mean (x - mean x)^2 + eps) w_j + bias_j

x [..., D] (bf16 or fp32, any D >= 1), w and bias [D] fp32; e.g. the hidden
states in front of a layer, or each head's output [B, T, H, dv].
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _all_well, _apart, _lib, _require


def _rows(x, w, bias=None):
    """(rows, D) of x [..., D], with x and the fp32 [D] parameters checked."""
    D = x.shape[-1] if x.dim() else 0
    if D == 0:
        raise ValueError(f"x must have a last axis of at least one value, got shape {tuple(x.shape)}")
    f32 = torch.float32
    specs = ((x, x.shape, x.dtype), (w, (D,), f32)) if bias is None else ((x, x.shape, x.dtype), (w, (D,), f32),
                                                                         (bias, (D,), f32))
    if not _all_well(*specs):
        _require(**dict(zip(("x", "w", "bias"), specs)))
    return x.numel() // D, D


def kda_layer_norm(x, w, bias=None, eps: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   return_stats: bool = False):
    """Layer norm of x [..., D]; eps 1e-6 unless given (> 0); out may be x
    (in place), else it shares no memory with the inputs.  With return_stats returns (y, mean, rstd), the rows' statistics [...] in fp32
    that the backward takes."""
    n, D = _rows(x, w, bias)
    if out is None:
        y = torch.empty_like(x)
    else:
        _require(out=(out, x.shape, x.dtype))
        _apart("out", out, ("x",), x=x, w=w, bias=bias)
        y = out
    mean = rstd = None
    if return_stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    _lib.kda_layer_norm_fwd(n, D, x.dtype, eps, x, w, bias, y, mean, rstd)
    return (y, mean, rstd) if return_stats else y


def kda_layer_norm_backward(x, w, dy, mean, rstd, want_dbias: bool = True, workspace: Optional[torch.Tensor] = None):
    """Backward of kda_layer_norm from its inputs and statistics: returns
    (dx, dw, dbias); dbias is None unless wanted."""
    n, D = _rows(x, w)
    _require(dy=(dy, x.shape, x.dtype), mean=(mean, x.shape[:-1], torch.float32),
             rstd=(rstd, x.shape[:-1], torch.float32))
    if workspace is None:
        workspace = torch.empty(_lib.kda_layer_norm_workspace_size(n, D, x.dtype) or 1, dtype=torch.uint8,
                                device=x.device)
    else:
        _require(workspace=(workspace, workspace.shape, torch.uint8))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db = torch.empty_like(w) if want_dbias else None
    _lib.kda_layer_norm_bwd(n, D, x.dtype, x, w, dy, mean, rstd, dx, dw, db, workspace)
    return dx, dw, db


__all__ = ["kda_layer_norm", "kda_layer_norm_backward"]
