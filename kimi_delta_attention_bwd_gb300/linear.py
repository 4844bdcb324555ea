"""Linear attention with one decay per head (kda_linear_*):

  S_t = exp(-a) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   a = exp(A_log[h])

per document and head; q and k enter as they are.  Shapes, dtypes and
documents as kda_forward: q, k [B, T, H, dk]; v, o [B, T, H, dv] (bf16 or fp32;
(dk, dv) = (32, 64), (64, 64), (64, 128), (128, 128)); A_log [H] fp32; states
[n_docs, H, dk, dv] fp32; optional cu_seqlens int32 [n_docs + 1].  States and
the decay gradient are formed with 24 bits of every operand; bf16 outputs are
rounded once (their computed operands are off by 2^-16 at most).
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import _all_well, _apart, _dims, _lib, _require


@dataclass
class LinearContext:
    """What kda_linear_backward needs from kda_linear_forward."""
    problem: object
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    A_log: torch.Tensor
    h0: Optional[torch.Tensor]
    cu_seqlens: Optional[torch.Tensor]
    cu_seqlens_host: object
    workspace: torch.Tensor
    n_docs: int
    saved: bool
    stream: Optional[int] = None  # the workspace's, where the forward allocated it


def _host_offsets(cu_seqlens_host, cu_seqlens):
    """cu_seqlens_host as the int32 host array the library reads (a tensor or
    a numpy array of cu_seqlens' length)."""
    if cu_seqlens_host is None:
        return None
    if cu_seqlens is None:
        raise ValueError("cu_seqlens_host comes with cu_seqlens")
    c = cu_seqlens_host
    if isinstance(c, torch.Tensor):
        if c.is_cuda or c.dtype != torch.int32 or not c.is_contiguous():
            raise ValueError("cu_seqlens_host must be a contiguous int32 tensor on the host")
        n = c.numel()
    else:
        if str(c.dtype) != "int32" or not c.flags["C_CONTIGUOUS"]:
            raise ValueError("cu_seqlens_host must be a contiguous int32 array")
        n = c.size
    if n != cu_seqlens.numel():
        raise ValueError(f"cu_seqlens_host has {n} offsets, cu_seqlens {cu_seqlens.numel()}")
    return c


def kda_linear_forward(q, k, v, A_log, scale: Optional[float] = None, h0=None, cu_seqlens=None, cu_seqlens_host=None,
                       save_for_backward: bool = True, workspace: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, want_final_state: bool = True,
                       final_state: Optional[torch.Tensor] = None):
    """Forward pass.  Returns (o, h_final or None, ctx); ctx feeds
    kda_linear_backward when save_for_backward is set.  scale: 1/sqrt(dk)
    unless given (> 0).  out / final_state: optional preallocated outputs that
    share no memory with the inputs; final_state may be h0 (states updated in
    place) unless the call saves for the backward, which reads h0."""
    _dims(q, "q", 4)
    _dims(v, "v", 4)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    io, f32 = q.dtype, torch.float32
    n_docs = B
    if cu_seqlens is not None:
        _dims(cu_seqlens, "cu_seqlens", 1)
        if cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must hold at least two offsets")
        n_docs = cu_seqlens.numel() - 1
    cu_seqlens_host = _host_offsets(cu_seqlens_host, cu_seqlens)
    states = (n_docs, H, dk, dv)
    more = [s for s in ((h0, states, f32), (out, v.shape, io), (final_state, states, f32),
                        (cu_seqlens, (n_docs + 1,), torch.int32)) if s[0] is not None]
    if not _all_well((q, q.shape, io), (k, q.shape, io), (v, (B, T, H, dv), io), (A_log, (H,), f32), *more):
        _require(q=(q, q.shape, io), k=(k, q.shape, io), v=(v, (B, T, H, dv), io), A_log=(A_log, (H,), f32),
                 h0=(h0, states, f32), out=(out, (B, T, H, dv), io), final_state=(final_state, states, f32),
                 cu_seqlens=(cu_seqlens, (n_docs + 1,), torch.int32))
    if save_for_backward and h0 is not None and final_state is not None and h0.data_ptr() == final_state.data_ptr():
        raise ValueError("final_state cannot be h0 when the call saves for the backward")
    if out is not None:
        _apart("out", out, q=q, k=k, v=v, h0=h0)
    if final_state is not None:
        _apart("final_state", final_state, ("h0",), q=q, k=k, v=v, h0=h0, out=out)
    if save_for_backward and cu_seqlens_host is not None:
        # the backward plans by them again: a buffer that the next batch's offsets overwrite must not change them
        cu_seqlens_host = (cu_seqlens_host.clone() if isinstance(cu_seqlens_host, torch.Tensor)
                           else cu_seqlens_host.copy())
    prob = _lib.make_problem(B, T, H, dk, dv, io, scale, cu_seqlens, cu_seqlens_host)
    stream = None
    if workspace is None:
        stream = _lib._stream()
        # (size 0 for a problem that the call below refuses with its own status)
        workspace = torch.empty(_lib.kda_linear_workspace_size(prob, save_for_backward) or 1, dtype=torch.uint8,
                                device=q.device)
    else:
        _require(workspace=(workspace, workspace.shape, torch.uint8))
    o = out if out is not None else torch.empty_like(v)
    hf = None
    if want_final_state:
        hf = final_state if final_state is not None else torch.empty(states, dtype=f32, device=q.device)
    _lib.kda_linear_fwd(prob, q, k, v, A_log, h0, o, hf, save_for_backward, workspace)
    return o, hf, LinearContext(prob, q, k, v, A_log, h0, cu_seqlens, cu_seqlens_host, workspace, n_docs,
                                bool(save_for_backward), stream)


def kda_linear_backward(ctx: LinearContext, dO, dh_final=None, want_dA_log: bool = True, want_dh0: bool = True):
    """Backward of sum(o * dO) + sum(h_final * dh_final).  Returns a dict with
    dq, dk, dv (io dtype), dA_log and dh0 (fp32; None where not wanted:
    without dA_log, e.g. for fixed decays, its products are skipped, and the
    others keep their bits)."""
    if not ctx.saved:
        raise ValueError("the forward saved nothing: call kda_linear_forward with save_for_backward=True")
    q, v = ctx.q, ctx.v
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    states = (ctx.n_docs, H, dk, dv)
    # (q stands for the forward's tensors: the current device may have changed since)
    specs = dict(q=(q, q.shape, q.dtype), dO=(dO, (B, T, H, dv), q.dtype), dh_final=(dh_final, states, torch.float32))
    if dh_final is None:
        del specs["dh_final"]
    if not _all_well(*specs.values()):
        _require(**specs)
    gr = {"dq": torch.empty_like(q), "dk": torch.empty_like(q), "dv": torch.empty_like(v),
          "dA_log": torch.empty_like(ctx.A_log) if want_dA_log else None,
          "dh0": torch.empty(states, dtype=torch.float32, device=q.device) if want_dh0 else None}
    if ctx.stream is not None and ctx.stream != _lib._stream():
        # a context dropped after this call must not give its memory to the forward's stream before the kernels end
        ctx.workspace.record_stream(torch.cuda.current_stream())
    _lib.kda_linear_bwd(ctx.problem, q, ctx.k, v, ctx.A_log, ctx.h0, dO, dh_final, gr["dq"], gr["dk"], gr["dv"],
                        gr["dA_log"], gr["dh0"], ctx.workspace)
    return gr


def kda_linear_decode_step(q, k, v, A_log, state, scale: Optional[float] = None,
                           out: Optional[torch.Tensor] = None):
    """One token for each of n sequences: q, k [n, H, dk], v [n, H, dv] (bf16 or
    fp32), A_log [H] and state [n, H, dk, dv] fp32, the state updated in place;
    out may be q, k or v, else it shares no memory with the inputs.
    Returns o [n, H, dv] in the io dtype."""
    _dims(q, "q", 3)
    _dims(v, "v", 3)
    n, H, dk = q.shape
    dv = v.shape[-1]
    io, f32 = q.dtype, torch.float32
    specs = ((q, q.shape, io), (k, q.shape, io), (v, (n, H, dv), io), (A_log, (H,), f32), (state, (n, H, dk, dv), f32))
    if out is not None:
        specs += ((out, v.shape, io),)
    if not _all_well(*specs):
        _require(**dict(zip(("q", "k", "v", "A_log", "state", "out"), specs)))
    if out is not None:
        _apart("out", out, ("q", "k", "v"), q=q, k=k, v=v, state=state)
    o = out if out is not None else torch.empty_like(v)
    _lib.kda_linear_decode(n, H, dk, dv, io, scale, q, k, v, A_log, state, o)
    return o


__all__ = ["LinearContext", "kda_linear_forward", "kda_linear_backward", "kda_linear_decode_step"]
