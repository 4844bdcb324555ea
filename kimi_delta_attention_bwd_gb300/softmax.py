"""Softmax attention with grouped heads (kda_softmax_*): the full-attention
layer that stands between the linear ones.

  o_i = sum_j p_ij v_j,   p_ij = exp(scale q_i k_j - lse_i)

per document and query head, over the keys j <= i + Lk - Lq (causal: the last
query sees every key) or over all keys.  q, o [B, T, Hq, D]; k, v [B, Tk, Hkv, D]
(bf16 or fp32; D = 64 or 128; Hq a multiple of Hkv); documents are the rows, or
cu_seqlens int32 [n_docs + 1] over the flattened B*T queries, with cu_seqlens_k
over the B*Tk keys where those differ (the next pieces of prompts whose keys are
already there).  A query that sees no key gives o = 0 and lse = -inf.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import _all_well, _apart, _dims, _lib, _positive, _require
from .linear import _host_offsets


@dataclass
class SoftmaxContext:
    """What kda_softmax_backward needs from kda_softmax_forward."""
    problem: object
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    o: torch.Tensor
    cu_seqlens: Optional[torch.Tensor]
    cu_seqlens_k: Optional[torch.Tensor]
    host: tuple
    workspace: torch.Tensor
    saved: bool
    stream: Optional[int] = None  # the forward's
    own: tuple = ()               # of what the backward reads, that the forward allocated there


def _offsets(cu, name):
    if cu is not None:
        _dims(cu, name, 1)
        if cu.numel() < 2:
            raise ValueError(f"{name} must hold at least two offsets")


def kda_softmax_forward(q, k, v, scale: Optional[float] = None, causal: bool = True, cu_seqlens=None,
                        cu_seqlens_k=None, cu_seqlens_host=None, cu_seqlens_k_host=None,
                        save_for_backward: bool = True, workspace: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None):
    """Forward pass.  Returns (o, lse, ctx): lse [B, T, Hq] fp32, the rows'
    log-sums; ctx feeds kda_softmax_backward when save_for_backward is set, which
    reads o too: leave it as it is until then (offsets on the device it reads no more).  scale: 1/sqrt(D) unless given
    (> 0).  out: optional preallocated o that shares no memory with the inputs or
    with a given workspace, which shares none with them either."""
    _dims(q, "q", 4)
    _dims(k, "k", 4)
    qs = q.shape
    B, T, Hq, D = qs
    _, Tk, Hkv, _ = k.shape
    io, keys = q.dtype, (B, Tk, Hkv, D)
    if Hkv == 0 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads are not a multiple of {Hkv} key heads")
    specs = [(q, qs, io), (k, keys, io), (v, keys, io)]
    names = ["q", "k", "v"]
    if cu_seqlens is not None or cu_seqlens_k is not None or cu_seqlens_host is not None \
            or cu_seqlens_k_host is not None:
        _offsets(cu_seqlens, "cu_seqlens")
        _offsets(cu_seqlens_k, "cu_seqlens_k")
        if cu_seqlens_k is not None and cu_seqlens is None:
            raise ValueError("cu_seqlens_k comes with cu_seqlens")
        if cu_seqlens_k is None and T != Tk and cu_seqlens is not None:
            raise ValueError(f"{B * Tk} keys for {B * T} queries need cu_seqlens_k")
        cu_seqlens_host = _host_offsets(cu_seqlens_host, cu_seqlens)
        if cu_seqlens_k_host is not None and cu_seqlens_k is None:
            raise ValueError("cu_seqlens_k_host comes with cu_seqlens_k")
        cu_seqlens_k_host = _host_offsets(cu_seqlens_k_host, cu_seqlens_k)
        n = cu_seqlens.numel()
        for name, cu in (("cu_seqlens", cu_seqlens), ("cu_seqlens_k", cu_seqlens_k)):
            if cu is not None:
                specs.append((cu, (n,), torch.int32))
                names.append(name)
        if save_for_backward:  # (a buffer that the next batch's offsets overwrite must not change what is checked)
            cu_seqlens_host, cu_seqlens_k_host = (
                c if c is None else c.clone() if isinstance(c, torch.Tensor) else c.copy()
                for c in (cu_seqlens_host, cu_seqlens_k_host))
    if out is not None:
        specs.append((out, qs, io))
        names.append("out")
    if not _all_well(*specs):
        _require(**dict(zip(names, specs)))
    if out is not None:
        _apart("out", out, q=q, k=k, v=v, cu_seqlens=cu_seqlens, cu_seqlens_k=cu_seqlens_k)
    if workspace is not None:
        _apart("workspace", workspace, q=q, k=k, v=v, out=out, cu_seqlens=cu_seqlens, cu_seqlens_k=cu_seqlens_k)
    if scale is not None:
        _positive(scale)
    prob = _lib.make_softmax_problem(B, T, Tk, Hq, Hkv, D, io, scale, causal, cu_seqlens, cu_seqlens_k,
                                     cu_seqlens_host, cu_seqlens_k_host)
    stream, own = _lib._stream(), ()
    if workspace is None:
        # (size 0 for a problem that the call below refuses with its own status)
        workspace = torch.empty(_lib.kda_softmax_workspace_size(prob, save_for_backward) or 1, dtype=torch.uint8,
                                device=q.device)
        own = (workspace,)
    else:
        _require(workspace=(workspace, workspace.shape, torch.uint8))
    o = out
    if o is None:
        o = torch.empty_like(q)
        own += (o,)
    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)
    _lib.kda_softmax_fwd(prob, q, k, v, o, lse, save_for_backward, workspace)
    return o, lse, SoftmaxContext(prob, q, k, v, o, cu_seqlens, cu_seqlens_k, (cu_seqlens_host, cu_seqlens_k_host),
                                  workspace, bool(save_for_backward), stream, own)


def kda_softmax_backward(ctx: SoftmaxContext, dO):
    """Backward of sum(o * dO): a dict with dq, dk, dv in the io dtype.  Sums run
    in a fixed order.  NaN where the device refused the forward's offsets, or the
    workspace (kda_device_status says which)."""
    if not ctx.saved:
        raise ValueError("the forward saved nothing: call kda_softmax_forward with save_for_backward=True")
    q, k = ctx.q, ctx.k
    # (q stands for the forward's tensors: the current device may have changed since)
    specs = dict(q=(q, q.shape, q.dtype), dO=(dO, q.shape, q.dtype))
    if not _all_well(*specs.values()):
        _require(**specs)
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(ctx.v)}
    if ctx.stream is not None and ctx.stream != _lib._stream():
        # a context dropped after this call must not give its memory to the forward's stream before the kernels end
        for t in ctx.own:
            t.record_stream(torch.cuda.current_stream())
    _lib.kda_softmax_bwd(ctx.problem, q, k, ctx.v, ctx.o, dO, g["dq"], g["dk"], g["dv"], ctx.workspace)
    return g


def kda_softmax_decode_step(q, k, v, k_cache, v_cache, lengths, scale: Optional[float] = None,
                            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """One token for each of n sequences: q [n, Hq, D], k, v [n, Hkv, D], caches
    [n, cap, Hkv, D] (one dtype), lengths [n] int32 on the device: the tokens in
    each cache.  k and v are written behind them, in place, and the query sees
    them all and its own; lengths stays as it is (the layers of a model share it).
    What places behind them hold reaches no result, but bf16 caches are read up to 63
    places further: nothing else writes there meanwhile.
    A negative length takes no step (o = 0, a padded batch), and neither does one
    of cap or more (kda_device_status of a given workspace reports it).  out shares
    no memory with the inputs, nor do the caches with each other or with the other
    inputs, nor a given workspace with any of them.
    Returns o [n, Hq, D]."""
    _dims(q, "q", 3)
    _dims(k_cache, "k_cache", 4)
    qs, cache = q.shape, k_cache.shape
    n, Hq, D = qs
    _, cap, Hkv, _ = cache
    io, new = q.dtype, (n, Hkv, D)
    if Hkv == 0 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads are not a multiple of {Hkv} key heads")
    if cache[0] != n or cache[3] != D:
        raise ValueError(f"k_cache must have shape {(n, cap, Hkv, D)}, got {tuple(cache)}")
    specs = ((q, qs, io), (k, new, io), (v, new, io), (k_cache, cache, io), (v_cache, cache, io),
             (lengths, (n,), torch.int32))
    if out is not None:
        specs += ((out, qs, io),)
    if not _all_well(*specs):
        _require(**dict(zip(("q", "k", "v", "k_cache", "v_cache", "lengths", "out"), specs)))
    # the caches share no memory with the other tensors or with each other (the named checks say which)
    kc, vc, size = k_cache.data_ptr(), v_cache.data_ptr(), k_cache.numel() * k_cache.element_size()
    near = kc < vc + size and vc < kc + size
    for t in (q, k, v, lengths):
        a = t.data_ptr()
        b = a + t.numel() * t.element_size()
        near = near or (a < kc + size and kc < b) or (a < vc + size and vc < b)
    if near:
        _apart("k_cache", k_cache, q=q, k=k, v=v, lengths=lengths, v_cache=v_cache)
        _apart("v_cache", v_cache, q=q, k=k, v=v, lengths=lengths)
    if out is not None:
        _apart("out", out, q=q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, lengths=lengths)
    if workspace is not None:
        _apart("workspace", workspace, q=q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, lengths=lengths, out=out)
    if scale is not None:
        _positive(scale)
    if workspace is None:
        workspace = torch.empty(_lib.kda_softmax_decode_workspace_size(n, cap, Hq, Hkv, D) or 1, dtype=torch.uint8,
                                device=q.device)
    else:
        _require(workspace=(workspace, workspace.shape, torch.uint8))
    o = out if out is not None else torch.empty_like(q)
    _lib.kda_softmax_decode(n, cap, Hq, Hkv, D, io, scale, q, k, v, k_cache, v_cache, lengths, o, workspace)
    return o


__all__ = ["SoftmaxContext", "kda_softmax_forward", "kda_softmax_backward", "kda_softmax_decode_step"]
