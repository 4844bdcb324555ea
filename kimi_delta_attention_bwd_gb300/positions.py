"""Rotary positions (kda_rotary): every head's first rot values turned in pairs
by position * inv_freq,

  (a, b) -> scale (a cos w - b sin w, b cos w + a sin w),

a pair being values i and i + rot/2, or (interleaved) 2 i and 2 i + 1.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _all_well, _apart, _dims, _lib, _positive, _require


def rotary_frequencies(rot: int, base: float = 10000.0, factor: float = 1.0, scaling: str = "none",
                       original_length: Optional[int] = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                       device="cuda"):
    """(inv_freq [rot/2] fp32, scale) for kda_rotary: base^(-2 i / rot), formed in
    64 bits, for contexts `factor` times as long as a model was trained on:
      "none":   as they are
      "linear": all divided by factor (position interpolation, arXiv:2306.15595)
      "ntk":    the base raised so that the slowest is divided by factor and the fastest kept:
                base factor^(rot / (rot - 2))
      "yarn":   by parts (arXiv:2309.00071): frequencies that turn more than beta_fast times over original_length
                tokens are kept, those that turn less than beta_slow times divided by factor, a linear ramp over
                the pair index between; scale = 0.1 ln(factor) + 1
    scale is 1 but for "yarn"."""
    if rot <= 0 or rot % 2:
        raise ValueError(f"rot must be even and positive, got {rot}")
    if not base > 1 or not factor >= 1:
        raise ValueError(f"base must be above 1 and factor at least 1, got {base} and {factor}")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot == 2:
            raise ValueError("ntk scaling needs at least two pairs")
        base = base * factor ** (rot / (rot - 2))
    freq = base ** (-2.0 * i / rot)
    scale = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if original_length is None or original_length <= 0 or not beta_fast > beta_slow > 0:
            raise ValueError("yarn scaling needs original_length and beta_fast > beta_slow > 0")

        def pair(turns):  # the pair index whose frequency turns so often over the original length
            return rot * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.float().to(device), scale


def _rotate(inverse, q, k, inv_freq, positions, cu_seqlens, interleaved, scale, out_q, out_k):
    qs = q.shape
    if len(qs) not in (3, 4):
        raise ValueError(f"q must be [B, T, H, D] or [n, H, D], got shape {tuple(qs)}")
    lead, (Hq, D) = qs[:-2], qs[-2:]
    _dims(inv_freq, "inv_freq", 1)
    rot = 2 * inv_freq.numel()
    if not 0 < rot <= D:
        raise ValueError(f"inv_freq of {rot // 2} pairs for heads of {D} values")
    _positive(scale)
    io, i32 = q.dtype, torch.int32
    specs, names = [(q, qs, io), (inv_freq, inv_freq.shape, torch.float32)], ["q", "inv_freq"]
    Hkv = 0
    if k is not None:
        _dims(k, "k", len(qs))
        Hkv = k.shape[-2]
        specs.append((k, (*lead, Hkv, D), io))
        names.append("k")
    elif out_k is not None:
        raise ValueError("out_k without k")
    if positions is not None:
        if cu_seqlens is not None:
            raise ValueError("positions or cu_seqlens, not both")
        specs.append((positions, lead, i32))
        names.append("positions")
    elif cu_seqlens is not None:
        _dims(cu_seqlens, "cu_seqlens", 1)
        if cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must hold at least two offsets")
        specs.append((cu_seqlens, cu_seqlens.shape, i32))
        names.append("cu_seqlens")
    elif len(qs) == 3:
        raise ValueError("single tokens [n, H, D] need positions")
    for name, t, shape in (("out_q", out_q, qs), ("out_k", out_k, (*lead, Hkv, D))):
        if t is not None:
            specs.append((t, shape, io))
            names.append(name)
    if not _all_well(*specs):
        _require(**dict(zip(names, specs)))
    if out_q is not None or out_k is not None:
        in_place = out_q is not None and out_q.data_ptr() == q.data_ptr()
        if out_q is not None:
            _apart("out_q", out_q, ("q",), q=q, k=k, inv_freq=inv_freq, positions=positions, cu_seqlens=cu_seqlens)
        if out_k is not None:
            _apart("out_k", out_k, ("k",), q=q, k=k, out_q=out_q, inv_freq=inv_freq, positions=positions,
                   cu_seqlens=cu_seqlens)
        if k is not None and in_place != (out_k is not None and out_k.data_ptr() == k.data_ptr()):
            raise ValueError("q and k are turned in place together or not at all")
    y = out_q if out_q is not None else torch.empty_like(q)
    z = None if k is None else out_k if out_k is not None else torch.empty_like(k)
    n = q.numel() // (Hq * D) if Hq else 0
    _lib.kda_rotary(n, qs[1] if len(qs) == 4 else 1, Hq, Hkv, D, rot, io, interleaved, inverse, scale, inv_freq,
                    positions, cu_seqlens, q, k, y, z)
    return y, z


def kda_rotary(q, k, inv_freq, positions=None, cu_seqlens=None, interleaved: bool = False, scale: float = 1.0,
               out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None):
    """Turns q [B, T, Hq, D] and k [B, T, Hkv, D] (or [n, H, D]; bf16 or fp32; k may
    be None) by their positions: returns (q', k').  inv_freq [rot/2] fp32
    (rotary_frequencies; rot <= D, the other values pass) is taken as exact.
    positions int32 [B, T] (or [n]); else places in the documents of cu_seqlens
    (int32 [n_docs + 1] over the flattened tokens; offsets that are not ascending
    from 0 to the tokens' number leave NaN in some tokens), else places in the rows.
    out_q and out_k may be q and k (in place, both), else they share no memory
    with the inputs."""
    return _rotate(False, q, k, inv_freq, positions, cu_seqlens, interleaved, scale, out_q, out_k)


def kda_rotary_backward(dq, dk, inv_freq, positions=None, cu_seqlens=None, interleaved: bool = False,
                        scale: float = 1.0, out_q: Optional[torch.Tensor] = None,
                        out_k: Optional[torch.Tensor] = None):
    """The gradients' way back: (dq, dk) of kda_rotary's outputs to those of its
    inputs (the same turn by minus the angles); arguments as there."""
    return _rotate(True, dq, dk, inv_freq, positions, cu_seqlens, interleaved, scale, out_q, out_k)


__all__ = ["rotary_frequencies", "kda_rotary", "kda_rotary_backward"]
