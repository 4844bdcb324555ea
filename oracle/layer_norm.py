"""Plain CPU oracle of layer norm (float64 numpy).

TEST INFRASTRUCTURE ONLY: the CUDA library never uses it.

Rows x [N, D], w and bias [D]:
    mu = mean x,  r = 1 / sqrt(mean (x - mu)^2 + eps),  xh = (x - mu) r
    y = xh w + bias
    g = dy w,  dx = r (g - mean g - xh mean(g xh)),  dw = sum dy xh,  dbias = sum dy
"""
from __future__ import annotations

import numpy as np

EPS = 1e-6


def _stats(x, eps):
    mu = x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    return mu, r


def forward(x, w, bias=None, eps: float = EPS):
    x = np.asarray(x, np.float64)
    mu, r = _stats(x, eps)
    y = (x - mu) * r * np.asarray(w, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64)


def backward(x, w, dy, eps: float = EPS):
    """Returns (dx, dw, dbias)."""
    x, w, dy = (np.asarray(t, np.float64) for t in (x, w, dy))
    mu, r = _stats(x, eps)
    xh = (x - mu) * r
    g = dy * w
    dx = r * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
