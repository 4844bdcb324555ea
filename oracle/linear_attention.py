"""Plain CPU oracle of linear attention with one decay per head (float64 numpy).

TEST INFRASTRUCTURE ONLY: the CUDA library never uses it.

Operation, per document and head, token by token with a = exp(A_log):
    S_t = exp(-a) S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t
Backward of L = sum(o * dO) + sum(h_final * dh_final), in reverse:
    dS  = dS_next + scale q_t dO_t^T          (gradient of S_t)
    dq_t = scale S_t dO_t,  dk_t = dS v_t,  dv_t = dS^T k_t
    da  -= exp(-a) <dS, S_{t-1}>,  dS_next = exp(-a) dS
Arrays: q, k [N, H, dk], v, dO [N, H, dv], A_log [H], h0 [n_docs, H, dk, dv],
cu [n_docs + 1] offsets into the N tokens.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, np.float64)


def forward(q, k, v, A_log, cu, scale, h0=None, states=False):
    """Returns (o, h_final), with states also S after every token [N, H, dk, dv]."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    N, H, dk = q.shape
    dv = v.shape[-1]
    dec = np.exp(-np.exp(_f64(A_log)))[:, None, None]
    o, hf = np.zeros((N, H, dv)), np.zeros((len(cu) - 1, H, dk, dv))
    all_s = np.zeros((N, H, dk, dv)) if states else None
    for d in range(len(cu) - 1):
        S = np.zeros((H, dk, dv)) if h0 is None else _f64(h0)[d].copy()
        for t in range(cu[d], cu[d + 1]):
            S = dec * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hi,hij->hj", q[t], S)
            if states:
                all_s[t] = S
        hf[d] = S
    return (o, hf, all_s) if states else (o, hf)


def backward(q, k, v, A_log, cu, scale, dO, h0=None, dh_final=None):
    """Returns a dict with dq, dk, dv, dA_log, dh0."""
    q, k, v, dO, A_log = _f64(q), _f64(k), _f64(v), _f64(dO), _f64(A_log)
    N, H, dk = q.shape
    dv = v.shape[-1]
    _, _, st = forward(q, k, v, A_log, cu, scale, h0, states=True)
    a = np.exp(A_log)
    dec = np.exp(-a)[:, None, None]
    g = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "da": np.zeros(H),
         "dh0": np.zeros((len(cu) - 1, H, dk, dv))}
    for d in range(len(cu) - 1):
        dS = np.zeros((H, dk, dv)) if dh_final is None else _f64(dh_final)[d].copy()
        for t in range(cu[d + 1] - 1, cu[d] - 1, -1):
            if t > cu[d]:
                prev = st[t - 1]
            else:
                prev = np.zeros((H, dk, dv)) if h0 is None else _f64(h0)[d]
            dS = dS + scale * q[t][:, :, None] * dO[t][:, None, :]
            g["dq"][t] = scale * np.einsum("hij,hj->hi", st[t], dO[t])
            g["dk"][t] = np.einsum("hij,hj->hi", dS, v[t])
            g["dv"][t] = np.einsum("hij,hi->hj", dS, k[t])
            g["da"] -= (dec * dS * prev).sum((1, 2))
            dS = dec * dS
        g["dh0"][d] = dS
    g["dA_log"] = a * g.pop("da")
    return g
