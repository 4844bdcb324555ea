"""Plain CPU oracle of softmax attention with grouped heads (float64 numpy).

TEST INFRASTRUCTURE ONLY: the CUDA library never uses it.

Per document (Lq queries, Lk keys) and query head h, key head h / G:
    s_ij = scale q_i k_j over the keys j <= i + Lk - Lq (causal) or all
    lse_i = log sum_j exp s_ij,  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
Backward of L = sum(o * dO):
    dv_j = sum_i p_ij dO_i,  ds_ij = p_ij (dO_i v_j - sum_m p_im dO_i v_m),
    dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
Rows that see no key: o = 0, lse = -inf, no gradients.
Arrays: q, dO [Nq, Hq, D], k, v [Nk, Hkv, D], cu, cu_k offsets.  Beside every
result stands the sum of its terms' magnitudes (mag), for error bounds.
"""
from __future__ import annotations

import numpy as np


def attend(q, k, v, cu, cu_k, scale, causal, dO=None):
    """({"o", "lse"[, "dq", "dk", "dv"]}, the same as magnitudes, largest logit magnitude)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    Nq, Hq, D = q.shape
    G = Hq // k.shape[1]
    ref = dict(o=np.zeros(q.shape), lse=np.full((Nq, Hq), -np.inf))
    mag = dict(o=np.zeros(q.shape), lse=np.zeros((Nq, Hq)))
    if dO is not None:
        dO = np.asarray(dO, np.float64)
        for d in (ref, mag):
            d.update(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape))
    top = 0.0
    for d in range(len(cu) - 1):
        a, b = slice(cu[d], cu[d + 1]), slice(cu_k[d], cu_k[d + 1])
        Lq, Lk = cu[d + 1] - cu[d], cu_k[d + 1] - cu_k[d]
        if Lq == 0 or Lk == 0:
            continue
        seen = np.ones((Lq, Lk), bool)
        if causal:
            seen = np.arange(Lk)[None] <= np.arange(Lq)[:, None] + (Lk - Lq)
        rows = seen.any(1)
        for h in range(Hq):
            Q, K, V = q[a, h], k[b, h // G], v[b, h // G]
            S = np.where(seen, scale * (Q @ K.T), -np.inf)
            top = max(top, (scale * (np.abs(Q) @ np.abs(K).T)).max())
            m = np.where(rows, S.max(1), 0.0)
            E = np.exp(S - m[:, None])
            t = E.sum(1)
            P = E / np.where(rows, t, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                ref["lse"][a, h] = np.where(rows, np.log(t) + m, -np.inf)
            mag["lse"][a, h] = np.where(rows, np.abs(ref["lse"][a, h]), 0.0)
            ref["o"][a, h] = P @ V
            mag["o"][a, h] = P @ np.abs(V)
            if dO is None:
                continue
            R = dO[a, h]
            ref["dv"][b, h // G] += P.T @ R
            mag["dv"][b, h // G] += P.T @ np.abs(R)
            M = R @ V.T
            dS = P * (M - (P * M).sum(1, keepdims=True))
            ref["dq"][a, h] = scale * (dS @ K)
            ref["dk"][b, h // G] += scale * (dS.T @ Q)
            X = P * (np.abs(R) @ np.abs(V).T + (mag["o"][a, h] * np.abs(R)).sum(1, keepdims=True))
            mag["dq"][a, h] = scale * (X @ np.abs(K))
            mag["dk"][b, h // G] += scale * (X.T @ np.abs(Q))
    return ref, mag, top
