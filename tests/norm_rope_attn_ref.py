"""Bounds of the attention backward's error, element by element, for tests that
check its gradients on the way into the norm's backward."""
from __future__ import annotations

import numpy as np

LSE = 1e-3                 # what the stored LSE may be off by


def attention_bounds(q, k, v, mask, scale, dout):
    """(bound of dQ, bound of dK) of the bf16 tensor-core passes, [s][h][d], for
    exact rows q, k, v, dout [s][h][d] and the selected keys mask [h][s][s],
    before dQ and dK are rounded to storage.

    P = exp(scale q.k - LSE) is off by LSE's error and that of two 128-term
    fp32 sums of exact products (the tensor cores cut their sums off: under
    2^-16 of the absolute products), e P in all.  dP has the same sum.  D = sum
    P dP comes from an output made with P in bf16 (2^-8) and kept in fp16
    (2^-11).  dS = P (dP - D) is rounded to fp16 (2^-11, 2^-24 where it is
    subnormal); each block's share of dQ is too (2^-11, and 2^-24 for each of
    at most 2^7 blocks); the sums over keys are fp32 (2^-14)."""
    bq, bk = np.empty(q.shape), np.empty(k.shape)
    for h in range(q.shape[1]):
        Q, K, V, G, m = q[:, h], k[:, h], v[:, h], dout[:, h], mask[h]
        s = np.where(m, scale * (Q @ K.T), -np.inf)
        top = s.max(1, keepdims=True)
        p = np.where(m, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
        p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
        e = LSE + 2.0 ** -14 * scale * (np.abs(Q) @ np.abs(K).T) + 2.0 ** -18
        dp, a = G @ V.T, 2.0 ** -16 * (np.abs(G) @ np.abs(V).T)
        D = (p * dp).sum(1, keepdims=True)
        o = np.abs(G) * np.abs(p @ V)
        eD = (p * ((2.0 ** -8 + e) * np.abs(dp) + a)).sum(1, keepdims=True) + \
            2.0 ** -11 * o.sum(1, keepdims=True)
        size = np.abs(dp) + np.abs(D)
        ds = np.abs(p * (dp - D))
        err = p * (e * size + a + eD) * (1 + 2.0 ** -7) + 2.0 ** -11 * ds
        err = np.where(m, err + 2.0 ** -24, 0.0)
        more = 2.0 ** -11 + 2.0 ** -14
        bq[:, h] = scale * ((err + more * ds) @ np.abs(K) + 2.0 ** -17)
        bk[:, h] = scale * ((err + 2.0 ** -14 * ds).T @ np.abs(Q))
    return bq, bk
