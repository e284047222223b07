"""Gradient of masked softmax attention (oracle; test infrastructure only), in
float64, one head at a time:

  p = softmax(scale q k^T) over the allowed pairs (a query without any: 0)
  dv = p^T go,  ds = p * (go v^T - rowsum(go * o)),
  dq = scale ds k,  dk = scale ds^T q
"""
from __future__ import annotations

import numpy as np


def probabilities(q, k, scale, mask):
    s = np.where(mask, scale * (q @ k.T), -np.inf)
    m = s.max(1, keepdims=True)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    l = e.sum(1, keepdims=True)
    return np.divide(e, l, out=np.zeros_like(e), where=l > 0)


def attention_back(go, q, k, v, scale, mask):
    """(dq, dk, dv), each [N, H, d]; mask [N, N] or [H, N, N]."""
    out = [np.zeros_like(q) for _ in range(3)]
    for h in range(q.shape[1]):
        p = probabilities(q[:, h], k[:, h], scale, mask if mask.ndim == 2 else mask[h])
        g = go[:, h]
        ds = p * (g @ v[:, h].T - (g * (p @ v[:, h])).sum(1, keepdims=True))
        out[0][:, h] = scale * ds @ k[:, h]
        out[1][:, h] = scale * ds.T @ q[:, h]
        out[2][:, h] = p.T @ g
    return tuple(out)
