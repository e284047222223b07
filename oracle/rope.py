"""Rotary positions over several axes and the per-head norm before them
(oracle; test infrastructure only), in float64.

Definitions, per token n, head h and pair j of the d channels of a row:
  * pairs are dealt to the axes in order, n_a to axis a; pair j_a of axis a at
    position p has the angle (start + step * p) * theta ** (-j_a / n_a);
    pairs behind the last axis, and tokens or axes without a position
    (negative), have the angle 0;
  * pair j joins channels 2j and 2j + 1 ("adjacent") or j and j + d/2
    ("split"); read as a complex number, it is multiplied by exp(i angle);
  * the norm divides a row by sqrt(mean of its squares + eps) and multiplies
    it by the weights, before the rotation.
"""
from __future__ import annotations

import numpy as np


def axis_angles(length, pairs, theta=10000.0, start=0.0, step=1.0):
    """[length, pairs] angles of one axis."""
    p = start + step * np.arange(length, dtype=np.float64)
    return p[:, None] * np.power(float(theta), -np.arange(pairs, dtype=np.float64) / max(pairs, 1))[None, :]


def grid_positions(grid, first, N):
    """[N, 3] positions of tokens in row-major order over the grid, -1 behind it."""
    pos = np.full((N, 3), -1, dtype=np.int64)
    n = int(np.prod(grid))
    pos[:n] = np.stack(np.unravel_index(np.arange(n), grid), 1) + np.asarray(first)
    return pos


def token_angles(angles, pos, d):
    """[N, d/2] angles of every token; ``angles``: one [len, pairs] per axis."""
    out = np.zeros((pos.shape[0], d // 2))
    j = 0
    for a, tab in enumerate(angles):
        p = pos[:, a]
        on = (p >= 0) & (p < tab.shape[0])
        out[on, j:j + tab.shape[1]] = tab[p[on]]
        j += tab.shape[1]
    return out


def _complex(x, pairing):
    d = x.shape[-1]
    if pairing == "adjacent":
        return x[..., 0::2] + 1j * x[..., 1::2]
    return x[..., :d // 2] + 1j * x[..., d // 2:]


def _real(z, pairing):
    if pairing == "adjacent":
        return np.stack([z.real, z.imag], -1).reshape(*z.shape[:-1], -1)
    return np.concatenate([z.real, z.imag], -1)


def turn(x, ang, pairing):
    """x [N, H, d] turned by ang [N, d/2]."""
    return _real(_complex(x, pairing) * np.exp(1j * ang)[:, None, :], pairing)


def norm_turn(x, w, ang, pairing, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return turn(x * r * w, ang, pairing)


def norm_turn_back(gy, x, w, ang, pairing, eps):
    """(dx, dw) for the gradient gy of norm_turn's result."""
    g = turn(gy, -ang, pairing)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    gw = g * w
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdims=True))
    return dx, (g * xh).sum((0, 1))
