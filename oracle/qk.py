"""FP64 oracle of the norm of q and k per head with the position rotation, forward and backward.

TEST INFRASTRUCTURE ONLY (see the package docstring).

For rows x [T, heads, D] of tokens at positions p [T]:
  x^ = x r, r = 1/sqrt(mean(x x) + eps) ("rms"), 1/sqrt(sum(x x) + eps) ("l2"), 1 ("none");  z = w x^
  y  = z with each pair i of its first rot values turned by the angle p f_i and scaled by m
the pairs (i, i + rot/2) ("half") or (2i, 2i + 1) ("pairs").  The rotation is applied as the full D x D matrix
of each position, and the backward is its transpose:
  g' = R^T dy;  dw = sum g' x^;  dx = r (w g' - x^ c sum(w g' x^)), c = 1/D, 1, 0
"""
from __future__ import annotations

import numpy as np


def rotation(p, freq, D, rot, layout, m):
    """The D x D matrix at position p."""
    R = np.eye(D)
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        # the angle is reduced before it is rounded to 64 bits: p is exact, f has 53 bits
        ang = float(np.fmod(np.longdouble(p) * np.longdouble(freq[i]), 2 * np.longdouble(np.pi)))
        R[a, a] = R[b, b] = m * np.cos(ang)
        R[a, b], R[b, a] = -m * np.sin(ang), m * np.sin(ang)
    return R


def positions(T, cu=None):
    """0, 1, ... in each document of cu (0, 1, ... T-1 without)."""
    if cu is None:
        return np.arange(T)
    return np.concatenate([np.arange(int(b) - int(a)) for a, b in zip(cu[:-1], cu[1:])])


def _r(x, norm, eps):
    ss = (x * x).sum(-1, keepdims=True)
    if norm == "none":
        return np.ones_like(ss), 0.0
    D = x.shape[-1]
    return (1 / np.sqrt(ss / D + eps), 1.0 / D) if norm == "rms" else (1 / np.sqrt(ss + eps), 1.0)


def forward(x, w, freq, pos, *, rot, layout="half", norm="rms", eps=1e-6, m=1.0):
    x = np.asarray(x, dtype=np.float64)
    z = x * _r(x, norm, eps)[0] * (1.0 if w is None else np.asarray(w, dtype=np.float64))
    return np.stack([z[t] @ rotation(pos[t], freq, x.shape[-1], rot, layout, m).T for t in range(x.shape[0])]) \
        if x.shape[0] else z


def backward(x, w, freq, pos, dy, *, rot, layout="half", norm="rms", eps=1e-6, m=1.0):
    """(dx, dw)."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, dtype=np.float64)
    r, c = _r(x, norm, eps)
    g = np.zeros_like(x)
    for t in range(x.shape[0]):
        g[t] = dy[t] @ rotation(pos[t], freq, x.shape[-1], rot, layout, m)
    xh = x * r
    return r * (w * g - xh * c * (w * g * xh).sum(-1, keepdims=True)), (g * xh).sum((0, 1))
