"""FP64 oracle of the recurrent form on a pool of states, and of the convolution on a pool of windows.

TEST INFRASTRUCTURE ONLY (see the package docstring).

N sequences take the tokens cu[n] .. cu[n+1]-1.  Sequence n starts from slot slot_in[n] (zero if -1); the
state after token t goes to slot slot_out[t] (nowhere if -1).  Sequences read the pool as it was before the call.  Per
token and value head h (q/k head h / G), with a_t = exp(g_t) a scalar or one value per key channel:

  S' = Diag(a) S;  S = S' + beta k^ (v - S'^T k^)^T;  o = scale S^T q^

The convolution: z = b + sum_i w[:, i] row(t - (W-1) + i), y = z sigma(z), where rows before the sequence's first
token are its window's; the window after token t holds the rows t-W+2 .. t.
"""
from __future__ import annotations

import numpy as np

EPS = 1e-6


def step(q, k, v, g, beta, states, cu, slot_in, slot_out, *, l2norm=True, scale=128 ** -0.5):
    """q, k [T, H, dk]; v [T, HV, dv]; g [T, HV] or [T, HV, dk]; beta [T, HV]; states [slots, HV, dk, dv].
    Returns o [T, HV, dv] and the new pool."""
    q, k, v, g, beta, states = (np.asarray(x, dtype=np.float64) for x in (q, k, v, g, beta, states))
    G = v.shape[1] // q.shape[1]
    if l2norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + EPS) for x in (q, k))
    o, pool = np.zeros(v.shape), states.copy()
    for n in range(len(cu) - 1):
        S = states[slot_in[n]].copy() if slot_in[n] >= 0 else np.zeros(states.shape[1:])
        for t in range(int(cu[n]), int(cu[n + 1])):
            for h in range(v.shape[1]):
                a = np.exp(g[t, h])
                S[h] *= a[:, None] if np.ndim(a) else a
                S[h] += beta[t, h] * np.outer(k[t, h // G], v[t, h] - S[h].T @ k[t, h // G])
                o[t, h] = scale * S[h].T @ q[t, h // G]
            if slot_out[t] >= 0:
                pool[slot_out[t]] = S
    return o, pool


def conv_step(x, w, b, window, cu, slot_in, slot_out):
    """x [T, C]; w [C, W]; b [C] or None; window [slots, W-1, C].  Returns y [T, C] and the new pool."""
    x, w, window = (np.asarray(a, dtype=np.float64) for a in (x, w, window))
    W = w.shape[1]
    y, pool = np.zeros(x.shape), window.copy()
    for n in range(len(cu) - 1):
        old = window[slot_in[n]] if slot_in[n] >= 0 else np.zeros(window.shape[1:])
        rows = np.concatenate([old, x[int(cu[n]):int(cu[n + 1])]])
        for j in range(int(cu[n + 1]) - int(cu[n])):
            t = int(cu[n]) + j
            z = (w.T * rows[j:j + W]).sum(0) + (0.0 if b is None else np.asarray(b, dtype=np.float64))
            y[t] = z / (1.0 + np.exp(-z))
            if W > 1 and slot_out[t] >= 0:
                pool[slot_out[t]] = rows[j + 1:j + W]
    return y, pool
