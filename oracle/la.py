"""FP64 linear attention with a fixed decay per head, token by token, and its reverse mode.

    S_t = a S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   a = exp(decay)

For one sequence and one value head: q, k [n, dk], v, dO [n, dv], S [dk, dv].  Test infrastructure only.
"""
import numpy as np


def forward(q, k, v, decay, scale, s_in=None):
    """(o [n, dv], S [n + 1, dk, dv]): S[0] is the state entered with, S[t + 1] the one after token t."""
    n, a = len(q), np.exp(np.float64(decay))
    S = np.zeros((n + 1, k.shape[1], v.shape[1]))
    if s_in is not None:
        S[0] = s_in
    o = np.zeros((n, v.shape[1]))
    for t in range(n):
        S[t + 1] = (a * S[t] if a else 0.0) + np.outer(k[t], v[t])
        o[t] = scale * (S[t + 1].T @ q[t])
    return o, S


def backward(q, k, v, decay, scale, dO, S, ds_out=None):
    """(dq, dk, dv, W [n + 1, dk, dv]): W[t] is the gradient of the state before token t that comes from token t on,
    W[n] = ds_out."""
    n, a = len(q), np.exp(np.float64(decay))
    W = np.zeros_like(S)
    if ds_out is not None:
        W[n] = ds_out
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for t in range(n - 1, -1, -1):
        dS = W[t + 1] + scale * np.outer(q[t], dO[t])
        dq[t] = scale * (S[t + 1] @ dO[t])
        dk[t] = dS @ v[t]
        dv[t] = dS.T @ k[t]
        W[t] = a * dS if a else 0.0
    return dq, dk, dv, W
