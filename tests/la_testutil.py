"""Shared by the GPU tests of the linear attention: inputs, the oracle over packed documents, and its tolerances."""
import numpy as np
import torch

from oracle import la
from tests.step_testutil import f64, strided

R = 2.0 ** -8     # of one rounding to BF16
CH = 128          # tokens of the kernels' chunks
SCALE = 128 ** -0.5


def make(lengths, H, HV, states=True, seed=0, decay=None):
    """Inputs on the CPU: q, k, v, dO BF16, states FP32, decays from 0.4 a token to one in a few thousand."""
    g = torch.Generator().manual_seed(seed)
    T, N = int(sum(lengths)), len(lengths)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = dict(q=n(T, H, 128).bfloat16(), k=(0.4 * n(T, H, 128)).bfloat16(), v=n(T, HV, 128).bfloat16(),
             dO=n(T, HV, 128).bfloat16(), s_in=n(N, HV, 128, 128) if states else None,
             ds_out=0.5 * n(N, HV, 128, 128) if states else None)
    x["decay"] = -torch.logspace(-0.4, -3.5, HV) if decay is None else torch.tensor(decay, dtype=torch.float32).expand(HV).clone()
    x["cu"] = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return x


def _spread(A, rows, row_decay, X, S):
    """What one walk's chunk adds up, in absolute values: |A| |rows| + a^.. |X| |S|."""
    return np.abs(A) @ np.abs(rows) + row_decay[:, None] * (np.abs(X) @ np.abs(S))


def expect(x, H, HV, backward=True):
    """{name: (value, tolerance)} of every output.

    Tolerances.  Each BF16 output is sum_c P_rc z_c + a^.. Z^T x_r with P and Z rounded to BF16 once (R each), then rounded
    itself (R): R (sum |P||z| + a^.. |Z|^T|x| + |out|), and a group's dq, dk the sum of these over its heads.  FP32 sums
    and products in between: at most 300 operations deep a chunk, 2^-15 of the absolute sums of the products x y z, which are
    at most 12 times (sqrt 128) sum |P||z| here on average; 2^-10 of the spread covers them.  States: FP32 with 3 terms of
    BF16 each (2^-25), 24 steps of the tensor core a chunk whose sums may be cut off below 2^-23 of them, powers to 3 2^-24, and
    one operation a chunk: (chunks + 40) 2^-22 of the sums of absolute values."""
    T, N, G = len(x["q"]), len(x["cu"]) - 1, HV // H
    q, k, v, dO = (f64(x[m]) for m in ("q", "k", "v", "dO"))
    out = {m: np.zeros((T, HV, 128)) for m in ("o", "dv", "to", "tv")}
    out.update({m: np.zeros((T, H, 128)) for m in ("dq", "dk", "tq", "tk")})
    out.update({m: np.zeros((N, HV, 128, 128)) for m in ("s_out", "ds_in", "ts", "tw")})
    for d in range(N):
        a, b = int(x["cu"][d]), int(x["cu"][d + 1])
        for h in range(HV):
            j, g = h // G, float(x["decay"][h])
            Q, K, V, DO = q[a:b, j], k[a:b, j], v[a:b, h], dO[a:b, h]
            s_in = None if x["s_in"] is None else f64(x["s_in"][d, h])
            ds = None if x["ds_out"] is None else f64(x["ds_out"][d, h])
            o, S = la.forward(Q, K, V, g, SCALE, s_in)
            dq, dk, dv, W = la.backward(Q, K, V, g, SCALE, DO, S, ds)
            _, Sabs = la.forward(np.abs(Q), np.abs(K), np.abs(V), g, SCALE, None if s_in is None else np.abs(s_in))
            *_, Wabs = la.backward(np.abs(Q), np.abs(K), np.abs(V), g, SCALE, np.abs(DO), Sabs, None if ds is None else np.abs(ds))
            n = b - a
            f = ((n + CH - 1) // CH + 40) * 2.0 ** -22
            out["o"][a:b, h], out["dv"][a:b, h], out["s_out"][d, h], out["ds_in"][d, h] = o, dv, S[n], W[0]
            out["dq"][a:b, j] += dq
            out["dk"][a:b, j] += dk
            out["ts"][d, h], out["tw"][d, h] = f * Sabs[n], f * Wabs[0]
            for c in range(0, n, CH):
                e = min(c + CH, n)
                t = np.arange(e - c)
                w = np.where(t[:, None] >= t, np.exp(np.maximum(g, -1e4) * np.maximum(t[:, None] - t, 0)), 0.0)
                A, B = SCALE * w * (Q[c:e] @ K[c:e].T), SCALE * w * (DO[c:e] @ V[c:e].T)
                before, after = np.exp(np.maximum(g, -1e4) * (t + 1)), np.exp(np.maximum(g, -1e4) * (e - c - 1 - t))
                r = slice(a + c, a + e)
                out["to"][r, h] = _spread(A, V[c:e], SCALE * before, Q[c:e], S[c])
                out["tv"][r, h] = _spread(A.T, DO[c:e], after, K[c:e], W[e])
                out["tq"][r, j] += _spread(B, K[c:e], SCALE * before, DO[c:e], S[c].T)
                out["tk"][r, j] += _spread(B.T, Q[c:e], after, V[c:e], W[e].T)
    bf = lambda v, t: (out[v], (R + 2.0 ** -10) * out[t] + R * np.abs(out[v]) + 1e-30)  # noqa: E731
    return dict(o=bf("o", "to"), dq=bf("dq", "tq"), dk=bf("dk", "tk"), dv=bf("dv", "tv"),
                s_out=(out["s_out"], out["ts"]), ds_in=(out["ds_in"], out["tw"]))


def on_gpu(x, pad=0):
    """The inputs on the GPU; pad: so many values (a multiple of 8) of poison between the tokens' rows of q, k and v."""
    d = {m: t.cuda() if torch.is_tensor(t) else t for m, t in x.items()}
    d["cu_dev"] = torch.from_numpy(x["cu"]).cuda()
    if pad:
        for m in "qkv":
            t = x[m]
            d[m] = strided(t.cuda(), t.shape[1] * 128 + pad, 128)
    d["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return d
