"""Pins of the linear attention's oracle: its closed form, central differences, and a cut with the state carried over."""
import numpy as np
import pytest

from oracle import la


def inputs(n, seed=0, dk=5, dv=3):
    r = np.random.default_rng(seed)
    return [r.standard_normal(s) for s in ((n, dk), (n, dk), (n, dv), (n, dv), (dk, dv), (dk, dv))]


@pytest.mark.parametrize("decay", [0.0, -0.3, -4.0])
def test_closed_form(decay):
    q, k, v, _, s, _ = inputs(9)
    o, S = la.forward(q, k, v, decay, 0.7, s)
    t = np.arange(9)
    w = np.where(t[:, None] >= t, np.exp(decay * (t[:, None] - t)), 0.0)
    want = 0.7 * ((w * (q @ k.T)) @ v + np.exp(decay * (t + 1))[:, None] * (q @ s))
    np.testing.assert_allclose(o, want, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S[9], np.exp(9 * decay) * s + (k * np.exp(decay * (8 - t))[:, None]).T @ v, atol=1e-12)


def test_no_memory():
    q, k, v, _, s, _ = inputs(4)
    o, S = la.forward(q, k, v, -np.inf, 1.0, s)
    np.testing.assert_allclose(o, (q * k).sum(1)[:, None] * v, atol=1e-14)


@pytest.mark.parametrize("name", ["q", "k", "v", "s"])
def test_gradients_are_central_differences(name):
    q, k, v, dO, s, ds = inputs(7, seed=3)
    x = dict(q=q, k=k, v=v, s=s)

    def loss():
        o, S = la.forward(x["q"], x["k"], x["v"], -0.2, 0.6, x["s"])
        return (o * dO).sum() + (S[-1] * ds).sum()

    _, S = la.forward(q, k, v, -0.2, 0.6, s)
    dq, dk, dv, W = la.backward(q, k, v, -0.2, 0.6, dO, S, ds)
    got = dict(q=dq, k=dk, v=dv, s=W[0])[name]
    for i in np.ndindex(got.shape):
        at = x[name][i]
        h = 1e-5
        x[name][i] = at + h
        up = loss()
        x[name][i] = at - h
        down = loss()
        x[name][i] = at
        assert abs((up - down) / (2 * h) - got[i]) < 1e-7


@pytest.mark.parametrize("m", [1, 4, 6])
def test_a_cut_carries_the_states(m):
    q, k, v, dO, s, ds = inputs(7, seed=5)
    o, S = la.forward(q, k, v, -0.2, 1.0, s)
    dq, dk, dv, W = la.backward(q, k, v, -0.2, 1.0, dO, S, ds)
    o1, S1 = la.forward(q[:m], k[:m], v[:m], -0.2, 1.0, s)
    o2, S2 = la.forward(q[m:], k[m:], v[m:], -0.2, 1.0, S1[-1])
    np.testing.assert_array_equal(np.concatenate([o1, o2]), o)
    b2 = la.backward(q[m:], k[m:], v[m:], -0.2, 1.0, dO[m:], S2, ds)
    b1 = la.backward(q[:m], k[:m], v[:m], -0.2, 1.0, dO[:m], S1, b2[3][0])
    for whole, first, second in zip((dq, dk, dv), b1, b2):
        np.testing.assert_array_equal(np.concatenate([first, second]), whole)
    np.testing.assert_array_equal(b1[3][0], W[0])
