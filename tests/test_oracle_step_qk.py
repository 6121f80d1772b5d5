"""Pins of the FP64 oracles of the recurrent step, the convolution on windows and the q/k norm with rotation
against things fixed independently of them: the per-token KDA oracle, the packed convolution oracle, the
rotation's group law and finite differences of every gradient."""
import numpy as np
import pytest

from oracle import conv1d, kda, qk, step


@pytest.mark.parametrize("per_channel", [False, True])
def test_step_is_the_recurrence_cut_into_calls(per_channel):
    """A sequence taken in two calls through the pool is the per-token KDA oracle's run over the whole of it."""
    rng = np.random.default_rng(0)
    L, H, HV, D = 9, 2, 4, 6
    q, k = rng.standard_normal((2, L, H, D))
    v = rng.standard_normal((L, HV, D))
    g = -rng.random((L, HV, D)) if per_channel else -rng.random((L, HV))
    beta = rng.random((L, HV))
    pool = rng.standard_normal((3, HV, D, D))
    outs, cut = [], 4
    for a, b in ((0, cut), (cut, L)):
        slot_out = np.full(b - a, -1)
        slot_out[-1] = 2
        o, pool = step.step(q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], pool, [0, b - a], [-1 if a == 0 else 2], slot_out)
        outs.append(o)
    o = np.concatenate(outs)
    gk = g if per_channel else np.repeat(g[..., None], D, -1)
    for h in range(H):
        hv = slice(h * 2, h * 2 + 2)
        r = kda.group(q[:, h], k[:, h], v[:, hv].transpose(1, 0, 2), gk[:, hv].transpose(1, 0, 2), beta[:, hv].T)
        assert np.allclose(o[:, hv], r["o"].transpose(1, 0, 2), rtol=1e-12, atol=1e-14)
        assert np.allclose(pool[2, hv], r["s_out"], rtol=1e-12, atol=1e-14)


def test_conv_step_is_the_packed_convolution_cut_into_calls():
    rng = np.random.default_rng(1)
    L, C, W = 11, 3, 4
    x, w, b = rng.standard_normal((L, C)), rng.standard_normal((C, W)), rng.standard_normal(C)
    pool = rng.standard_normal((2, W - 1, C))
    outs = []
    for i, (a, e) in enumerate(((0, 1), (1, 3), (3, 4), (4, 11))):
        out = np.full(e - a, -1)
        out[-1] = 1
        y, pool = step.conv_step(x[a:e], w, b, pool, [0, e - a], [-1 if i == 0 else 1], out)
        outs.append(y)
    assert np.allclose(np.concatenate(outs), conv1d.forward(x, w, b, [0, L]), rtol=1e-13, atol=1e-14)
    assert np.array_equal(pool[1], x[-(W - 1):])


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rotation_keeps_lengths_and_depends_on_distance(layout):
    f = np.array([1.0, 0.3, 0.01])
    R = [qk.rotation(p, f, 8, 6, layout, 1.0) for p in (5, 12)]
    assert np.allclose(R[0] @ R[0].T, np.eye(8), atol=1e-15)
    assert np.allclose(R[0].T @ R[1], qk.rotation(7, f, 8, 6, layout, 1.0), atol=1e-14)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
def test_qk_gradients_by_differences(layout, norm):
    rng = np.random.default_rng(2)
    T, H, D, rot = 3, 2, 8, 6
    x, dy = rng.standard_normal((2, T, H, D))
    w = 1 + 0.3 * rng.standard_normal(D)
    f, pos = np.array([1.0, 0.4, 0.05]), np.array([3, 0, 17])
    kw = dict(rot=rot, layout=layout, norm=norm, eps=1e-3, m=1.2)
    dx, dw = qk.backward(x, w, f, pos, dy, **kw)
    loss = lambda x, w: (qk.forward(x, w, f, pos, **kw) * dy).sum()  # noqa: E731
    e = 1e-6
    for idx in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[idx] = e
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * e) - dx[idx]) < 1e-8
    for i in range(D):
        d = np.zeros(D)
        d[i] = e
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * e) - dw[i]) < 1e-8
