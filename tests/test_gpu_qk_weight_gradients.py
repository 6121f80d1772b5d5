"""The weights' gradients of the norm with rotation (gdn_qk_norm_rope_bwd), against FP64 to a bound that a lost part of the
sum exceeds.

dw[d] = sum over tokens and heads of g' x^.  With G = m (|g_a| + |g_b|) over a value's pair and X = |x r|, so that no
term exceeds G X:
  each term   r: a sum of squares (at most 16 additions in a lane and 5 over lanes, halved by the root), share and eps,
              the root: 14 roundings; the pair's two products, the sum, g' x and the step into the sum: 5; the sine and
              cosine within `angle` each:                                              (19 U + angle) G X
  the sum     a lane's chain, then up to 32 groups of a CTA in order, 64 CTAs an SM over 128 threads (76), and 7 of
              the tree:                                                                (chain + 115) U sum |g' x^|
where a lane's chain is at most twice its even share (whole runs of heads) of the rows over 152 CTAs of four warps, and 16.
Angles: FP32 rows by sincospi of a turn's fraction (6 U); 16-bit rows by the hardware's functions (2^-20, 16 U)."""
import numpy as np
import pytest
import torch

from oracle import qk as oracle
from tests.step_testutil import TYPES, U, f64
from tests.test_gpu_qk import freqs, make, run


def terms(a, g, freq, pos, *, rot, layout, norm, eps, m):
    """(g' x^, G X) [T, heads, D] in FP64: the rotation by pairs, all tokens together."""
    r, _ = oracle._r(a, norm, eps)
    ang = np.fmod(np.asarray(pos, np.longdouble)[:, None] * np.asarray(freq, np.longdouble), 2 * np.longdouble(np.pi))
    c, s = (m * f(ang.astype(np.float64))[:, None, :] for f in (np.cos, np.sin))
    turned, size = g.copy(), np.abs(g)
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    if rot:
        turned[..., i], turned[..., j] = g[..., i] * c + g[..., j] * s, g[..., j] * c - g[..., i] * s
        size[..., i] = size[..., j] = abs(m) * (np.abs(g[..., i]) + np.abs(g[..., j]))
    return turned * (a * r), size * np.abs(a * r)


def bound(term, size, dtype):
    rows, D = term.shape[0] * term.shape[1], term.shape[2]
    lanes = 8 if D <= 64 else 16 if D <= 128 else 32   # (fewer, where three pieces lie in one: more rows at a time)
    chain = 2 * rows / (152 * 4 * (32 // lanes)) + 16
    angle = 6 * U if dtype == "fp32" else 2.0 ** -20
    return (chain + 115) * U * np.abs(term).sum((0, 1)) + (19 * U + angle) * size.sum((0, 1))


KW = dict(rot=128, layout="half", norm="rms", eps=1e-6, m=1.0)
CASES = [   # (T, HQ, HK, D, dtype, other than KW)
    (12000, 16, 4, 128, "bf16", {}), (9001, 24, 3, 96, "fp32", dict(rot=48, layout="pairs", norm="l2")),
    (6007, 7, 1, 80, "bf16", dict(rot=80)), (6007, 7, 1, 80, "fp16", dict(rot=20, norm="l2")),
    (3001, 20, 5, 8, "bf16", dict(rot=8)), (700, 16, 16, 128, "bf16", dict(layout="pairs")),
    (20000, 1, 1, 64, "bf16", dict(rot=64, m=1.2)), (3000, 8, 2, 256, "bf16", dict(rot=64)),
    (4000, 8, 2, 192, "fp16", dict(rot=192, layout="pairs")), (3000, 4, 2, 130, "fp32", dict(rot=64)),
    (5000, 6, 2, 33, "bf16", dict(rot=32, norm="none")), (1, 2, 1, 128, "fp32", {}),
]


def problem(case):
    T, HQ, HK, D, dtype, other = case
    kw = {**KW, "eps": 1e-6, **other}
    rng = np.random.default_rng(T + D)
    return make(T, HQ, HK, D, dtype, seed=T + D), freqs(kw["rot"]), rng.integers(0, 300000, T), kw


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_weight_gradients(case):
    x, f, pos, kw = problem(case)
    got = run(x, f, pos=pos.tolist(), **kw)
    for i, n in enumerate(("q", "k")):
        term, size = terms(f64(x[n]), f64(x["g" + n]), f, pos, **kw)
        off, tol = np.abs(f64(got[4 + i]) - term.sum((0, 1))), bound(term, size, x["dtype"])
        assert (off <= tol).all(), (n, (off / tol).max())


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_a_lost_part_of_the_sum_is_seen(case):
    """The bound is below the whole, and below what one CTA's partial sums hold (there are at most 64 CTAs an SM, of four
    warps with a row each at least)."""
    x, f, pos, kw = problem(case)
    for n in ("q", "k"):
        term, size = terms(f64(x[n]), f64(x["g" + n]), f, pos, **kw)
        tol = bound(term, size, x["dtype"])
        whole = term.sum((0, 1))
        assert (np.abs(whole) > tol).any()
        rows = term.reshape(-1, term.shape[2])
        part = rows[-max(1, len(rows) // (152 * 64)) * 4:]
        assert (np.abs(part.sum(0)) > tol).any()


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
def test_terms_are_the_oracles(layout, norm):
    rng = np.random.default_rng(5)
    a, g = rng.standard_normal((2, 9, 3, 12))
    f, pos, kw = np.array([1.0, 0.3, 0.01]), np.arange(9) * 1001, dict(rot=6, layout=layout, norm=norm, eps=1e-3, m=1.3)
    term, size = terms(a, g, f, pos, **kw)
    want = oracle.backward(a, None, f, pos, g, **kw)[1]
    assert np.allclose(term.sum((0, 1)), want, rtol=1e-12, atol=1e-13)
    assert (np.abs(term) <= size * (1 + 1e-12)).all()
