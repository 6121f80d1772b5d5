"""The recurrent form keeps its states, sums and norms in FP32: errors against FP64 that a state or products of fewer bits
would exceed.

Two measures over all columns of all states (128 values each), and the same for o of FP32 rows:
  worst      A step's error in a column s, in the 2-norm, is at most 40 U (|s| + |v|): the decay 4, u's sum of 128 products
             21 (16 in a lane, 5 over lanes), the norm of k, beta and the difference 14 on a d of no more than |u| + |v|, the
             update 1.  The rule contracts (unit keys, beta at most 1), so it decays with the state:
             E_t = 40 U (|s_t| + |v_t|) + max(a_t) E_{t-1}.
  typical    The root of the mean square of (error / size) is at most 8 times that of the recurrence taken in FP32 by
             NumPy: sums in another order, and room for a decay's exponential that is off by a few last places.
A copy that keeps its state in 11 bits, or takes its products of 11 bits' operands, fails the second."""
import numpy as np
import pytest
import torch

from tests.step_testutil import TYPES, U, f64

SHAPES = [   # (lengths, H, HV): single tokens, a few, few heads in blocks, many heads in blocks
    ([1] * 4, 16, 48), ([1] * 3, 2, 4), ([5, 9, 3], 16, 48), ([20, 11], 1, 3), ([257], 2, 6), ([64, 100], 1, 3),
    ([90, 61], 13, 52), ([1, 0, 300], 2, 4),
]


def short(x, bits):
    """x to `bits` bits of mantissa."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 2.0 ** bits), e - bits)


def recurrence(x, kda, dtype=np.float64, state_bits=None, operand_bits=None):
    """(o [T, HV, 128], the state after each sequence, per token the column sizes |s| + |v| [T, HV, 128]) from the slots 0,
    1, .., in one type."""
    cut = (lambda a: a) if operand_bits is None else (lambda a: short(a, operand_bits).astype(dtype))
    q, k, v, g, beta, S0 = (f64(x[n]).astype(dtype) for n in ("q", "k", "v", "g", "beta", "states"))
    q, k = (a / np.sqrt((a * a).sum(-1, keepdims=True) + dtype(1e-6)) for a in (q, k))
    G, a = v.shape[1] // q.shape[1], np.exp(g)
    q, k = (np.repeat(y, G, 1) for y in (q, k))
    o, size, ends = np.zeros_like(v), np.zeros(v.shape), []
    for n in range(len(x["cu"]) - 1):
        S = S0[n].copy()
        for t in range(int(x["cu"][n]), int(x["cu"][n + 1])):
            S *= a[t][:, :, None] if kda else a[t][:, None, None]
            u = np.matmul(cut(k[t])[:, None, :], cut(S))[:, 0]
            d = beta[t][:, None] * (v[t] - u)
            S += cut(k[t])[:, :, None] * cut(d)[:, None, :]
            if state_bits is not None:
                S = short(S, state_bits).astype(dtype)
            o[t] = dtype(128 ** -0.5) * np.matmul(cut(q[t])[:, None, :], cut(S))[:, 0]
            size[t] = np.sqrt((S.astype(np.float64) ** 2).sum(1)) + np.abs(v[t])
        ends.append(S)
    return o, np.stack(ends), size


def worst(x, kda, size):
    """E after every token [T, HV, 128]."""
    a = np.exp(f64(x["g"]))
    a = a.max(-1) if kda else a
    E = np.zeros(size.shape)
    for n in range(len(x["cu"]) - 1):
        before = 0.0
        for t in range(int(x["cu"][n]), int(x["cu"][n + 1])):
            before = E[t] = 40 * U * size[t] + a[t][:, None] * before
    return E


def measures(x, kda, exact, states, o=None):
    """(the largest error by its worst-case bound, the typical error) of the states, and of o where it is given."""
    want_o, want, size = exact
    E, ends = worst(x, kda, size), [int(e) - 1 for e, b in zip(x["cu"][1:], x["cu"][:-1]) if e > b]
    some = [n for n in range(len(want)) if x["cu"][n + 1] > x["cu"][n]]
    off = np.sqrt(((states - want)[some] ** 2).sum(2))
    got = [(off / E[ends]).max(), np.sqrt(((off / size[ends]) ** 2).mean())]
    if o is not None:   # 25 U |s| of its own sum, and one rounding
        tol = 128 ** -0.5 * (E + 25 * U * size) + U * np.abs(want_o) + 2.0 ** -149
        got += [(np.abs(o - want_o) / tol).max(), np.sqrt(((np.abs(o - want_o) / size) ** 2).mean())]
    return np.array(got)


def case(shape, dtype, kda):
    from tests.test_gpu_step import make
    lens, H, HV = shape
    return make(lens, H, HV, len(lens), dtype, kda, seed=sum(lens) + HV + kda)


@pytest.mark.gpu
@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_states_are_as_near_as_fp32(shape, dtype, kda):
    from tests.test_gpu_step import run
    x = case(shape, dtype, kda)
    o, pool, status = run(x, kda, None, None)
    assert status == 0
    exact, plain = recurrence(x, kda), recurrence(x, kda, np.float32)
    own = f64(o) if dtype == "fp32" else None
    got, ref = measures(x, kda, exact, f64(pool), own), measures(x, kda, exact, plain[1], plain[0])[:4 if dtype == "fp32" else 2]
    assert (got[::2] <= 1).all(), got
    assert (got[1::2] <= 8 * ref[1::2]).all(), (got, ref)


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("shape", SHAPES[-5:], ids=str)
def test_fewer_bits_are_seen(shape, kda):
    """The FP32 recurrence passes; states of 11 bits, and products of 11 bits' operands, do not."""
    x = case(shape, "fp32", kda)
    exact = recurrence(x, kda)
    ref = measures(x, kda, exact, *recurrence(x, kda, np.float32)[1::-1])
    assert (ref[::2] <= 1).all()
    for fewer in (dict(state_bits=11), dict(operand_bits=11)):
        got = measures(x, kda, exact, *recurrence(x, kda, np.float32, **fewer)[1::-1])
        assert (got[1::2] > 8 * ref[1::2]).all(), (fewer, got, ref)
