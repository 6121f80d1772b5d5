"""The recurrent form of the linear attention on a pool of states, against the FP64 oracle."""
import numpy as np
import pytest
import torch

import linear_attention_gdn_gb300 as gdn
from oracle import la
from tests.step_testutil import TINY, TYPES, U, f64, strided, within

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def run(lengths, H, HV, dtype="bf16", keep="last", fresh=(), spare=2, pad=0, decay=None, seed=0, cu=None, slot_in="own",
        tail=0):
    """One call and its oracle; the outputs and the pool are checked.  tail: rows behind the last sequence."""
    dt, unit = TYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    N, n = len(lengths), int(sum(lengths))
    T = n + tail
    r = np.random.default_rng(seed)
    order = r.permutation(N + (n if keep == "all" else 0) + spare).astype(np.int32)
    slots = len(order)
    home = order[:N] if slot_in == "own" else np.arange(N, dtype=np.int32)
    start = home.copy()
    start[list(fresh)] = -1
    starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    out = np.full(T, -1, np.int32)
    if keep == "all":
        out[:n] = order[N:N + n]
    for i in range(N):
        if keep == "last" and lengths[i]:
            out[starts[i + 1] - 1] = home[i]
    q, k, v = (torch.randn(T, h, 128, generator=g).to(dt) for h in (H, H, HV))
    states = torch.randn(slots, HV, 128, 128, generator=g)
    dec = -torch.logspace(-0.3, -3, HV) if decay is None else torch.full((HV,), decay)
    dq, dk, dv = (strided(t.cuda(), t.shape[1] * 128 + pad, 128) if pad else t.cuda() for t in (q, k, v))
    pool, o = states.cuda(), torch.full((T, HV, 128), float("nan"), dtype=dt, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    prob = gdn.step_problem(T, N, H, HV, slots, SCALE, False, dt, tuple(t.stride(0) for t in (dq, dk, dv)))
    on = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    gdn.gdn_la_step(prob, dq, dk, dv, dec.cuda(), pool, o, err, None if cu is None and tail == 0 and set(lengths) == {1} else on(starts),
                    None if slot_in is None else on(start), None if keep is None else on(out))
    assert gdn.gdn_device_status(err) == 0
    Q, K, V, S0 = f64(q), f64(k), f64(v), f64(states)
    want, ow, ot = S0.copy(), np.zeros((n, HV, 128)), np.zeros((n, HV, 128))
    tol = np.zeros_like(want)
    for i in range(N):
        a, b = starts[i], starts[i + 1]
        for h in range(HV):
            j = h // (HV // H)
            s = S0[start[i], h] if start[i] >= 0 else None
            oo, S = la.forward(Q[a:b, j], K[a:b, j], V[a:b, h], float(dec[h]), SCALE, s)
            _, A = la.forward(np.abs(Q[a:b, j]), np.abs(K[a:b, j]), np.abs(V[a:b, h]), float(dec[h]), SCALE, None if s is None else np.abs(s))
            ow[a:b, h] = oo
            for t in range(b - a):
                # the state: a product and a sum a token, and exp's 2 last places; the output: 128 products of that, summed
                # in at most 20 steps, and k.q the same
                e = (4 * (t + 1) + 2) * U * A[t + 1]
                ot[a + t, h] = SCALE * (e + 26 * U * A[t + 1]).T @ np.abs(Q[a + t, j]) + unit * np.abs(oo[t])
                if (to := out[a + t] if keep else (home[i] if t == b - a - 1 and start[i] >= 0 else -1)) >= 0:
                    want[to, h], tol[to, h] = S[t + 1], e
    within("o", o[:n], ow, ot + TINY)
    assert o[n:].isnan().all()
    within("states", pool, want, tol)
    return o, pool


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("lengths,H,HV", [([1], 1, 1), ([1], 16, 48), ([1] * 5, 2, 6), ([1] * 40, 4, 4), ([3], 1, 2), ([2, 0, 7, 1], 2, 2),
                                          ([5, 1, 9], 8, 32), ([33], 1, 3)])
def test_lengths(dtype, lengths, H, HV):
    run(lengths, H, HV, dtype, seed=len(lengths))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("lengths", [[4], [1, 8, 0, 3]])
def test_every_tokens_state(dtype, lengths):
    run(lengths, 2, 4, dtype, keep="all", fresh=[0])


@pytest.mark.parametrize("N", [3, 30])
def test_own_slots_and_zero_states(N):
    run([1] * N, 2, 2, fresh=[1])
    run([1] * N, 2, 2, slot_in=None)
    run([2] * N, 2, 2, slot_in=None, keep=None)
    run([2, 0, 1], 2, 2, fresh=[0, 2], keep=None)


@pytest.mark.parametrize("decay", [0.0, -20.0, float("-inf")])
def test_decays(decay):
    run([1, 5], 1, 2, decay=decay)


@pytest.mark.parametrize("pad", [8, 72])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_strides_and_rows_behind(pad, dtype):
    run([2, 3], 1, 2, dtype, pad=pad, tail=3)


def test_single_tokens_are_a_sequences_bits():
    """A sequence's tokens in one call or one by one: the same bits."""
    g = torch.Generator().manual_seed(2)
    for H, HV, N in ((1, 2, 2), (4, 8, 12)):
        q, k, v = (torch.randn(3 * N, h, 128, generator=g).bfloat16().cuda() for h in (H, H, HV))
        dec, err = -torch.rand(HV, generator=g).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
        pool = torch.randn(N, HV, 128, 128, generator=g).cuda()
        one, o = pool.clone(), torch.empty_like(v)
        cu = torch.arange(N + 1, dtype=torch.int32, device="cuda") * 3
        gdn.gdn_la_step(gdn.step_problem(3 * N, N, H, HV, N, l2norm=False), q, k, v, dec, pool, o, err, cu)
        for t in range(3):
            x = [y.view(N, 3, -1, 128)[:, t].contiguous() for y in (q, k, v)]
            p = torch.empty_like(x[2])
            gdn.gdn_la_step(gdn.step_problem(N, N, H, HV, N, l2norm=False), *x, dec, one, p, err)
            assert torch.equal(p, o.view(N, 3, HV, 128)[:, t])
        assert torch.equal(one, pool)


def test_bad_tables_are_reported_and_left_out():
    H, HV, N = 1, 2, 3
    x = [torch.randn(N, h, 128, device="cuda").bfloat16() for h in (H, H, HV)]
    dec = torch.zeros(HV, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for cu, slot_in, slot_out, skipped in ((None, i32(0, 3, 1), None, [1]), (None, i32(-2, 1, 2), None, [0]), (i32(0, 1, 1, 4), None, None, [1, 2]),
                                           (i32(0, 2, 1, 3), None, None, []), (None, None, i32(0, 7, 2), []), (None, None, i32(-3, 1, 2), [])):
        pool, o = torch.zeros(3, HV, 128, 128, device="cuda"), torch.full((N, HV, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_la_step(gdn.step_problem(N, N, H, HV, 3, l2norm=False), *x, dec, pool, o, err, cu, slot_in, slot_out)
        assert gdn.gdn_device_status(err) == 7
        assert all(o[i].isnan().all() for i in skipped)
        assert pool.isfinite().all()
