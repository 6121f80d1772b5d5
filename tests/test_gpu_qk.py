"""GPU parity of the norm of q and k per head with the position rotation (gdn_qk_norm_rope_fwd / _bwd) against the
FP64 oracle.

Tolerances: a row's sums of D products and the few operations after them are each rounded by 2^-24, relative to the
row's largest value (forward) or the norm of w g' r (backward); the angle is rounded to 2^-24 of a turn, 2 pi of it in the 32.
One rounding to the type follows. A weight's gradient is a sum of one term a row."""
import numpy as np
import pytest
import torch

from oracle import qk as oracle
from tests.step_testutil import TINY, TYPES, U, f64, strided, within

pytestmark = pytest.mark.gpu
NORMS = {"none": 0, "rms": 1, "l2": 2}


def make(T, HQ, HK, D, dtype, seed=0, weights=True):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    dt = TYPES[dtype][0]
    x = {n: rnd(T, h, D).to(dt) for n, h in (("q", HQ), ("k", HK), ("gq", HQ), ("gk", HK))}
    x.update({n: 1 + 0.3 * rnd(D) if weights else None for n in ("wq", "wk")}, dtype=dtype)
    return x


def run(x, freq, rot, layout="half", norm="rms", eps=1e-6, m=1.0, pos=None, cu=None, pad=None, in_place=False, dw=True):
    """Forward and backward: (yq, yk, dq, dk, dwq, dwk)."""
    import linear_attention_gdn_gb300 as gdn
    T, HQ, D = x["q"].shape
    HK, dt = x["k"].shape[1], x["q"].dtype
    head = D if pad is None else D + pad
    token = {n: h * head + (0 if pad is None else pad) for n, h in (("q", HQ), ("k", HK))}
    st = {n: (token[n], head) for n in ("q", "k")}
    dev = lambda a, n: strided(a, max(token[n], 1), head)  # noqa: E731
    nan = lambda n: torch.full_like(x[n], float("nan"))  # noqa: E731
    cuda = lambda a: None if a is None else a.cuda()  # noqa: E731
    prob = gdn.qk_problem(T, HQ, HK, D=D, rot=rot, layout=0 if layout == "half" else 1, norm=NORMS[norm], eps=eps,
                          mscale=m, N=0 if cu is None else len(cu) - 1, dtype=dt, q_strides=st["q"], k_strides=st["k"],
                          qo_strides=st["q"], ko_strides=st["k"])
    f = torch.from_numpy(np.asarray(freq, np.float64)).cuda()
    p = None if pos is None else torch.tensor(pos, dtype=torch.int32, device="cuda")
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    d = {n: dev(x[n], n[-1]) for n in ("q", "k", "gq", "gk")}
    w = [cuda(x[n]) for n in ("wq", "wk")]
    xin = (d["q"], d["k"])
    if in_place:
        y = tuple(dev(x[n], n) for n in ("q", "k"))
        gdn.gdn_qk_norm_rope_fwd(prob, *y, *w, f, p, c, *y)
    else:
        y = tuple(dev(nan(n), n) for n in ("q", "k"))
        gdn.gdn_qk_norm_rope_fwd(prob, *xin, *w, f, p, c, *y)
    ws = torch.full((gdn.gdn_qk_workspace_bytes(prob),), 255, dtype=torch.uint8, device="cuda") if dw else None
    dws = [torch.full((D,), float("nan"), device="cuda") for _ in range(2)] if dw else [None, None]
    dx = (d["gq"], d["gk"]) if in_place else tuple(dev(nan(n), n) for n in ("q", "k"))
    gdn.gdn_qk_norm_rope_bwd(prob, *xin, *w, f, p, c, d["gq"], d["gk"], *dx, *dws, ws)
    torch.cuda.synchronize()
    return (*y, *dx, *dws)


def check(x, got, freq, rot, layout="half", norm="rms", eps=1e-6, m=1.0, pos=None, cu=None, **_):
    T, _, D = x["q"].shape
    u = TYPES[x["dtype"]][1]
    p = oracle.positions(T, cu) if pos is None else pos
    kw = dict(rot=rot, layout=layout, norm=norm, eps=eps, m=m)
    for i, n in enumerate(("q", "k")):
        a, w, g = f64(x[n]), None if x["w" + n] is None else f64(x["w" + n]), f64(x["g" + n])
        y = oracle.forward(a, w, freq, p, **kw)
        r, _ = oracle._r(a, norm, eps)
        ww = np.ones(D) if w is None else w
        size = np.abs(a * r * ww).max(-1, keepdims=True) * max(m, 1.0) if a.size else a
        within("y" + n, got[i], y, u * np.abs(y) + TINY + 2 * (D + 32) * U * size)
        dx, dw = oracle.backward(a, w, freq, p, g, **kw)
        gsize = np.linalg.norm(g, axis=-1, keepdims=True) * max(m, 1.0) * np.abs(ww).max()
        within("d" + n, got[2 + i], dx, u * np.abs(dx) + TINY + 4 * (D + 32) * U * r * gsize)
        if got[4 + i] is not None:
            each = np.abs(a * r).max(initial=0) * np.abs(g).max(initial=0) * max(m, 1.0) * 2
            rows = T * a.shape[1]
            within("dw" + n, got[4 + i], dw, np.full(D, (D + 32 + rows) * U * each * rows))


def freqs(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2) / max(rot, 1))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 32), (64, 64), (256, 256), (96, 48), (80, 40), (192, 24), (8, 8),
                                   (40, 8)])
def test_vector_rows(D, rot, layout, dtype):
    """Head sizes and rotated parts that the 16-byte kernels take (whole rows, parts, parts that end inside a thread's 8
    values), shared k heads, packed documents with an empty one."""
    x = make(37, 6, 2, D, dtype, seed=D + rot)
    kw = dict(rot=rot, layout=layout, cu=[0, 5, 5, 30, 37])
    check(x, run(x, freqs(rot), **kw), freqs(rot), **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("D,rot,pad", [(128, 12, None), (33, 32, None), (7, 4, None), (1, 0, None), (320, 300, None),
                                       (512, 512, None), (64, 64, 3), (50, 50, 1)])
def test_rows_of_any_kind(D, rot, pad, layout, dtype):
    """Odd sizes and strides, parts that are not whole vectors."""
    x = make(19, 3, 2, D, dtype, seed=D)
    kw = dict(rot=rot, layout=layout, pad=pad, pos=[3 * i for i in range(19)])
    check(x, run(x, freqs(rot), **kw), freqs(rot), **kw)


@pytest.mark.parametrize("norm", list(NORMS))
@pytest.mark.parametrize("D,rot", [(128, 64), (30, 10)])
@pytest.mark.parametrize("weights", [True, False])
def test_norms_and_weights(norm, D, rot, weights):
    x = make(11, 4, 4, D, "fp32", seed=1, weights=weights)
    kw = dict(rot=rot, norm=norm, eps=1e-2, m=1.3)
    check(x, run(x, freqs(rot), **kw), freqs(rot), **kw)


@pytest.mark.parametrize("T", [1, 2, 700])
@pytest.mark.parametrize("HQ,HK", [(16, 16), (1, 0), (0, 3), (20, 5), (9, 1)])
def test_heads_and_lengths(T, HQ, HK):
    """One kind of head only, head counts that are no whole runs, single tokens; more tokens than the CTAs take at once."""
    if T == 700 and HQ == 20:
        T = 3001   # tiles of several tokens, several tiles a CTA
        x = make(T, HQ, HK, 8, "bf16", seed=2)
        rot = 8
    else:
        x, rot = make(T, HQ, HK, 128, "bf16", seed=T + HQ), 128
    check(x, run(x, freqs(rot), rot), freqs(rot), rot)


def test_strided_and_in_place():
    x = make(21, 5, 3, 128, "bf16", seed=3)
    kw = dict(rot=128, pad=16, pos=list(range(100, 121)))
    want = run(x, freqs(128), **kw)
    check(x, want, freqs(128), **kw)
    got = run(x, freqs(128), in_place=True, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = make(6, 2, 2, 30, "fp32", seed=4)
    kw = dict(rot=30, pad=2)
    want, got = run(x, freqs(30), **kw), run(x, freqs(30), in_place=True, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_far_positions_keep_their_angle(layout):
    pos = [0, 1, 524287, 10 ** 6 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -5]
    x = make(len(pos), 2, 2, 64, "fp32", seed=5)
    kw = dict(rot=64, layout=layout, pos=pos)
    check(x, run(x, freqs(64), **kw), freqs(64), **kw)


@pytest.mark.parametrize("D,rot", [(128, 64), (130, 64)])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_infinities_stay_in_their_values(layout, D, rot):
    """Without a norm an infinite or NaN value reaches its own pair only, and zero rows of a norm give zeros."""
    x = make(3, 1, 1, D, "fp32", seed=6)
    x["q"][0, 0, 70], x["q"][0, 0, 100], x["q"][1, 0, 3] = float("inf"), float("nan"), float("inf")
    y = run(x, freqs(rot), rot, layout=layout, norm="none")[0]
    bad = torch.zeros(3, 1, D, dtype=torch.bool)
    bad[0, 0, 70] = bad[0, 0, 100] = bad[1, 0, 3] = True
    bad[1, 0, 3 + rot // 2 if layout == "half" else 2] = True
    assert torch.equal(torch.isfinite(y.cpu()), ~bad)
    x["q"][:] = 0
    for norm in ("rms", "l2"):
        got = run(x, freqs(rot), rot, layout=layout, norm=norm)
        assert (got[0] == 0).all() and torch.isfinite(got[2]).all()


def test_reproducible_and_without_weight_gradients():
    x = make(900, 8, 2, 128, "bf16", seed=7)
    a, b = run(x, freqs(128), 128), run(x, freqs(128), 128)
    assert all(torch.equal(i, j) for i, j in zip(a, b))
    c = run(x, freqs(128), 128, dw=False)
    assert torch.equal(a[2], c[2]) and torch.equal(a[3], c[3])


def test_no_tokens_zero_the_weight_gradients():
    x = make(0, 2, 2, 64, "bf16")
    got = run(x, freqs(64), 64)
    assert (got[4] == 0).all() and (got[5] == 0).all()


def test_offsets_past_32_bits():
    """Rows past 2^31 elements of a packed tensor."""
    import linear_attention_gdn_gb300 as gdn
    T, row = 240000, 9216
    x = torch.empty((T, row), dtype=torch.bfloat16, device="cuda")   # 2.2e9 values
    part = make(64, 2, 2, 128, "bf16", seed=8)
    q, k = x[:, :256].unflatten(1, (2, 128)), x[:, 256:512].unflatten(1, (2, 128))
    q.zero_(), k.zero_()
    q[-64:], k[-64:] = part["q"].cuda(), part["k"].cuda()
    f = torch.from_numpy(freqs(128)).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % 64
    pos[-64:] = torch.arange(64, dtype=torch.int32, device="cuda")
    prob = gdn.qk_problem(T, 2, 2, dtype=torch.bfloat16, q_strides=(row, 128), k_strides=(row, 128),
                          qo_strides=(row, 128), ko_strides=(row, 128))
    gdn.gdn_qk_norm_rope_fwd(prob, q, k, part["wq"].cuda(), part["wk"].cuda(), f, pos, None, q, k)
    want = run(part, freqs(128), 128)
    assert torch.equal(q[-64:], want[0]) and torch.equal(k[-64:], want[1])


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype,D,rot,norm", [("bf16", 72, 72, "rms"), ("bf16", 80, 80, "l2"), ("fp16", 88, 24, "rms"),
                                              ("bf16", 96, 96, "rms"), ("fp16", 96, 8, "none"), ("bf16", 96, 0, "rms"),
                                              ("bf16", 136, 136, "rms"), ("fp16", 160, 40, "l2"),
                                              ("bf16", 192, 192, "rms"), ("bf16", 184, 96, "none")])
def test_rows_of_three_pieces_a_lane(dtype, D, rot, norm, layout):
    """Head sizes between powers of two, in enough rows: padded ones, also in place."""
    x = make(211, 5, 2, D, dtype, seed=D + rot)
    kw = dict(rot=rot, layout=layout, norm=norm, pad=8, pos=[7 * i - 3 for i in range(211)], m=1.1)
    want = run(x, freqs(rot), **kw)
    check(x, want, freqs(rot), **kw)
    got = run(x, freqs(rot), in_place=True, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 8, 100, 200])
@pytest.mark.parametrize("D", [96, 192])
def test_rows_around_the_choice_of_pieces(T, D):
    x = make(T, 9, 3, D, "fp16", seed=T)
    check(x, run(x, freqs(48), 48), freqs(48), 48)


@pytest.mark.parametrize("D,rot,layout", [(80, 80, "half"), (96, 48, "pairs"), (192, 96, "half")])
def test_many_rows_of_three_pieces_a_lane(D, rot, layout):
    x = make(6007, 7, 1, D, "bf16", seed=D)
    kw = dict(rot=rot, layout=layout, cu=[0, 1000, 1000, 6007])
    check(x, run(x, freqs(rot), **kw), freqs(rot), **kw)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("D", [96, 192])
def test_infinities_stay_in_their_values_of_three_pieces(layout, D):
    rot = D // 2
    x = make(1500, 1, 1, D, "bf16", seed=8)
    x["q"][0, 0, D - 9], x["q"][0, 0, D - 1], x["q"][1, 0, 3] = float("inf"), float("nan"), float("inf")
    y = run(x, freqs(rot), rot, layout=layout, norm="none")[0]
    bad = torch.zeros(1500, 1, D, dtype=torch.bool)
    bad[0, 0, D - 9] = bad[0, 0, D - 1] = bad[1, 0, 3] = True
    bad[1, 0, 3 + rot // 2 if layout == "half" else 2] = True
    assert torch.equal(torch.isfinite(y.cpu()), ~bad)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D,rot", [(80, 20), (96, 12), (128, 4), (64, 60), (256, 100), (192, 180), (8, 4), (136, 68)])
def test_halves_of_rotated_parts_that_are_4_and_a_multiple_of_8(D, rot, dtype):
    """A rotated half that is an even number of values, no multiple of 4: few rows, and enough for all kernels; padded."""
    for T in (5, 301):
        x = make(T, 4, 1, D, dtype, seed=D + rot)
        kw = dict(rot=rot, pad=8, norm="l2" if T == 5 else "rms", cu=[0, 3, T])
        want = run(x, freqs(rot), **kw)
        check(x, want, freqs(rot), **kw)
        got = run(x, freqs(rot), in_place=True, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [3, 1300])
def test_infinities_stay_in_their_values_of_such_halves(T):
    D, rot = 80, 20
    x = make(T, 1, 1, D, "bf16", seed=9)
    for d in (20, 22, 79):   # the first values that are not rotated, and the last
        x["q"][0, 0, d] = float("inf")
    x["q"][1, 0, 9], x["q"][2, 0, 11] = float("nan"), float("inf")
    y = run(x, freqs(rot), rot, norm="none")[0]
    bad = torch.zeros(T, 1, D, dtype=torch.bool)
    bad[0, 0, [20, 22, 79]] = bad[1, 0, [9, 19]] = bad[2, 0, [1, 11]] = True
    assert torch.equal(torch.isfinite(y.cpu()), ~bad)
