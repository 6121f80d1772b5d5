"""The convolution step (gdn_conv1d_step) with bounds that are none: the error word is set wherever in the batch they
lie, what is wrong is skipped, and the sequences beside are served."""
import numpy as np
import pytest
import torch

from tests.test_gpu_conv_step import last_slots, make, run

pytestmark = pytest.mark.gpu


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


@pytest.mark.parametrize("C", [16, 10240])   # ranges of one token and of many
@pytest.mark.parametrize("lens,change,bad", [
    ([400, 0], {2: 500}, 1),             # a sequence behind the last token
    ([400, 0, 0], {2: 500, 3: 500}, 1),  # (and an empty one behind that)
    ([0, 400], {0: -5}, 0),              # a negative start in front of a sequence at 0
    ([200, 192, 0, 8], {3: 390}, 2),     # bounds that go back, between sequences
    ([392, 0, 8], {2: 380}, 1),
])
def test_bad_bounds_of_long_sequences_are_reported(lens, change, bad, C):
    """Few sequences of many tokens, whose ranges are not walked through the bad one."""
    N, T = len(lens), sum(lens)
    x = make(lens, C, 4, N + 1, "bf16", seed=C + N)
    good = run(x, None, None)
    assert good[2] == 0
    cu = x["cu"].copy()
    for i, v in change.items():
        cu[i] = v
    y, win, status = run(dict(x, cu=cu), None, None)
    assert status == 7
    assert torch.equal(win[bad].cpu(), x["window"][bad]) and torch.equal(win[N].cpu(), x["window"][N])
    first = min([T] + [int(v) for v in cu if 0 <= v <= T and v not in x["cu"]])   # (a start moved back overlaps what is before)
    assert torch.equal(y[:first], good[0][:first])
    for n in range(N):
        if n != bad and lens[n] and cu[n] == x["cu"][n] and cu[n + 1] == x["cu"][n + 1]:
            assert torch.equal(win[n], good[1][n])


@pytest.mark.parametrize("at,value", [(33000, 10 ** 6), (20001, 10 ** 6), (0, -3), (7, -1), (32999, 5)])
def test_bad_bounds_among_very_many_sequences_are_reported(at, value):
    rng = np.random.default_rng(6)
    lens = list(rng.integers(0, 3, 33000))
    x = make(lens, 8, 4, 33001, "bf16", seed=24)
    cu = x["cu"].copy()
    cu[at] = value
    _, win, status = run(dict(x, cu=cu), None, None)
    assert status == 7 and torch.equal(win[33000].cpu(), x["window"][33000])


def test_graph_replay_with_more_tokens_than_it_was_captured_for():
    """Replayed with lengths whose sum is past the captured T, at a sequence's start: reported, the others served."""
    import linear_attention_gdn_gb300 as gdn
    lens = [300, 60, 40]
    x = make(lens, 512, 4, 3, "bf16", seed=25)
    want = run(x, None, None)
    T, C = x["x"].shape
    win, y = x["window"].cuda(), torch.full((T, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.from_numpy(x["cu"]).cuda()
    d, w, b = x["x"].cuda(), x["w"].cuda(), x["b"].cuda()
    prob = gdn.conv_step_problem(T, 3, C, 3)
    gdn.gdn_conv1d_step(prob, d, w, b, win.clone(), y, err, cu_seqlens_dev=cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_conv1d_step(prob, d, w, b, win, y, err, cu_seqlens_dev=cu)
    assert gdn.gdn_device_status(err) == 0
    cu.copy_(torch.from_numpy(starts([300, 100, 70])))
    graph.replay()
    assert gdn.gdn_device_status(err) == 7
    assert torch.equal(y[:360], want[0][:360]) and torch.equal(win[0], want[1][0])
    assert torch.equal(win[2].cpu(), x["window"][2])


@pytest.mark.parametrize("lens", [[1, 1], [2, 2], [3, 40]])
@pytest.mark.parametrize("slot", [2, -2])
def test_width_one_reports_slots_outside_the_pool(lens, slot):
    """A convolution of one tap keeps no window, but its tables are checked like any other's."""
    x = make(lens, 16, 1, 2, "bf16", seed=26)
    good = run(x, [0, 1], list(last_slots(lens, [0, 1])), cu=None if lens == [1, 1] else "dev")
    assert good[2] == 0
    out = last_slots(lens, [0, slot])
    y, _, status = run(x, [0, 1], list(out), cu=None if lens == [1, 1] else "dev")
    assert status == 7 and torch.equal(y, good[0])


def test_more_tokens_than_ranges_of_256():
    """More tokens than 65,535 ranges (the rows of a grid) of 256 hold; the windows in place, y against FP64."""
    import linear_attention_gdn_gb300 as gdn
    W, C, T = 4, 8, 65535 * 256 + 257
    cu = np.array([0, 1000, 1000, 7000001, T - 2, T], np.int32)
    gen = torch.Generator(device="cuda").manual_seed(27)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, window = rnd(T, C).to(torch.bfloat16), rnd(5, W - 1, C).to(torch.bfloat16)
    w, b = 0.5 * rnd(C, W), 0.1 * rnd(C)
    y, win, err = torch.full_like(x, float("nan")), window.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_conv1d_step(gdn.conv_step_problem(T, 5, C, 5, W=W), x, w, b, win, y, err,
                        cu_seqlens_dev=torch.from_numpy(cu).cuda())
    assert gdn.gdn_device_status(err) == 0
    for n in range(5):
        a, e = int(cu[n]), int(cu[n + 1])
        rows = torch.cat([window[n], x[a:e]]).double()
        z = b.double() + sum(w[:, i].double() * rows[i:i + e - a] for i in range(W))
        want = z * torch.sigmoid(z)
        # W products and the sigmoid, in FP32, then one rounding to BF16
        most = w.double().abs().sum(1) * rows.abs().max() + b.double().abs()
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -24 + 1.1 * (W + 12) * 2.0 ** -24 * most
        assert ((y[a:e].double() - want).abs() <= tol).all(), n
        assert torch.equal(win[n].double(), rows[e - a:])


@pytest.mark.parametrize("way", ["single", "short", "long"])
def test_sigmoid_of_fp32_rows(way):
    """One tap of one: y = z / (1 + exp(-z)) of the rows themselves, relative to y's own size down to z = -87.  In 2^-24: the
    exponential's argument z log2(e) is rounded once, as is the constant (1.25 |z| of the exponential), the exponential 4,
    the sum 1, the reciprocal 2, the product 1."""
    T = 4096
    lens = {"single": [1] * T, "short": [4] * (T // 4), "long": [T]}[way]
    x = make(lens, 16, 1, len(lens), "fp32", bias=False, seed=28)
    x["w"][:] = 1.0
    x["x"] = torch.linspace(-87.0, 40.0, T * 16).reshape(T, 16)
    y, _, status = run(x, None, None, cu=None if way == "single" else "dev")
    z = x["x"].double()
    want = z / (1.0 + torch.exp(-z))
    assert status == 0
    assert ((y.cpu().double() - want).abs() <= (1.25 * z.abs() + 8) * 2.0 ** -24 * want.abs()).all()


def test_sigmoid_at_the_ends():
    """Infinities and NaN as the formula has them; values below the exponential's range are zero."""
    x = make([1] * 2, 8, 1, 2, "fp32", bias=False, seed=29)
    x["w"][:] = 1.0
    inf, nan = float("inf"), float("nan")
    x["x"][:] = torch.tensor([inf, -inf, nan, -100.0, -3e38, 3e38, 0.0, -0.0])
    y = run(x, None, None, cu=None)[0][0].cpu()
    assert y[0] == inf and torch.isnan(y[1]) and torch.isnan(y[2]) and y[5] == x["x"][0, 5]
    assert (y[[3, 4, 6, 7]] == 0).all()
