"""GPU parity of the convolution on a pool of windows (gdn_conv1d_step) against the FP64 oracle. Windows are copies of
input rows and have to be equal; y is within the FP32 errors of W products and the sigmoid (whose slope is at most
1.1), then rounded once."""
import numpy as np
import pytest
import torch

from oracle import step as oracle
from tests.step_testutil import TINY, TYPES, U, f64, strided, within

pytestmark = pytest.mark.gpu


def make(lens, C, W, slots, dtype, bias=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    dt = TYPES[dtype][0]
    return dict(x=rnd(int(sum(lens)), C).to(dt), w=0.5 * rnd(C, W), b=0.1 * rnd(C) if bias else None,
                window=rnd(slots, W - 1, C).to(dt), cu=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32),
                dtype=dtype)


def run(x, slot_in, slot_out, pad=0, cu="dev"):
    import linear_attention_gdn_gb300 as gdn
    (T, C), W, dt = x["x"].shape, x["w"].shape[1], x["x"].dtype
    d = strided(x["x"], C + pad)
    y = strided(torch.full((T, C), float("nan"), dtype=dt), C + pad)
    win = x["window"].cuda()
    prob = gdn.conv_step_problem(T, len(x["cu"]) - 1, C, x["window"].shape[0], W=W, dtype=dt,
                                 strides=(C + pad, C + pad) if pad else (0, 0))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = lambda a: None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    gdn.gdn_conv1d_step(prob, d, x["w"].cuda(), None if x["b"] is None else x["b"].cuda(), win, y, err,
                        cu_seqlens_dev=torch.from_numpy(x["cu"]).cuda() if cu == "dev" else cu,
                        slot_in=table(slot_in), slot_out=table(slot_out))
    return y, win, gdn.gdn_device_status(err)


def check(x, got, slot_in, slot_out):
    y, win, status = got
    assert status == 0
    want_y, want = oracle.conv_step(f64(x["x"]), f64(x["w"]), None if x["b"] is None else f64(x["b"]), f64(x["window"]),
                                    x["cu"], slot_in, slot_out)
    W = x["w"].shape[1]
    big = max(f64(x["x"]).__abs__().max(initial=0), f64(x["window"]).__abs__().max(initial=0))
    most = np.abs(f64(x["w"])).sum(1) * big + (0 if x["b"] is None else np.abs(f64(x["b"])))
    within("y", y, want_y, TYPES[x["dtype"]][1] * np.abs(want_y) + TINY + 1.1 * (W + 12) * U * most[None])
    assert np.array_equal(f64(win), want)


def last_slots(lens, slots):
    out = np.full(int(sum(lens)), -1)
    for n, end in enumerate(np.cumsum(lens)):
        if lens[n]:
            out[end - 1] = slots[n]
    return out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W", [1, 2, 3, 4])
def test_single_tokens(W, dtype):
    x = make([1] * 5, 40, W, 8, dtype, seed=W)
    slot_in, slot_out = [6, -1, 0, 3, 2], [6, 1, -1, 3, 7]
    check(x, run(x, slot_in, slot_out), slot_in, slot_out)
    check(x, run(x, slot_in, slot_out, pad=24, cu=None), slot_in, slot_out)


@pytest.mark.parametrize("lens", [[2, 0, 1, 3, 0, 0, 9, 4], [1, 2, 3, 4, 5, 6], [0, 0, 7], [200], [63, 1, 65, 2, 129, 64]])
def test_ragged_in_place(lens):
    """Sequences shorter and longer than the window and than a range of tokens, in place: whoever reads a window reads
    what was there before the call."""
    N = len(lens)
    x = make(lens, 64, 4, N + 1, "bf16", seed=7)
    order = [(5 * n + 1) % (N + 1) if (N + 1) % 5 else n for n in range(N)]
    out = last_slots(lens, order)
    check(x, run(x, order, out), order, out)
    check(x, run(x, None, None), list(range(N)), last_slots(lens, range(N)))


def test_every_window_kept():
    lens = [5, 1, 0, 140, 2]
    T = sum(lens)
    x = make(lens, 72, 4, T + 5, "fp16", bias=False, seed=8)
    slot_in, slot_out = [0, -1, 1, 2, 4], list(range(5, T + 5))
    check(x, run(x, slot_in, slot_out), slot_in, slot_out)


@pytest.mark.parametrize("W", [2, 4])
def test_many_ranges(W):
    """Enough tokens for ranges of many tokens, the cuts inside and at the ends of sequences."""
    lens = [3000, 1, 2, 4093, 0, 5000, 64, 3]
    x = make(lens, 512, W, 8, "bf16", seed=9)
    slot_in = [3, 1, -1, 0, 2, 4, -1, 7]
    out = last_slots(lens, [3, 1, 2, 0, 0, 4, 6, 7])
    check(x, run(x, slot_in, out), slot_in, out)


def test_many_sequences():
    """More sequences than one probe of the search covers."""
    rng = np.random.default_rng(3)
    lens = list(rng.integers(0, 4, 1500))
    x = make(lens, 16, 4, 1500, "bf16", seed=10)
    check(x, run(x, None, None), list(range(1500)), last_slots(lens, range(1500)))


def test_bad_tables_are_reported_and_stay_in_bounds():
    x = make([2, 2], 16, 4, 3, "bf16", seed=11)
    good = run(x, [0, 1], [-1, 0, -1, 1])
    for slot_in, slot_out, cu in (([3, 1], [-1, 0, -1, 1], [0, 2, 4]), ([0, 1], [-1, 9, -1, 1], [0, 2, 4]),
                                  ([-7, 1], [-1, 0, -1, 1], [0, 2, 4])):
        y, win, status = run(dict(x, cu=np.array(cu, np.int32)), slot_in, slot_out)
        assert status == 7
        assert torch.equal(y[2:], good[0][2:]) and torch.equal(win[1:], good[1][1:])
    for cu in ([0, 2, 5], [-3, 2, 4], [0, 3, 2]):
        _, win, status = run(dict(x, cu=np.array(cu, np.int32)), [0, 1], [-1, 0, -1, 1])
        assert status == 7
        assert torch.equal(win[2].cpu(), x["window"][2])


def test_single_tokens_are_the_sequence():
    """Token by token through the windows gives the bits of the packed training convolution."""
    import linear_attention_gdn_gb300 as gdn
    x = make([6, 6], 48, 4, 2, "bf16", seed=12)
    x["window"].zero_()
    want, win, _ = run(x, None, None)
    cu = x["cu"]
    y = torch.empty((12, 48), dtype=torch.bfloat16, device="cuda")
    gdn.gdn_conv1d_fwd(gdn.conv_problem(12, 2, 48, 4), x["x"].cuda(), x["w"].cuda(), x["b"].cuda(),
                       torch.from_numpy(cu).cuda(), cu, y)
    torch.cuda.synchronize()
    within("fwd", y, f64(want), 2.0 ** -7 * np.abs(f64(want)) + 1e-6)
    one = dict(x, window=x["window"].clone())
    for j in range(6):
        part = dict(one, x=x["x"][[j, 6 + j]], cu=np.array([0, 1, 2], np.int32))
        yj, w2, status = run(part, None, None)
        assert status == 0 and torch.equal(yj, want[[j, 6 + j]])
        one["window"] = w2.cpu()
    assert torch.equal(one["window"], win.cpu())


@pytest.mark.parametrize("N", [131, 701])
@pytest.mark.parametrize("W", [1, 3, 4])
def test_more_single_tokens_than_the_gpu_holds(N, W):
    """Single tokens of so many channels that a thread takes two sequences at a time, an odd number of them, and then goes
    on to further ones; slots of no order, some of none."""
    rng = np.random.default_rng(N + W)
    x = make([1] * N, 4096, W, N + 5, "bf16", seed=N)
    slot_in = rng.permutation(N + 5)[:N]
    slot_out = slot_in.copy()
    slot_in[::7] = -1
    slot_out[3::11] = -1
    check(x, run(x, list(slot_in), list(slot_out), cu=None), slot_in, slot_out)
    bad = slot_in.copy()
    bad[N - 1] = N + 5
    y, win, status = run(x, list(bad), list(slot_out), cu=None)
    good = run(x, list(slot_in), list(slot_out), cu=None)
    assert status == 7 and torch.equal(y[:N - 1], good[0][:N - 1])


@pytest.mark.parametrize("dtype,W,C", [("bf16", 4, 1032), ("fp16", 3, 520), ("fp32", 2, 64), ("fp32", 4, 520), ("bf16", 1, 8)])
def test_short_sequences_among_long_ones(dtype, W, C):
    """Few tokens on average: sequences around the length up to which they are taken apart from the long ones' ranges, long ones
    in a row, at the start, across several ranges and at the end; in place, from nowhere and to nowhere."""
    rng = np.random.default_rng(C + W)
    for lens in ([17, 16, 15, 0] + [1] * 60 + [300, 31, 0, 33] + [2, 4, 3, 1] * 10, [1] * 100 + [400], [18] + [0] * 3,
                 [1, 0, 40, 41, 0, 1] + [1] * 34):
        N = len(lens)
        x = make(lens, C, W, N + 4, dtype, seed=N)
        order = rng.permutation(N + 4)[:N]
        out = last_slots(lens, order)
        check(x, run(x, list(order), out, pad=8), order, out)
        slot_in = order.copy()
        slot_in[::5] = -1
        out[::3] = -1
        check(x, run(x, list(slot_in), list(out)), slot_in, out)


def test_every_window_of_short_and_long_sequences_kept():
    lens = [4, 1, 0, 16, 17, 2, 50, 3] + [2] * 12 + [0] * 8
    T = sum(lens)
    x = make(lens, 136, 4, T + 5, "bf16", seed=21)
    slot_in = [n % 5 if n % 4 else -1 for n in range(len(lens))]
    slot_out = [5 + (7 * t + 3) % T for t in range(T)]   # (T = 117: every slot once)
    check(x, run(x, slot_in, slot_out), slot_in, slot_out)


def test_bad_tables_among_short_and_long_sequences():
    """What is wrong is reported and skipped, the other sequences are served; nothing outside the tables is touched."""
    lens = [1] * 10 + [40] + [2] * 10
    T, N = sum(lens), len(lens)
    x = make(lens, 24, 4, N + 1, "bf16", seed=22)
    out = last_slots(lens, range(N))
    good = run(x, list(range(N)), out)
    rows = np.repeat(np.arange(N), lens)
    for n, slot in ((10, N + 1), (10, -4), (3, N + 9), (15, -2)):
        slot_in = list(range(N))
        slot_in[n] = slot
        y, win, status = run(x, slot_in, out)
        keep = torch.from_numpy(rows != n)
        assert status == 7 and torch.equal(y.cpu()[keep], good[0].cpu()[keep])
        assert torch.equal(win[n].cpu(), x["window"][n])
    for n in (10, 3):
        bad = out.copy()
        bad[np.cumsum(lens)[n] - 1] = N + 1
        y, win, status = run(x, list(range(N)), list(bad))
        assert status == 7 and torch.equal(y, good[0]) and torch.equal(win[n].cpu(), x["window"][n])
    for i, v in ((N, T + 3), (0, -2), (11, 5), (10, 60), (11, T + 40)):
        cu = x["cu"].copy()
        cu[i] = v
        _, win, status = run(dict(x, cu=cu), list(range(N)), out)
        assert status == 7 and torch.equal(win[N].cpu(), x["window"][N])


def test_more_sequences_than_rows_of_the_grid():
    rng = np.random.default_rng(5)
    lens = list(rng.integers(0, 3, 33000))
    x = make(lens, 8, 4, 33000, "bf16", seed=23)
    check(x, run(x, None, None), list(range(33000)), last_slots(lens, range(33000)))
