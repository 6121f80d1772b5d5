"""Linear attention with a fixed decay per head on the GPU: forward, backward and states against the FP64 oracle."""
import numpy as np
import pytest
import torch

import linear_attention_gdn_gb300 as gdn
from tests.la_testutil import SCALE, expect, f64, make, on_gpu
from tests.step_testutil import within

pytestmark = pytest.mark.gpu


def problem(x, d, segment=0):
    return gdn.la_problem(len(x["q"]), len(x["cu"]) - 1, x["q"].shape[1], x["v"].shape[1], SCALE, segment,
                          tuple(d[m].stride(0) for m in "qkv"))


def run(x, d, segment=0, states=True, poison=float("nan"), stream=None):
    """Every output, from buffers filled with poison."""
    prob = problem(x, d, segment)
    fill = lambda t: torch.full(t.shape, poison, dtype=t.dtype, device="cuda")  # noqa: E731
    f, b = gdn.gdn_la_workspace_bytes(prob, x["cu"])
    ws = torch.full((max(f, b, 16),), 255, dtype=torch.uint8, device="cuda")   # (all NaN)
    r = dict(o=fill(d["dO"]), s_out=None, ds_in=None)
    if states:
        N, HV = len(x["cu"]) - 1, x["v"].shape[1]
        r["s_out"], r["ds_in"] = (torch.full((N, HV, 128, 128), poison, device="cuda") for _ in range(2))
    for m in "qkv":   # laid out as q, k, v, poison between the rows, too
        flat = torch.full((d[m].shape[0] * d[m].stride(0) + 1,), poison, dtype=d[m].dtype, device="cuda")
        r["d" + m] = flat.as_strided(d[m].shape, d[m].stride())
    gdn.gdn_la_fwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], d["s_in"], r["o"], r["s_out"], d["err"],
                   ws, f, stream=stream)
    ws.fill_(255)
    gdn.gdn_la_bwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], d["s_in"], d["dO"], d["ds_out"], r["dq"],
                   r["dk"], r["dv"], r["ds_in"], d["err"], ws, b, stream=stream)
    assert gdn.gdn_device_status(d["err"]) == 0
    return r


def check(x, r):
    want = expect(x, x["q"].shape[1], x["v"].shape[1])
    for name, t in r.items():
        if t is not None:
            within(name, t, *want[name])


CASES = [
    ([1], 1, 1), ([2, 0, 1], 1, 2), ([0, 5], 2, 2), ([128], 1, 1), ([127, 129], 1, 3), ([256, 1], 2, 2), ([64, 200, 0, 33], 2, 6),
    ([300], 1, 4), ([513, 140], 1, 1), ([1409], 1, 2),
    ([200, 70], 1, 8), ([150], 1, 11), ([300, 5], 1, 16), ([140], 2, 14),
]


@pytest.mark.parametrize("lengths,H,HV", CASES)
def test_documents(lengths, H, HV):
    x = make(lengths, H, HV, seed=sum(lengths))
    d = on_gpu(x)
    check(x, run(x, d))


@pytest.mark.parametrize("segment", [1, 2, 3])
@pytest.mark.parametrize("lengths,H,HV", [([700], 1, 2), ([300, 0, 129, 1], 1, 1), ([128, 513], 2, 2), ([1290], 1, 1)])
def test_segments(lengths, H, HV, segment):
    x = make(lengths, H, HV, seed=segment)
    d = on_gpu(x)
    check(x, run(x, d, segment))


@pytest.mark.parametrize("segment", [0, 1, 5])
@pytest.mark.parametrize("lengths", [[200, 300], [1500, 1]])
def test_without_states(segment, lengths):
    x = make(lengths, 1, 2, states=False)
    d = on_gpu(x)
    check(x, run(x, d, segment, states=False))


@pytest.mark.parametrize("decay", [0.0, -1e-6, -0.3, -0.69, -0.71, -2.0, -30.0, -1e9, float("-inf")])
@pytest.mark.parametrize("segment", [0, 1])
def test_decays(decay, segment):
    x = make([290], 1, 1, seed=7, decay=decay)
    d = on_gpu(x)
    check(x, run(x, d, segment))


@pytest.mark.parametrize("decay", [-0.001, -0.69, -2.0])
@pytest.mark.parametrize("size", [1e-6, 3e4])
def test_sizes_of_values(size, decay):
    """Small and large values: the tolerances are relative to what is added up."""
    x = make([200], 1, 2, seed=13, decay=decay)
    for m in ("q", "k", "v", "dO"):
        x[m] = (x[m].float() * size).bfloat16()
    for m in ("s_in", "ds_out"):
        x[m] = x[m] * size * size
    check(x, run(x, on_gpu(x)))


@pytest.mark.parametrize("scale", [0.0, -0.5, 4.0])
def test_scales(scale):
    x = make([200], 1, 2, seed=14)
    d = on_gpu(x)
    one = run(x, d)
    prob = gdn.la_problem(200, 1, 1, 2, scale)
    o, dv = torch.empty_like(one["o"]), torch.empty_like(one["dv"])
    dq, dk = torch.empty_like(one["dq"]), torch.empty_like(one["dk"])
    ws = torch.empty(max(16, *gdn.gdn_la_workspace_bytes(prob, x["cu"])), dtype=torch.uint8, device="cuda")
    gdn.gdn_la_fwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], d["s_in"], o, None, d["err"], ws)
    gdn.gdn_la_bwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], d["s_in"], d["dO"], None, dq, dk, dv, None, d["err"], ws)
    zero = torch.zeros_like(d["s_in"])
    y = dict(x, ds_out=zero.cpu())
    r = run(y, on_gpu(y))
    for got, want in ((o, one["o"]), (dq, r["dq"]), (dk, r["dk"]), (dv, r["dv"])):
        w = f64(want) * (scale / SCALE)
        # the same sums, rounded at other places: three roundings of each part, as in `expect`, on either side
        assert np.abs(f64(got) - w).max() <= 6 * 2.0 ** -8 * np.abs(w).max() + 1e-30


@pytest.mark.parametrize("pad", [8, 128])
def test_strided_rows(pad):
    """Views of wider rows, in and out: what lies between is neither read nor written."""
    x = make([140, 7], 2, 4, seed=pad)
    d = on_gpu(x, pad)
    r = run(x, d)
    check(x, r)
    for m in "qkv":
        t = r["d" + m]
        rest = t.as_strided((t.shape[0] - 1, pad), (t.stride(0), 1), t.shape[1] * 128)   # (the last row has none behind it)
        assert rest.isnan().all()


def test_views_of_one_packed_row():
    H, HV, T = 1, 2, 150
    x = make([T], H, HV, seed=3)
    d = on_gpu(x)
    rows = torch.cat([d["q"], d["k"], d["v"]], 1)
    d["q"], d["k"], d["v"] = rows[:, :H], rows[:, H:2 * H], rows[:, 2 * H:]
    check(x, run(x, d))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("segment", [0, 1])
def test_other_documents_values_take_no_part(bad, segment):
    """A document of infinite or NaN values changes no bit of those before and behind it, in its chunks' rows or not."""
    lengths = [130, 70, 131]
    x = make(lengths, 1, 2, seed=11)
    clean = run(x, on_gpu(x), segment)
    y = {m: t.clone() if torch.is_tensor(t) else t for m, t in x.items()}
    for m in ("q", "k", "v", "dO"):
        y[m][130:200] = bad
    y["s_in"][1] = bad
    got = run(y, on_gpu(y), segment)
    for m, t in got.items():
        if m in ("s_out", "ds_in"):
            assert torch.equal(t[[0, 2]], clean[m][[0, 2]])
        else:
            assert torch.equal(t[:130], clean[m][:130]) and torch.equal(t[200:], clean[m][200:])


@pytest.mark.parametrize("segment", [0, 2])
def test_same_bits_again_and_in_place(segment):
    x = make([400, 3], 1, 3, seed=2)
    d = on_gpu(x)
    first, second = run(x, d, segment), run(x, d, segment)
    for m in first:
        assert torch.equal(first[m], second[m])
    prob = problem(x, d, segment)
    f, b = gdn.gdn_la_workspace_bytes(prob, x["cu"])
    ws = torch.empty(max(f, b, 16), dtype=torch.uint8, device="cuda")
    states, grads = d["s_in"].clone(), d["ds_out"].clone()
    o = torch.empty_like(first["o"])
    gdn.gdn_la_fwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], states, o, states, d["err"], ws)
    assert torch.equal(states, first["s_out"]) and torch.equal(o, first["o"])
    gdn.gdn_la_bwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], d["s_in"], d["dO"], grads, first["dq"],
                   first["dk"], first["dv"], grads, d["err"], ws)
    assert torch.equal(grads, first["ds_in"])


@pytest.mark.parametrize("HV", [1, 3])
@pytest.mark.parametrize("segment", [0, 1])
def test_state_gradients_in_place_leave_the_others(segment, HV):
    """ds_in over ds_out: dk, which needs ds_out too, has what it has with buffers of their own."""
    x = make([200, 0, 140], 1, HV, seed=3)
    d = on_gpu(x)
    want = run(x, d, segment)
    prob = problem(x, d, segment)
    ws = torch.empty(max(16, gdn.gdn_la_workspace_bytes(prob, x["cu"])[1]), dtype=torch.uint8, device="cuda")
    grads, got = d["ds_out"].clone(), {m: torch.full_like(want[m], float("nan")) for m in ("dq", "dk", "dv")}
    gdn.gdn_la_bwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], d["s_in"], d["dO"], grads, got["dq"],
                   got["dk"], got["dv"], grads, d["err"], ws)
    assert gdn.gdn_device_status(d["err"]) == 0 and torch.equal(grads, want["ds_in"])
    for m in got:
        assert torch.equal(got[m], want[m]), m


def test_no_tokens():
    x = make([0, 0], 1, 2)
    d = on_gpu(x)
    r = run(x, d)
    assert torch.equal(r["s_out"], d["s_in"]) and torch.equal(r["ds_in"], d["ds_out"])


def test_a_wrong_device_copy_is_reported():
    x = make([100, 60], 1, 1)
    d = on_gpu(x)
    for wrong in ([0, 100, 159], [0, 161, 160], [1, 100, 160], [0, -5, 160], [0, 100, 2 ** 30]):
        prob = problem(x, d)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.empty_like(d["dO"])
        gdn.gdn_la_fwd(prob, d["q"], d["k"], d["v"], d["decay"], torch.tensor(wrong, dtype=torch.int32, device="cuda"), x["cu"],
                       None, o, None, err, None)
        assert gdn.gdn_device_status(err) == 1


def test_other_stream_and_graph():
    x = make([260, 50], 1, 2, seed=4)
    d = on_gpu(x)
    want = run(x, d, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(x, d, 1, stream=s)
    s.synchronize()
    for m in want:
        assert torch.equal(want[m], got[m])
    prob = problem(x, d, 1)
    f, _ = gdn.gdn_la_workspace_bytes(prob, x["cu"])
    ws = torch.empty(f, dtype=torch.uint8, device="cuda")
    o, s_out = torch.empty_like(want["o"]), torch.empty_like(want["s_out"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_la_fwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], d["s_in"], o, s_out, d["err"], ws)
    for _ in range(2):
        o.fill_(float("nan"))
        s_out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want["o"]) and torch.equal(s_out, want["s_out"])


def test_gradients_are_differences():
    """The forward is linear in v, so a forward of a step in v is an exact difference: its product with dO is dv's with
    the step.  Both sides are sums of values whose roundings are independent, each at most its tolerance off: within six
    times the root of the sum of their squares."""
    x = make([150], 1, 2, states=False, seed=9)
    y = dict(x, v=torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(1)).bfloat16())
    r, moved = run(x, on_gpu(x), states=False), run(y, on_gpu(y), states=False)
    dO, step = f64(x["dO"]), f64(y["v"])
    left, right = (f64(moved["o"]) * dO).sum(), (f64(r["dv"]) * step).sum()
    off = ((expect(y, 1, 2)["o"][1] * dO) ** 2).sum() + ((expect(x, 1, 2)["dv"][1] * step) ** 2).sum()
    assert abs(left - right) <= 6 * np.sqrt(off)


@pytest.mark.parametrize("lengths,H,HV", [([1], 1, 1), ([3, 0, 1], 1, 1), ([1, 1, 2, 5], 2, 6), ([17, 64], 1, 2), ([33, 128 + 7], 1, 1)])
def test_short_chunks_are_rounded_once(lengths, H, HV):
    """Chunks of up to 64 tokens give the pairs' factors in two BF16 terms, so without a state before them only the result
    is rounded.  With x the result before its rounding and w the exact one, |bf(x) - x| <= |bf(w) - x|, so
    |bf(x) - w| <= |bf(w) - w| + 2 |x - w|; |x - w| <= 2^-16 of the sums of absolute values A: the terms' 2^-17, and 2^-17 for
    the FP32 sums and products (under 64 operations, each 2^-23 or 2^-24)."""
    x = make(lengths, H, HV, states=False, seed=5)
    d = on_gpu(x)
    r = run(x, d, states=False)
    want, G, outside = expect(x, H, HV), HV // H, 0
    bf = lambda t: torch.from_numpy(t).to(torch.bfloat16).double().numpy()  # noqa: E731
    for m in ("o", "dq", "dk", "dv"):
        got, w = f64(r[m].cpu()), want[m][0]
        once = np.zeros(w.shape)   # with the factors rounded
        for i, n in enumerate(lengths):
            a, b = int(x["cu"][i]), int(x["cu"][i + 1])
            if not 0 < n <= 64:
                continue
            A = np.zeros((n,) + w.shape[1:])
            for h in range(HV):
                Q, K, V, DO = (f64(x[c])[a:b, h // G if c in "qk" else h] for c in ("q", "k", "v", "dO"))
                g = float(x["decay"][h])
                t = np.arange(n)
                decay = np.where(t[:, None] >= t, SCALE * np.exp(g * np.maximum(t[:, None] - t, 0)), 0.0)
                if m == "o":
                    X, Y, Z, D = Q, K, V, decay
                elif m == "dv":
                    X, Y, Z, D = K, Q, DO, decay.T
                elif m == "dq":
                    X, Y, Z, D = DO, V, K, decay
                else:
                    X, Y, Z, D = V, DO, Q, decay.T
                j = h if m in ("o", "dv") else h // G
                A[:, j] += (D * (np.abs(X) @ np.abs(Y).T)) @ np.abs(Z)
                once[a:b, j] += bf(D * (X @ Y.T)) @ Z
            near = np.abs(bf(w[a:b]) - w[a:b]) + 2.0 ** -15 * A
            assert (np.abs(got[a:b] - w[a:b]) <= near).all()
            outside += int((np.abs(bf(once[a:b]) - w[a:b]) > near).sum())
    assert outside   # factors of one term would not do


@pytest.mark.parametrize("N,H,HV,most", [(40, 1, 8, 140), (21, 1, 16, 300), (3, 2, 128, 150)])
def test_groups_of_more_heads_than_run_side_by_side(N, H, HV, most):
    """320 to 384 CTAs whose heads add up in order, on fewer SMs, by falling length or, past 32 documents, in their order."""
    lengths = np.random.RandomState(N).randint(0, most, N).tolist()
    x = make(lengths, H, HV, states=False, seed=N)
    d = on_gpu(x)
    first = run(x, d, states=False)
    check(x, first)
    again = run(x, d, states=False)
    for m in ("dq", "dk", "dv"):
        assert torch.equal(first[m], again[m])


def test_two_backward_passes_at_once():
    """On two streams, each with its workspace, and then both captured in graphs with one workspace that run in turn."""
    xs = [make([200, 90, 0, 300], 1, 6, seed=s) for s in (31, 32)]
    ds = [on_gpu(x) for x in xs]
    want = [run(x, d) for x, d in zip(xs, ds)]
    streams = [torch.cuda.Stream() for _ in xs]
    probs = [problem(x, d) for x, d in zip(xs, ds)]
    b = gdn.gdn_la_workspace_bytes(probs[0], xs[0]["cu"])[1]
    ws = [torch.empty(b, dtype=torch.uint8, device="cuda") for _ in xs]
    got = [{m: torch.empty_like(w[m]) for m in ("dq", "dk", "dv", "ds_in")} for w in want]

    def call(i, w, stream=None):
        d, g = ds[i], got[i]
        gdn.gdn_la_bwd(probs[i], d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], xs[i]["cu"], d["s_in"], d["dO"], d["ds_out"],
                       g["dq"], g["dk"], g["dv"], g["ds_in"], d["err"], w, b, stream=stream)

    def same():
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for m in g:
                assert torch.equal(g[m], w[m])
                g[m].fill_(float("nan"))
        assert all(gdn.gdn_device_status(d["err"]) == 0 for d in ds)

    torch.cuda.synchronize()
    for _ in range(10):
        for i in (0, 1):
            call(i, ws[i], streams[i])
    same()
    graphs = [torch.cuda.CUDAGraph() for _ in xs]
    for i in (0, 1):
        with torch.cuda.graph(graphs[i]):
            call(i, ws[0])
    for _ in range(3):
        for g in graphs:
            g.replay()
    same()


def test_a_wrong_device_copy_is_reported_by_the_backward():
    x = make([100, 60], 1, 3)
    d = on_gpu(x)
    prob = problem(x, d)
    ws = torch.empty(gdn.gdn_la_workspace_bytes(prob, x["cu"])[1], dtype=torch.uint8, device="cuda")
    for wrong in ([0, 100, 159], [0, 161, 160], [1, 100, 160], [0, -5, 160], [0, 100, 2 ** 30]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = [torch.empty_like(d[m]) for m in "qkv"]
        gdn.gdn_la_bwd(prob, d["q"], d["k"], d["v"], d["decay"], torch.tensor(wrong, dtype=torch.int32, device="cuda"), x["cu"],
                       None, d["dO"], None, *out, None, err, ws)
        assert gdn.gdn_device_status(err) == 1
    check(x, run(x, d))   # and nothing is left behind


@pytest.mark.parametrize("in_place", [False, True])
def test_all_gradients_are_there_when_the_call_has_ended(in_place):
    """The walks run side by side, but what comes behind them, on this stream or one that waits for it, sees all three; also
    from a graph, which writes the states' gradients in place if so wished."""
    x = make([900, 3, 140, 2], 1, 5, seed=41)
    d = on_gpu(x)
    want = run(x, d)
    prob = problem(x, d)
    ws = torch.empty(gdn.gdn_la_workspace_bytes(prob, x["cu"])[1], dtype=torch.uint8, device="cuda")
    out = {m: torch.empty_like(want[m]) for m in ("dq", "dk", "dv", "ds_in")}
    incoming = out["ds_in"] if in_place else d["ds_out"]
    side = torch.cuda.Stream()

    def call():
        gdn.gdn_la_bwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], d["s_in"], d["dO"], incoming, out["dq"],
                       out["dk"], out["dv"], out["ds_in"], d["err"], ws)

    graph = torch.cuda.CUDAGraph()
    out["ds_in"].copy_(d["ds_out"])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for go in (call, graph.replay) * 4:
        for m in ("dq", "dk", "dv", "ds_in"):
            out[m].fill_(float("nan"))
        out["ds_in"].copy_(d["ds_out"])
        go()
        here = {m: t.clone() for m, t in out.items()}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            there = {m: t.clone() for m, t in out.items()}
        torch.cuda.current_stream().wait_stream(side)
        for m in out:
            assert torch.equal(here[m], want[m]) and torch.equal(there[m], want[m]), m
    assert gdn.gdn_device_status(d["err"]) == 0
