"""The linear attention where the device's cu_seqlens are in order and end where the host's do, but cut the tokens otherwise:
nothing outside the outputs and the workspace is written, and nothing is left behind for the next call; and what the workspace
held before a call is of no account."""
import numpy as np
import pytest
import torch

import linear_attention_gdn_gb300 as gdn
from tests.la_testutil import SCALE, make, on_gpu
from tests.test_gpu_la import check, run

pytestmark = pytest.mark.gpu
GUARD = 8 * 65536   # bytes: more than the segments that the tables below have too many, of four heads


def guarded(size):
    """size bytes (a multiple of 16) with a guard on either side, and what tells whether the guards are whole."""
    flat = torch.full((size + 2 * GUARD,), 0x5a, dtype=torch.uint8, device="cuda")
    return flat[GUARD:GUARD + size], lambda: bool((flat[:GUARD] == 0x5a).all()) and bool((flat[GUARD + size:] == 0x5a).all())


def wrong_call(lengths, wrong, H, HV, segment, states):
    """Forward and backward with another table on the device; all outputs and the workspace between guards.  Returns the
    error words of both."""
    x = make(lengths, H, HV, states=states, seed=1)
    d = on_gpu(x)
    T, N = len(x["q"]), len(lengths)
    prob = gdn.la_problem(T, N, H, HV, SCALE, segment)
    f, b = gdn.gdn_la_workspace_bytes(prob, x["cu"])
    cu = torch.tensor(wrong, dtype=torch.int32, device="cuda")
    sizes = dict(o=T * HV * 256, dq=T * H * 256, dk=T * H * 256, dv=T * HV * 256, fwd=f, bwd=b)
    if states:
        sizes.update(s_out=N * HV * 65536, ds_in=N * HV * 65536)
    out = {m: guarded(n) for m, n in sizes.items()}
    at = {m: t.data_ptr() for m, (t, _) in out.items()}
    errs = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    gdn.gdn_la_fwd(prob, d["q"], d["k"], d["v"], d["decay"], cu, x["cu"], d["s_in"], at["o"], at.get("s_out"), errs[0], at["fwd"], f)
    gdn.gdn_la_bwd(prob, d["q"], d["k"], d["v"], d["decay"], cu, x["cu"], d["s_in"], d["dO"], d["ds_out"], at["dq"], at["dk"], at["dv"],
                   at.get("ds_in"), errs[1], at["bwd"], b)
    codes = [gdn.gdn_device_status(e) for e in errs]
    for m, (_, whole) in out.items():
        assert whole(), m
    return codes


# host's lengths, the device's bounds, chunks of a segment: the device has more segments than the host (places by length, and past
# 32 documents in order), or fewer
CUT = [([1000, 1000], [0, 0, 2000], 3), ([1024, 512, 512], [0, 128, 1280, 2048], 4), ([256, 256], [0, 129, 512], 1),
       ([128] * 40, [0] + [128 * i - 100 for i in range(1, 40)] + [5120], 1), ([300] + [2] * 39, [0] + [4 * i for i in range(1, 40)] + [378], 1),
       ([2, 1300, 2], [0, 600, 700, 1304], 2)]


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("H,HV", [(2, 2), (1, 4)])
@pytest.mark.parametrize("lengths,wrong,segment", CUT)
def test_segments_past_the_workspace_are_left_out(lengths, wrong, segment, H, HV, states):
    assert wrong_call(lengths, wrong, H, HV, segment, states) == [1, 1]


@pytest.mark.parametrize("H,HV", [(2, 2), (1, 4)])
@pytest.mark.parametrize("lengths,wrong", [([200, 300], [0, 20, 500]), ([200, 300], [0, 480, 500]),
                                           ([128, 256, 1], [0, 383, 384, 385])])
def test_documents_longer_than_the_hosts_longest_are_left_out(lengths, wrong, H, HV):
    """Uncut, a document has one segment: those that would have more are not begun again from s_in."""
    assert wrong_call(lengths, wrong, H, HV, 0, True) == [1, 1]
    x = make(lengths, H, HV, seed=2)
    d = on_gpu(x)
    prob = gdn.la_problem(len(x["q"]), len(lengths), H, HV, SCALE)
    o, s_out = torch.full_like(d["dO"], float("nan")), torch.full_like(d["s_in"], float("nan"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_la_fwd(prob, d["q"], d["k"], d["v"], d["decay"], torch.tensor(wrong, dtype=torch.int32, device="cuda"), x["cu"], d["s_in"], o,
                   s_out, err, None)
    longest = int(np.argmax(np.diff(wrong)))
    assert gdn.gdn_device_status(err) == 1
    assert o[wrong[longest]:wrong[longest + 1]].isnan().all() and s_out[longest].isnan().all()


@pytest.mark.parametrize("H,HV", [(2, 2), (1, 4)])
@pytest.mark.parametrize("lengths,wrong,segment", [
    ([100, 60], [0, 60, 160], 0), ([100, 60], [0, 99, 160], 0), ([1, 1, 1], [0, 2, 2, 3], 0), ([100, 0, 60], [0, 100, 101, 160], 0),
    ([60, 100], [0, 100, 160], 0), ([500, 500], [0, 490, 1000], 2), ([3] * 50, [0] + [3 * i - (i == 49) for i in range(1, 50)] + [150], 0),
    ([3] * 40, [0] + [3 * i + (i == 1) - (i == 2) for i in range(1, 40)] + [120], 1)])
def test_other_bounds_of_as_many_segments_are_reported(lengths, wrong, segment, H, HV):
    assert wrong_call(lengths, wrong, H, HV, segment, True) == [1, 1]
    assert wrong_call(lengths, [0] + np.cumsum(lengths).tolist(), H, HV, segment, True) == [0, 0]


@pytest.mark.parametrize("H,HV", [(2, 2), (1, 4)])
def test_nothing_is_left_behind(H, HV):
    wrong_call([1000, 1000], [0, 0, 2000], H, HV, 3, True)
    x = make([300, 140], H, HV, seed=3)
    check(x, run(x, on_gpu(x), 1))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("segment", [0, 1])
def test_the_workspace_may_hold_anything(segment, in_place):
    """Counts of heads and tickets are cleared ahead of all walks of a call: a call, a captured one and its replays behind one
    another give the same bits, whatever the workspace held before each."""
    x = make([130, 0, 500, 60], 2, 10, seed=8)
    d = on_gpu(x)
    want = run(x, d, segment)
    prob = gdn.la_problem(len(x["q"]), 4, 2, 10, SCALE, segment)
    ws = torch.empty(gdn.gdn_la_workspace_bytes(prob, x["cu"])[1], dtype=torch.uint8, device="cuda")
    out = {m: torch.empty_like(want[m]) for m in ("dq", "dk", "dv", "ds_in")}
    incoming = out["ds_in"] if in_place else d["ds_out"]

    def call():
        gdn.gdn_la_bwd(prob, d["q"], d["k"], d["v"], d["decay"], d["cu_dev"], x["cu"], d["s_in"], d["dO"], incoming, out["dq"], out["dk"],
                       out["dv"], out["ds_in"], d["err"], ws)

    graph = torch.cuda.CUDAGraph()
    out["ds_in"].copy_(d["ds_out"])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for go, held in ((call, 0), (graph.replay, 0), (graph.replay, 1), (call, 3), (call, 127), (graph.replay, 255), (graph.replay, 128)):
        for m in ("dq", "dk", "dv"):
            out[m].fill_(float("nan"))
        out["ds_in"].copy_(d["ds_out"])
        ws.fill_(held)
        go()
        for m in out:
            assert torch.equal(out[m], want[m]), (m, held)
    assert gdn.gdn_device_status(d["err"]) == 0
