"""GPU parity of the recurrent form (gdn_step, gdn_kda_step) against the FP64 oracle, through the C ABI.

Tolerances: a state's column after n tokens differs from the exact one by at most n steps' FP32 errors. A step sums 128
products and applies a few more operations, each rounded by 2^-24, on values no larger than the column's norm
and v; the norms' and exponential's few last places are in the 140. o is then rounded once to its type."""
import numpy as np
import pytest
import torch

from oracle import step as oracle
from tests.step_testutil import TINY, TYPES, U, f64, strided, within

pytestmark = pytest.mark.gpu


def make(lens, H, HV, slots, dtype, kda, seed=0, steep=False):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    T, dt = int(sum(lens)), TYPES[dtype][0]
    shape = (T, HV, 128) if kda else (T, HV)
    g = torch.nn.functional.logsigmoid((-8.0 if steep else 2.0) + 4.0 * torch.rand(shape, generator=gen))
    return dict(q=rnd(T, H, 128).to(dt), k=rnd(T, H, 128).to(dt), v=rnd(T, HV, 128).to(dt), g=g,
                beta=torch.sigmoid(rnd(T, HV)), states=0.5 * rnd(slots, HV, 128, 128),
                cu=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))


def run(x, kda, slot_in, slot_out, l2norm=True, scale=128 ** -0.5, packed=False, stream=None, cu="dev"):
    """(o, pool, error word) of the library; slot tables None: NULL."""
    import linear_attention_gdn_gb300 as gdn
    T, H, HV, slots = x["q"].shape[0], x["q"].shape[1], x["v"].shape[1], x["states"].shape[0]
    d = {n: x[n].cuda() for n in ("q", "k", "v", "g", "beta", "states")}
    strides = (0, 0, 0)
    if packed:   # one row of q, k, v per token, and 8 more values
        row = torch.full((T, (2 * H + HV) * 128 + 8), float("nan"), dtype=x["q"].dtype, device="cuda")
        views = {}
        for n, a, b in (("q", 0, H), ("k", H, 2 * H), ("v", 2 * H, 2 * H + HV)):
            views[n] = row[:, a * 128:b * 128].unflatten(1, (b - a, 128))
            views[n].copy_(x[n])
        d.update(views)
        strides = (row.stride(0),) * 3
    N = len(x["cu"]) - 1
    prob = gdn.step_problem(T, N, H, HV, slots, scale=scale, l2norm=l2norm, dtype=x["q"].dtype, strides=strides)
    o = torch.full((T, HV, 128), float("nan"), dtype=x["q"].dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = lambda a: None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cu_dev = torch.from_numpy(x["cu"]).cuda() if cu == "dev" else cu
    (gdn.gdn_kda_step if kda else gdn.gdn_step)(prob, d["q"], d["k"], d["v"], d["g"], d["beta"], d["states"], o, err,
                                                cu_seqlens_dev=cu_dev, slot_in=table(slot_in),
                                                slot_out=table(slot_out), stream=stream)
    return o, d["states"], gdn.gdn_device_status(err, stream)


def check(x, got, slot_in, slot_out, l2norm=True, scale=128 ** -0.5):
    o, pool, status = got
    assert status == 0
    want_o, want = oracle.step(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta", "states")), x["cu"], slot_in, slot_out,
                               l2norm=l2norm, scale=scale)
    n = max(1, int(np.diff(x["cu"]).max()))
    kn = 1.0 if l2norm else np.linalg.norm(f64(x["k"]), axis=-1).max() if len(o) else 1.0
    qn = 1.0 if l2norm else np.linalg.norm(f64(x["q"]), axis=-1).max() if len(o) else 1.0
    size = np.sqrt((want ** 2).sum(-2)).max() + np.sqrt((f64(x["states"]) ** 2).sum(-2)).max()
    size = size * max(1.0, kn * kn) + kn * (np.abs(f64(x["v"])).max() if len(o) else 0.0)
    within("states", pool, want, n * 140 * U * size)
    within("o", o, want_o, TYPES[str_type(x)][1] * np.abs(want_o) + TINY + scale * qn * n * 140 * U * size)
    # nothing but the written slots changes, bit for bit
    same = [s for s in range(pool.shape[0]) if s not in set(int(i) for i in slot_out)]
    assert torch.equal(pool.cpu()[same], x["states"][same])


def str_type(x):
    return next(n for n, (t, _) in TYPES.items() if t == x["q"].dtype)


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("H,HV", [(1, 1), (2, 6), (3, 3)])
def test_single_tokens(H, HV, dtype, kda):
    """A batch of single tokens in slots of no order, one from no state, one kept nowhere; packed rows."""
    N, slots = 5, 9
    x = make([1] * N, H, HV, slots, dtype, kda, seed=H * 10 + HV)
    slot_in, slot_out = [7, 2, -1, 0, 5], [7, 2, 8, -1, 5]
    check(x, run(x, kda, slot_in, slot_out), slot_in, slot_out)
    check(x, run(x, kda, slot_in, slot_out, packed=True, cu=None), slot_in, slot_out)


@pytest.mark.parametrize("kda", [False, True])
def test_ragged_lengths_with_every_state_kept(kda):
    lens = [3, 0, 1, 70, 0, 2, 8]
    T = sum(lens)
    x = make(lens, 2, 4, T + 4, "bf16", kda, seed=3)
    slot_in = [1, 0, -1, 3, 2, -1, 0]
    slot_out = list(range(4, T + 4))
    check(x, run(x, kda, slot_in, slot_out), slot_in, slot_out)


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("lens", [[12], [13, 14], [33, 0, 7], [64, 100], [1, 0, 300]])
def test_long_sequences(lens, dtype, kda):
    """Lengths at which several tokens are taken at a time, with ends at every place of such a block, and states
    wanted in the middle and nowhere."""
    T = sum(lens)
    x = make(lens, 1, 3, 12, dtype, kda, seed=T)
    slot_in = [2, -1, 0][:len(lens)]
    slot_out = np.full(T, -1)
    ends = np.cumsum(lens)
    slot_out[ends[0] - 1] = 2
    slot_out[[T // 2, T // 2 + 1, T - 2]] = [3, 4, 5]
    check(x, run(x, kda, slot_in, slot_out), slot_in, slot_out)


@pytest.mark.parametrize("kda", [False, True])
def test_long_sequences_with_steep_gates(kda):
    x = make([40], 1, 2, 2, "fp32", kda, seed=13, steep=True)
    x["g"][7] = -float("inf")
    slot_out = np.full(40, -1)
    slot_out[[8, 39]] = [0, 1]
    check(x, run(x, kda, [1], slot_out), [1], slot_out)


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("lens", [[257], [200, 61], [33, 0, 230], [1, 90, 170], [64, 64, 64, 65, 5]])
def test_enough_tokens_to_be_taken_in_blocks(lens, dtype, kda):
    """Sums of tokens and heads at which four tokens are taken at a time: ends at every place of a block and of a
    phase of blocks, unlike lengths, states wanted in the middle of a block, in a row, and nowhere."""
    T = sum(lens)
    x = make(lens, 16, 48, 14, dtype, kda, seed=T + len(lens))
    slot_in = [2, -1, 0, 7, 9][:len(lens)]
    slot_out = np.full(T, -1)
    ends = np.cumsum(lens)
    slot_out[ends[0] - 1], slot_out[-1] = 2, 6
    slot_out[[T // 2, T // 2 + 1, T - 2]] = [3, 4, 5]
    check(x, run(x, kda, slot_in, slot_out), slot_in, slot_out)


def test_blocks_with_steep_gates_in_place():
    x = make([140, 130], 2, 48, 2, "fp32", True, seed=14, steep=True)
    x["g"][7] = x["g"][141] = -float("inf")
    x["g"][20, :, ::2] = 0.0
    slot_out = np.full(270, -1)
    slot_out[[139, 269]] = [0, 1]
    check(x, run(x, True, None, None), [0, 1], slot_out)


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("lens", [[257], [200, 62], [130, 133]])
def test_blocks_end_with_their_last_token(lens, kda):
    """An infinite value at the last token of a block that is not full makes its state's column infinite, with k's
    signs: what the block lacks takes no part.  All else has the bits of a finite value's run."""
    T = sum(lens)
    x = make(lens, 16, 48, len(lens), "bf16", kda, seed=T)
    x["k"][T - 1][x["k"][T - 1] == 0] = 1.0
    good = run(x, kda, None, None)
    x["v"][T - 1, 5, 17] = float("inf")
    o, pool, status = run(x, kda, None, None)
    assert status == 0 and good[2] == 0
    column = pool[-1, 5, :, 17].cpu()
    assert torch.equal(column, torch.sign(x["k"][T - 1, 5 // 3].float()) * float("inf"))
    pool[-1, 5, :, 17] = good[1][-1, 5, :, 17]
    assert torch.equal(pool, good[1])
    assert not torch.isfinite(o[T - 1, 5, 17])
    o[T - 1, 5, 17] = good[0][T - 1, 5, 17]
    assert torch.equal(o, good[0])


def test_blocks_report_bad_tables():
    x = make([150, 150], 1, 48, 3, "bf16", False, seed=15)
    good = run(x, False, [0, 1], None)
    slot_out = np.full(300, -1)
    slot_out[[77, 149, 299]] = [9, 0, 1]
    o, pool, status = run(x, False, [0, 1], slot_out)
    # (a state that is wanted ends a block, so the first sequence's sums are taken in another order)
    assert status == 7 and torch.equal(o[150:], good[0][150:]) and torch.equal(pool[1], good[1][1])
    slot_out[77] = -1
    check(x, (o, pool, 0), [0, 1], slot_out)
    for slot_in, cu in (([3, 1], [0, 150, 300]), ([0, 1], [-1, 150, 300])):
        o, pool, status = run(dict(x, cu=np.array(cu, np.int32)), False, slot_in, None)
        assert status == 7 and torch.equal(o[150:], good[0][150:]) and torch.equal(pool[1], good[1][1])
    _, pool, status = run(dict(x, cu=np.array([0, 150, 301], np.int32)), False, [0, 1], None)
    assert status == 7 and torch.equal(pool[0], good[1][0]) and torch.equal(pool[1].cpu(), x["states"][1])


def test_default_slots_update_in_place():
    """Without tables sequence n lives in slot n, and is written back after its last token."""
    lens = [2, 0, 5, 1]
    x = make(lens, 1, 2, 5, "fp32", False, seed=4)
    last = np.cumsum(lens) - 1
    slot_out = np.full(sum(lens), -1)
    slot_out[[last[0], last[2], last[3]]] = [0, 2, 3]
    check(x, run(x, False, None, None), [0, 1, 2, 3], slot_out)
    # with slot_in alone: back to where it came from
    slot_in = [3, 1, -1, 0]
    slot_out[[last[0], last[2], last[3]]] = [3, -1, 0]
    check(x, run(x, False, slot_in, None), slot_in, slot_out)


@pytest.mark.parametrize("kda", [False, True])
def test_no_norm_and_steep_gates(kda):
    """q, k as given (scaled down so that the rule contracts), decays down to e^-8 a token, then to nothing."""
    x = make([6, 9], 2, 2, 3, "fp32", kda, seed=5, steep=True)
    x["q"] *= 0.08
    x["k"] *= 0.08
    x["g"][4] = -float("inf")   # forgets everything
    slot_in, slot_out = [0, 2], [-1] * 5 + [1] + [-1] * 8 + [2]
    check(x, run(x, kda, slot_in, slot_out, l2norm=False, scale=0.5), slot_in, slot_out, l2norm=False, scale=0.5)


def test_zero_rows():
    """Rows of zeros have norm zero: no division by it."""
    x = make([2, 2], 1, 2, 2, "bf16", False, seed=6)
    x["q"][1], x["k"][2] = 0, 0
    check(x, run(x, False, None, None), [0, 1], [-1, 0, -1, 1])


def test_own_slot_may_be_written_before_the_last_token():
    """A sequence reads its slot before it writes any: its own slots may repeat."""
    x = make([4], 1, 3, 2, "bf16", False, seed=7)
    check(x, run(x, False, [1], [1, 0, 1, 1]), [1], [1, 0, 1, 1])


def test_no_tokens():
    x = make([0, 0], 1, 1, 2, "bf16", False)
    _, pool, status = run(x, False, None, None)
    assert status == 0 and torch.equal(pool.cpu(), x["states"])


def test_single_tokens_are_the_sequence():
    """Token by token through the pool gives the bits of all tokens in one call, on another stream as well."""
    import linear_attention_gdn_gb300 as gdn
    x = make([7, 7], 2, 4, 2, "bf16", True, seed=8)
    want_o, want, _ = run(x, True, None, None)
    s = torch.cuda.Stream()
    pool, outs = x["states"].cuda(), []
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    prob = gdn.step_problem(2, 2, 2, 4, 2)
    parts = [{n: x[n][[j, 7 + j]].cuda() for n in ("q", "k", "v", "g", "beta")} for j in range(7)]
    torch.cuda.synchronize()
    for d in parts:
        o = torch.empty((2, 4, 128), dtype=torch.bfloat16, device="cuda")
        gdn.gdn_kda_step(prob, d["q"], d["k"], d["v"], d["g"], d["beta"], pool, o, err, stream=s)
        outs.append(o)
    assert gdn.gdn_device_status(err, s) == 0
    assert torch.equal(pool, want)
    assert torch.equal(torch.stack(outs).transpose(0, 1).reshape(14, 4, 128), want_o)


def test_prefill_writes_the_pool_and_the_step_goes_on():
    """gdn_fwd_states writes the pool's slots; tokens stepped from there are the longer prefill's, within the
    chunked form's budget."""
    import linear_attention_gdn_gb300 as gdn
    from tests.gdn_testutil import compare
    L, M, H, HV = 130, 5, 2, 4
    x = make([L + M], H, HV, 1, "bf16", False, seed=9)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "g", "beta")}
    pool = torch.full((1, HV, 128, 128), float("nan"), device="cuda")
    for n, s_out in ((L + M, None), (L, pool)):
        cu = np.array([0, n], np.int32)
        prob = gdn.problem(n, 1, H, HV)
        buf = gdn.Buffers(prob, cu)
        o = torch.empty((n, HV, 128), dtype=torch.bfloat16, device="cuda")
        gdn.gdn_fwd_states(prob, d["q"], d["k"], d["v"], d["g"], d["beta"], torch.from_numpy(cu).cuda(), cu, None, o,
                           s_out, None, buf.workspace)
        assert gdn.gdn_device_status(buf.workspace) == 0
        if s_out is None:
            whole = o
    y = torch.empty((M, HV, 128), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_step(gdn.step_problem(M, 1, H, HV, 1), *(d[n][L:] for n in ("q", "k", "v", "g", "beta")), pool, y, err,
                 cu_seqlens_dev=torch.tensor([0, M], dtype=torch.int32, device="cuda"))
    assert gdn.gdn_device_status(err) == 0
    compare("o", f64(y), f64(whole[L:]))


def test_offsets_past_32_bits():
    """Slots past 2^32 elements of the pool."""
    HV, slots = 48, 5600   # 4.4e9 values
    x = make([1, 1], 16, HV, 2, "bf16", False, seed=10)
    big = torch.empty((slots, HV, 128, 128), device="cuda")
    slot_in, slot_out = [slots - 1, 5470], [slots - 2, 5470]
    big[slot_in[0]], big[slot_in[1]] = x["states"][0].cuda(), x["states"][1].cuda()
    y = dict(x, states=big)
    import linear_attention_gdn_gb300 as gdn
    d = {n: x[n].cuda() for n in ("q", "k", "v", "g", "beta")}
    o = torch.empty((2, HV, 128), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    gdn.gdn_step(gdn.step_problem(2, 2, 16, HV, slots), *d.values(), y["states"], o, err, slot_in=t(slot_in),
                 slot_out=t(slot_out))
    small = run(x, False, None, None)
    assert gdn.gdn_device_status(err) == 0
    assert torch.equal(o, small[0])
    assert torch.equal(big[slot_out[0]], small[1][0]) and torch.equal(big[slot_out[1]], small[1][1])


@pytest.mark.parametrize("slot_in,slot_out,cu", [
    ([3, 1], [0, 1], [0, 1, 2]),      # a start outside the pool
    ([-2, 1], [0, 1], [0, 1, 2]),
    ([0, 1], [0, 3], [0, 1, 2]),      # a target outside the pool
    ([0, 1], [0, -5], [0, 1, 2]),
    ([0, 1], [0, 1], [0, 1, 3]),      # tokens past T
    ([0, 1], [0, 1], [0, 2, 1]),      # bounds that go back
    ([0, 1], [0, 1], [-1, 1, 2]),
])
def test_bad_tables_are_reported_and_stay_in_bounds(slot_in, slot_out, cu):
    """The error word is set, what is wrong is skipped, the other sequence is served."""
    x = make([1, 1], 1, 2, 3, "bf16", False, seed=11)
    bad = dict(x, cu=np.array(cu, np.int32))
    o, pool, status = run(bad, False, slot_in, slot_out)
    assert status == 7
    assert torch.equal(pool[2].cpu(), x["states"][2])
    good = run(x, False, [0, 1], [0, 1])
    n = 1 if slot_in[0] not in (0, 1) or cu[0] < 0 else 0
    if cu != [0, 2, 1]:
        assert torch.equal(o[n], good[0][n]) and torch.equal(pool[n], good[1][n])


def test_graph_replay_takes_new_lengths():
    """A captured step reads cu_seqlens and the slots anew at every replay."""
    import linear_attention_gdn_gb300 as gdn
    x = make([2, 2], 1, 2, 2, "bf16", False, seed=12)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "g", "beta", "states")}
    o = torch.empty((4, 2, 128), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    prob = gdn.step_problem(4, 2, 1, 2, 2)
    args = [d[n] for n in ("q", "k", "v", "g", "beta", "states")]
    gdn.gdn_step(prob, *args, o, err, cu_seqlens_dev=cu)   # loads the kernel
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_step(prob, *args, o, err, cu_seqlens_dev=cu)
    for lens in ([1, 3], [4, 0]):
        d["states"].copy_(x["states"])
        y = dict(x, cu=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        cu.copy_(torch.from_numpy(y["cu"]))
        graph.replay()
        want = run(y, False, None, None)
        assert torch.equal(o, want[0]) and torch.equal(d["states"], want[1])


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,H,HV", [(1, 1, 1), (3, 2, 4), (2, 19, 19), (1, 13, 39), (20, 1, 2), (160, 1, 1)])
def test_head_counts_around_the_kernels_choice(N, H, HV, dtype, kda):
    """Few heads, a middle number and many, each with single tokens and with a few: the kernels differ in how they spread a
    state over warps."""
    for lens in ([1] * N, [1 + (3 * n + 1) % 5 for n in range(N)]):
        T = sum(lens)
        x = make(lens, H, HV, N + 2, dtype, kda, seed=N * HV + T)
        slot_in = [(n + 1) % (N + 2) if n % 3 else -1 for n in range(N)]
        slot_out = np.full(T, -1)
        for n, end in enumerate(np.cumsum(lens)):
            slot_out[end - 1] = (n + 1) % (N + 2)
        check(x, run(x, kda, slot_in, slot_out, packed=True), slot_in, slot_out)


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("H,HV,lens", [(16, 48, [24, 24]), (16, 48, [24, 23]), (13, 39, [30, 21]), (19, 38, [30, 21]),
                                       (2, 4, [24] * 20), (8, 16, [0, 60, 1, 80, 4, 0]), (1, 1, [25] * 80)])
def test_lengths_around_the_choice_of_blocks(H, HV, lens, kda):
    """Lengths from which a CTA a head takes four tokens at a time, and heads for which it does: a state wanted within."""
    T, N = sum(lens), len(lens)
    x = make(lens, H, HV, N + 3, "bf16", kda, seed=T + HV)
    slot_out = np.full(T, -1)
    ends = np.cumsum(lens)
    for n in range(N):
        if lens[n]:
            slot_out[ends[n] - 1] = n
    slot_out[10:13] = [N, N + 1, N + 2]
    check(x, run(x, kda, list(range(N)), slot_out), list(range(N)), slot_out)


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("H,HV,lens", [(1, 1, [32]), (2, 4, [33, 40]), (1, 3, [31, 0, 90, 2]), (1, 1, [200]),
                                       (1, 2, [35] * 18), (16, 64, [67])])
def test_few_heads_in_blocks(H, HV, lens, dtype, kda):
    """Few heads and long sequences, whose blocks are prepared by other warps: states wanted in a row, in the middle and at
    the end, from a slot and from none."""
    T, N = sum(lens), len(lens)
    x = make(lens, H, HV, 2 * N + 9, dtype, kda, seed=T + HV)
    slot_in = [n if n % 3 != 1 else -1 for n in range(N)]
    slot_out = np.full(T, -1)
    ends = np.cumsum(lens)
    for n in range(N):
        if lens[n]:
            slot_out[ends[n] - 1] = N + n
    first = list(range(3, 8)) + [17, 30]
    slot_out[first] = [2 * N + i for i in range(len(first))]
    check(x, run(x, kda, slot_in, slot_out, packed=N == 2), slot_in, slot_out)


def test_few_heads_in_blocks_keep_every_state_and_report_bad_tables():
    x = make([60, 50], 1, 3, 112, "fp32", True, seed=31, steep=True)
    x["g"][7] = x["g"][61] = -float("inf")
    every = [2 + t for t in range(110)]
    check(x, run(x, True, [0, 1], every), [0, 1], every)
    good = run(x, True, [0, 1], None)
    bad = np.full(110, -1)
    bad[[20, 59, 109]] = [112, 0, 1]
    o, pool, status = run(x, True, [0, 1], bad)
    bad[20] = -1
    assert status == 7 and torch.equal(o[60:], good[0][60:])
    check(x, (o, pool, 0), [0, 1], bad)
    for slot_in, cu in (([112, 1], [0, 60, 110]), ([0, 1], [-1, 60, 110])):
        o, pool, status = run(dict(x, cu=np.array(cu, np.int32)), True, slot_in, None)
        assert status == 7 and torch.equal(o[60:], good[0][60:]) and torch.equal(pool[1], good[1][1])
    _, pool, status = run(dict(x, cu=np.array([0, 60, 111], np.int32)), True, [0, 1], None)
    assert status == 7 and torch.equal(pool[0], good[1][0]) and torch.equal(pool[1].cpu(), x["states"][1])
