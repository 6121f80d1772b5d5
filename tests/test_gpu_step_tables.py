"""The tables of a generation step on the GPU against the oracle's, entry by entry."""
import numpy as np
import pytest
import torch

import linear_attention_gdn_gb300 as gdn
from oracle import step_tables

pytestmark = pytest.mark.gpu
i32 = torch.int32


def books(N, block, row, context, spare, seed, done=0, lo=0, hi=5):
    r = np.random.default_rng(seed)
    ctx = r.integers(0, context + 1, N)
    lengths = r.integers(lo, hi + 1, N)
    lengths[r.permutation(N)[:done]] = -1
    held = -(-ctx // block)
    slots = int(held.sum()) + spare
    order = r.permutation(slots)
    table = np.full((N, row), -7)
    at = 0
    for n in range(N):
        table[n, :held[n]] = order[at:at + held[n]]
        at += held[n]
    stack = np.full(slots, -9)
    stack[:spare] = order[at:]
    return lengths, ctx, table, stack, spare, slots


def run(lengths, ctx, table, stack, count, slots, T, block, in_place=False, positions=True, offset=0):
    N, row = table.shape

    def put(a):   # at any element of a longer tensor
        a = np.asarray(a)
        flat = torch.full((a.size + offset + 1,), -123, dtype=i32, device="cuda")
        v = flat[offset:offset + a.size].view(a.shape)
        v.copy_(torch.from_numpy(a.astype(np.int32)))
        return v

    want = step_tables.tables(lengths, ctx, table, stack, count, T, block, slots)
    dl, dc, db, ds, dn = put(lengths), put(ctx), put(table), put(stack), put([count])
    new = lambda n: put(np.full(n, -55))  # noqa: E731
    out, left = (dc, dn) if in_place else (new(N), new(1))
    cu, pos, sin, sout = new(N + 1), new(T) if positions else None, new(N), new(T)
    err = torch.zeros(1, dtype=i32, device="cuda")
    gdn.gdn_step_tables(gdn.tables_problem(N, T, block, row, slots), dl, dc, out, db, ds, dn, left, cu, pos, sin, sout, err)
    assert gdn.gdn_device_status(err) == (7 if want["error"] else 0)
    for name, t in (("cu", cu), ("positions", pos), ("slot_in", sin), ("slot_out", sout), ("context", out), ("blocks", db),
                    ("free_list", ds), ("free_count", left)):
        if t is not None:
            np.testing.assert_array_equal(t.cpu().numpy().reshape(-1), np.asarray(want[name]).reshape(-1), err_msg=name)
    return want


@pytest.mark.parametrize("N,block,row,context,hi,done", [
    (1, 64, 4, 100, 1, 0), (1, 1, 50, 20, 9, 0), (3, 4, 9, 20, 8, 1), (64, 64, 70, 4000, 1, 0), (33, 16, 9, 60, 40, 5), (1000, 100, 12, 900, 7, 100),
    (1025, 64, 5, 200, 64, 30), (2500, 7, 40, 200, 50, 0), (5000, 64, 3, 90, 1, 1000),
])
@pytest.mark.parametrize("offset", [0, 1])
def test_against_the_oracle(N, block, row, context, hi, done, offset):
    for lo in (0, min(1, hi)):
        b = books(N, block, row, context, spare=N * (hi // block + 2), seed=N + lo, done=done, lo=lo, hi=hi)
        T = int(np.maximum(b[0], 0).sum())
        run(*b, T=T + 5, block=block, offset=offset)
        run(*b, T=T, block=block, in_place=True, positions=bool(offset))


@pytest.mark.parametrize("N", [5, 300, 3000])
def test_requests_that_do_not_fit_wait(N):
    for spare in (0, 1, N // 3):
        b = books(N, 4, 10, 20, spare=spare, seed=spare, done=N // 10, lo=0, hi=9)
        total = int(np.maximum(b[0], 0).sum())
        want = run(*b, T=total, block=4)
        assert want["cu"][-1] < total or spare
        run(*b, T=total // 2, block=4)
        run(*b, T=0, block=4)


def test_what_ended_requests_give_back_is_taken_again():
    want = run(np.array([8, -1, 4]), np.array([4, 12, 0]), np.array([[5, -1, -1], [2, 0, 4], [-1, -1, -1]]), np.full(6, -1), 0, 6, 12, 4)
    assert want["slot_out"][:12] == [-1, -1, -1, 4, -1, -1, -1, 0, -1, -1, -1, 2] and want["free_count"] == 0


@pytest.mark.parametrize("change", [dict(length=-2), dict(length=10 ** 9), dict(ctx=-1), dict(ctx=2 ** 31 - 1), dict(count=-1), dict(count=10 ** 6)])
def test_bad_books_are_reported(change):
    lengths, ctx, table, stack, count, slots = books(6, 4, 8, 16, spare=20, seed=1, done=1)
    i = int(np.nonzero(lengths >= 0)[0][0])
    lengths[i] = change.get("length", lengths[i])
    ctx[i] = change.get("ctx", ctx[i])
    run(lengths, ctx, table, stack, change.get("count", count), slots, 40, 4)


def test_more_given_back_than_there_are():
    lengths, ctx = np.array([-1, 1]), np.array([8, 0])
    run(lengths, ctx, np.array([[0, 1], [-1, -1]]), np.array([2, -1]), 1, 2, 4, 4)


def test_no_requests_and_no_tokens():
    run(np.zeros(0), np.zeros(0), np.zeros((0, 3)), np.array([1, 0]), 2, 2, 3, 4)
    run(np.array([0]), np.array([5]), np.array([[1, 0]]), np.array([-1, -1]), 0, 2, 0, 4)


def test_one_long_prompt():
    N, block = 1, 64
    b = (np.array([100001]), np.array([37]), np.full((1, 1600), -1), np.arange(2000), 1999, 2000)
    b[2][0, 0] = 1999
    run(*b, T=100001, block=block)


def test_a_captured_step_goes_on():
    """In place and in a graph: every replay takes the next tokens, block after block."""
    N, block, row, slots = 3, 4, 6, 20
    lengths = torch.tensor([1, 2, 0], dtype=i32, device="cuda")
    ctx, table = torch.zeros(N, dtype=i32, device="cuda"), torch.full((N, row), -1, dtype=i32, device="cuda")
    free, count = torch.arange(slots, dtype=i32, device="cuda"), torch.tensor([slots], dtype=i32, device="cuda")
    cu, sin = torch.empty(N + 1, dtype=i32, device="cuda"), torch.empty(N, dtype=i32, device="cuda")
    pos, sout, err = (torch.empty(n, dtype=i32, device="cuda") for n in (4, 4, 1))
    err.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_step_tables(gdn.tables_problem(N, 4, block, row, slots), lengths, ctx, ctx, table, free, count, count, cu, pos, sin, sout, err)
    host = dict(context=[0] * N, blocks=np.full((N, row), -1), free_list=np.arange(slots), free_count=slots)
    for step in range(9):
        if step == 5:   # the scheduler takes another request in
            lengths.copy_(torch.tensor([1, 0, 1]))
        host = step_tables.tables(lengths.tolist(), host["context"], host["blocks"], host["free_list"], host["free_count"], 4, block, slots)
        graph.replay()
        torch.cuda.synchronize()
        for name, t in (("cu", cu), ("positions", pos), ("slot_in", sin), ("slot_out", sout), ("context", ctx), ("blocks", table),
                        ("free_count", count)):
            np.testing.assert_array_equal(t.cpu().numpy().reshape(-1), np.asarray(host[name]).reshape(-1), err_msg=name)
    assert gdn.gdn_device_status(err) == 0
