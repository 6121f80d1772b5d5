"""A generation step of a model with both kinds of layers in one captured graph: the step's tables, the norm with the residual's
addition, the rule's step and the linear attention's on their pools.  And requests that begin as others did."""
import numpy as np
import pytest
import torch

import linear_attention_gdn_gb300 as gdn
from tests.la_testutil import R, SCALE, f64
from tests.step_testutil import U, within
from tests.test_gpu_norm import EPS, inverse, root
from tests.test_gpu_step import check

pytestmark = pytest.mark.gpu
i32 = torch.int32
N, H, HV, B, ROWS, SLOTS = 3, 1, 2, 2, 5, 12
C = (2 * H + HV) * 128


class Step:
    """Buffers of a step of up to N tokens, and its kernels."""

    def __init__(self):
        g = torch.Generator().manual_seed(0)
        rnd = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
        new = lambda *s: torch.zeros(s, dtype=i32, device="cuda")  # noqa: E731
        self.lengths, self.err = new(N), new(1)
        self.books = dict(ctx=new(N), table=new(N, ROWS) - 1, free=torch.randperm(SLOTS, generator=g).to(i32).cuda(), count=new(1) + SLOTS,
                          rule=rnd(SLOTS, HV, 128, 128), linear=rnd(SLOTS, HV, 128, 128))
        self.cu, self.pos, self.slot_in, self.slot_out = new(N + 1), new(N), new(N), new(N)
        self.x, self.r, self.h, self.y, self.h2, self.y2 = (rnd(N, C).bfloat16() for _ in range(6))
        self.w, self.w2 = 1 + 0.2 * rnd(C), 1 + 0.2 * rnd(C)
        self.g, self.beta = -torch.rand(N, HV, generator=g).cuda(), torch.rand(N, HV, generator=g).cuda()
        self.decay = torch.tensor([-0.05, -0.5], device="cuda")
        self.o, self.o2 = (torch.zeros(N, HV, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.norm = gdn.norm_problem(N, C, EPS)
        self.rule, self.linear = (gdn.step_problem(N, N, H, HV, SLOTS, SCALE, l2, torch.bfloat16, (C, C, C)) for l2 in (True, False))

    def heads(self, y):
        y = y.view(N, -1, 128)
        return y[:, :H], y[:, H:2 * H], y[:, 2 * H:]

    def __call__(self):
        b, tables = self.books, (self.cu, self.slot_in, self.slot_out)
        gdn.gdn_step_tables(gdn.tables_problem(N, N, B, ROWS, SLOTS), self.lengths, b["ctx"], b["ctx"], b["table"], b["free"], b["count"],
                            b["count"], self.cu, self.pos, self.slot_in, self.slot_out, self.err)
        gdn.gdn_add_norm_fwd(self.norm, self.x, self.r, self.w, self.h, self.y)
        gdn.gdn_step(self.rule, *self.heads(self.y), self.g, self.beta, b["rule"], self.o, self.err, *tables)
        o = self.o.view(N, HV * 128)
        gdn.gdn_add_norm_fwd(self.norm, torch.cat([o, o], 1), self.h, self.w2, self.h2, self.y2)   # (in place of a projection)
        gdn.gdn_la_step(self.linear, *self.heads(self.y2), self.decay, b["linear"], self.o2, self.err, *tables)

    def outputs(self):
        return dict(h=self.h, y=self.y, o=self.o, h2=self.h2, y2=self.y2, o2=self.o2, cu=self.cu, pos=self.pos, slot_in=self.slot_in,
                    slot_out=self.slot_out, **self.books)


def test_a_captured_step_of_both_layers():
    """Every replay has the bits of the same calls one by one, and each operator's values are right for what it was given: the
    norm's and the linear attention's by their formulas, the rule's by its oracle."""
    s = Step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s()
    gen = torch.Generator().manual_seed(1)
    for lengths in ([1, 1, 1], [1, 0, 1], [1, 1, 0], [0, 1, -1], [1, -1, 1], [1, 1, 1]):
        s.lengths.copy_(torch.tensor(lengths))
        for t in (s.x, s.r):
            t.copy_(torch.randn(N, C, generator=gen))
        for t in (s.o, s.o2):
            t.zero_()
        before = {m: t.clone() for m, t in s.books.items()}
        graph.replay()
        got = {m: t.clone() for m, t in s.outputs().items()}
        for m, t in before.items():
            s.books[m].copy_(t)
        for t in (s.o, s.o2):
            t.zero_()
        s()
        for m, t in s.outputs().items():
            assert torch.equal(t, got[m]), m
        assert gdn.gdn_device_status(s.err) == 0

        n = sum(max(a, 0) for a in lengths)
        assert got["cu"].tolist() == np.cumsum([0] + [max(a, 0) for a in lengths]).tolist()
        slot_in, slot_out = got["slot_in"].tolist(), got["slot_out"].tolist()
        for x, r, w, h, y in ((s.x, s.r, s.w, got["h"], got["y"]),
                              (torch.cat([got["o"].view(N, -1)] * 2, 1), got["h"], s.w2, got["h2"], got["y2"])):
            within("h", h, f64(x) + f64(r), R * np.abs(f64(x) + f64(r)))
            z = f64(h) * inverse(f64(h), C) * f64(w)
            within("y", y, z, (R + root(C) + 2 * U) * np.abs(z))
        q, k, v = s.heads(got["y"])
        check(dict(q=q, k=k, v=v, g=s.g, beta=s.beta, states=before["rule"].cpu(), cu=got["cu"].cpu().numpy()), (got["o"], got["rule"], 0),
              slot_in, slot_out)
        q, k, v = (f64(t) for t in s.heads(got["y2"]))
        old, pool = f64(before["linear"]), f64(got["linear"])
        for i in range(N):
            if lengths[i] != 1:
                continue
            t = int(got["cu"][i])
            for e in range(HV):
                a, S = np.exp(float(s.decay[e])), old[slot_in[i], e] if slot_in[i] >= 0 else np.zeros((128, 128))
                S1, A = a * S + np.outer(k[t, 0], v[t, e]), a * np.abs(S) + np.abs(np.outer(k[t, 0], v[t, e]))
                # a state: the exponential (2 last places, 4 U), a product and a sum; o: 128 products and 26 operations more in their sums
                assert (np.abs(pool[slot_out[t], e] - S1) <= 8 * U * A).all()
                o = SCALE * S1.T @ q[t, 0]
                within("o", f64(got["o2"][t, e]), o, R * np.abs(o) + 34 * U * SCALE * A.T @ np.abs(q[t, 0]) + 1e-30)
        written = {slot_out[t] for t in range(n)}
        rest = [i for i in range(SLOTS) if i not in written]
        assert torch.equal(got["linear"][rest], before["linear"][rest])


def test_a_request_begins_with_a_copy_of_anothers_block():
    """A slot stands in one request's row, with which it goes back.  A request that begins as another did has a copy of its block's
    state in a slot of its own; in the end every slot is free once."""
    block, rows, slots = 8, 4, 10
    i = lambda *a: torch.tensor(a, dtype=i32, device="cuda")  # noqa: E731
    lengths, ctx, table = i(20, 0), i(0, 0), torch.full((2, rows), -1, dtype=i32, device="cuda")
    free, count, err = torch.arange(slots, dtype=i32, device="cuda"), i(slots), i(0)
    pool = torch.randn(slots, 4, device="cuda")
    cu, pos, slot_in, slot_out = i(0, 0, 0), torch.zeros(20, dtype=i32, device="cuda"), i(0, 0), torch.zeros(20, dtype=i32, device="cuda")

    def step():
        gdn.gdn_step_tables(gdn.tables_problem(2, 20, block, rows, slots), lengths, ctx, ctx, table, free, count, count, cu, pos, slot_in,
                            slot_out, err)
        held = [int(x) for n in range(2) for x in table[n, :-(-int(ctx[n]) // block)]]
        assert sorted(held + free[:int(count)].tolist()) == list(range(slots))

    step()
    count -= 1   # a slot of its own, between two steps
    slot = free[count.long()]
    pool[slot.long()] = pool[table[0, :1].long()]
    table[1, :1] = slot
    ctx[1] = 8
    lengths.copy_(i(-1, 6))
    step()
    assert slot_in.tolist() == [-1, int(slot)] and pos[:6].tolist() == list(range(8, 14)) and int(ctx[0]) == 0
    lengths.copy_(i(0, -1))
    step()
    assert int(count) == slots and gdn.gdn_device_status(err) == 0
