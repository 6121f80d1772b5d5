"""The linear attention, the norm of the residual stream and the step's tables used together: a prompt, then generation with
states kept on the way, and a layer's gradients."""
import numpy as np
import pytest
import torch

import linear_attention_gdn_gb300 as gdn
from oracle import la
from tests.la_testutil import R, SCALE, f64
from tests.step_testutil import within

pytestmark = pytest.mark.gpu
i32 = torch.int32


def test_prompts_then_generation_by_captured_steps():
    """Three requests: their prompts by the chunked form, then single tokens by a graph that makes its own tables and takes
    the step; a state stays every 8 tokens, from which a fourth request goes on."""
    H, HV, B, rows, slots, steps = 1, 2, 8, 12, 40, 19
    prompts = [5, 16, 0]
    N, total = 4, [p + steps for p in prompts] + [0]
    g = torch.Generator().manual_seed(0)
    q, k, v = ([torch.randn(steps + 40, h, 128, generator=g).bfloat16() for _ in range(N)] for h in (H, H, HV))
    q[3][:8], k[3][:8], v[3][:8] = q[0][:8], k[0][:8], v[0][:8]   # the fourth begins as the first did
    decay = torch.tensor([-0.05, -0.5])
    dec, err = decay.cuda(), torch.zeros(1, dtype=i32, device="cuda")
    i = lambda *a: torch.tensor(a, dtype=i32, device="cuda")  # noqa: E731
    new = lambda n: torch.empty(n, dtype=i32, device="cuda")  # noqa: E731
    lengths, ctx, table = i(*prompts, 0), i(0, 0, 0, 0), torch.full((N, rows), -1, dtype=i32, device="cuda")
    free, count = torch.randperm(slots, generator=g).to(i32).cuda(), i(slots)
    pool = torch.full((slots, HV, 128, 128), float("nan"), device="cuda")

    def tables(T):
        out = dict(cu=new(N + 1), pos=new(T), slot_in=new(N), slot_out=new(T))
        return out, lambda: gdn.gdn_step_tables(gdn.tables_problem(N, T, B, rows, slots), lengths, ctx, ctx, table, free, count, count,
                                                out["cu"], out["pos"], out["slot_in"], out["slot_out"], err)

    # the prompts: token by token where states are to stay, else by the chunked form, whose last state goes to the last token's slot
    T = sum(prompts)
    tab, make = tables(T)
    make()
    cu = np.concatenate([[0], np.cumsum(prompts), [T]]).astype(np.int32)
    assert tab["cu"].tolist() == cu.tolist()
    x = [torch.cat([y[n][:prompts[n]] for n in range(3)]).cuda() for y in (q, k, v)]
    o = torch.empty_like(x[2])
    gdn.gdn_la_step(gdn.step_problem(T, N, H, HV, slots, SCALE, False), *x, dec, pool, o, err, tab["cu"], tab["slot_in"], tab["slot_out"])
    o2, s_out = torch.empty_like(o), torch.zeros(N, HV, 128, 128, device="cuda")
    gdn.gdn_la_fwd(gdn.la_problem(T, N, H, HV, SCALE), *x, dec, tab["cu"], cu, None, o2, s_out, err, None)
    outs = [[o[cu[n]:cu[n + 1]]] for n in range(N)]
    chunked = [o2[cu[n]:cu[n + 1]] for n in range(N)]
    for n in (0, 1):   # both forms leave the same state
        slot = int(tab["slot_out"][cu[n + 1] - 1])
        torch.testing.assert_close(pool[slot], s_out[n], rtol=1e-5, atol=1e-5 * float(s_out[n].abs().max()))
        pool[slot] = s_out[n]

    # single tokens, captured
    lengths.copy_(i(1, 1, 1, 0))
    tab, make = tables(3)
    xs = [torch.empty(3, h, 128, dtype=torch.bfloat16, device="cuda") for h in (H, H, HV)]
    o = torch.empty_like(xs[2])

    def step():
        make()
        gdn.gdn_la_step(gdn.step_problem(3, N, H, HV, slots, SCALE, False), *xs, dec, pool, o, err, tab["cu"], tab["slot_in"], tab["slot_out"])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(steps):
        for dst, src in zip(xs, (q, k, v)):
            dst.copy_(torch.stack([src[n][prompts[n] + t] for n in range(3)]))
        graph.replay()
        assert tab["pos"].tolist() == [p + t for p in prompts]
        for n in range(3):
            outs[n].append(o[n:n + 1].clone())
    torch.cuda.synchronize()
    assert ctx.tolist() == total

    # the fourth request takes over the first one's block of 8 tokens and goes on from its state
    table[3, 0] = table[0, 0]
    ctx[3] = 8
    lengths.copy_(i(-1, 0, 0, 6))
    before = int(count)
    tab, make = tables(8)
    make()
    assert tab["slot_in"].tolist()[3] == int(table[0, 0]) and tab["cu"].tolist() == [0, 0, 0, 0, 6]
    assert int(count) == before + -(-total[0] // B) - 1 and int(ctx[0]) == 0
    pad = lambda y: torch.cat([y[3][8:14], y[3][:2]]).cuda()  # noqa: E731  (two rows behind the last sequence)
    o = torch.full((8, HV, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    gdn.gdn_la_step(gdn.step_problem(8, N, H, HV, slots, SCALE, False), pad(q), pad(k), pad(v), dec, pool, o, err, tab["cu"], tab["slot_in"],
                    tab["slot_out"])
    assert o[6:].isnan().all()
    assert gdn.gdn_device_status(err) == 0

    for n, m in ((0, total[0]), (1, total[1]), (2, total[2]), (3, 14)):
        got = torch.cat(outs[n]) if n < 3 else o[:6]
        for h in range(HV):
            Q, K, V = f64(q[n][:m, 0]), f64(k[n][:m, 0]), f64(v[n][:m, h])
            want, S = la.forward(Q, K, V, float(decay[h]), SCALE)
            _, A = la.forward(np.abs(Q), np.abs(K), np.abs(V), float(decay[h]), SCALE)
            # the step: FP32 sums, and one rounding; a state that came from the chunked form is FP32's, too
            size = SCALE * np.einsum("tij,ti->tj", A[1:], np.abs(Q))
            tol = R * np.abs(want) + (4 * m + 60) * 2.0 ** -22 * size
            first = 0 if n < 3 else 8
            within(f"request {n}", got[:, h].contiguous(), want[first:], tol[first:])
            if n < 2:   # the chunked form's outputs: P and the state rounded, too
                p = len(chunked[n])
                spread = SCALE * np.abs(np.tril(np.exp(float(decay[h]) * np.maximum(np.subtract.outer(np.arange(p), np.arange(p)), 0))) * (Q[:p] @ K[:p].T)) @ np.abs(V[:p])
                within("chunked", chunked[n][:, h].contiguous(), want[:p], (R + 2.0 ** -10) * spread + R * np.abs(want[:p]) + 1e-30)


@pytest.mark.parametrize("lengths", [[150], [1, 0, 200]])
def test_a_layers_gradients(lengths):
    """x + r, its norm, whose rows are q, k and v, and the attention over them: dx and dw against FP64 autograd."""
    H, HV = 1, 2
    T, C, N = sum(lengths), (2 * H + HV) * 128, len(lengths)
    g = torch.Generator().manual_seed(1)
    x, r, do = (torch.randn(T, c, generator=g).bfloat16().cuda() for c in (C, C, HV * 128))
    along = torch.randn(T, C, generator=g).bfloat16().cuda()
    w = (0.5 + torch.rand(C, generator=g)).cuda()
    decay = torch.tensor([-0.02, -0.4]).cuda()
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    cud, err = torch.from_numpy(cu).cuda(), torch.zeros(1, dtype=i32, device="cuda")
    norm, att = gdn.norm_problem(T, C), gdn.la_problem(T, N, H, HV, SCALE, strides=(C, C, C))
    h, y = torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_add_norm_fwd(norm, x, r, w, h, y)
    rows = y.view(T, -1, 128)
    split = lambda t: (t[:, :H], t[:, H:2 * H], t[:, 2 * H:])  # noqa: E731
    o = torch.empty(T, HV, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, *gdn.gdn_la_workspace_bytes(att, cu), gdn.gdn_add_norm_workspace_bytes(norm)), dtype=torch.uint8, device="cuda")
    gdn.gdn_la_fwd(att, *split(rows), decay, cud, cu, None, o, None, err, ws)
    grows = torch.empty_like(rows)
    gdn.gdn_la_bwd(att, *split(rows), decay, cud, cu, None, do.view(T, HV, 128), None, *split(grows), None, err, ws)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    gdn.gdn_add_norm_bwd(norm, h, w, grows.view(T, C), along, dx, dw, ws)
    assert gdn.gdn_device_status(err) == 0

    hd, wd = h.double().requires_grad_(), w.double().requires_grad_()
    z = hd / torch.sqrt((hd ** 2).mean(-1, keepdim=True) + 1e-6) * wd
    q, k, v = split(z.view(T, -1, 128))
    out = []
    for d in range(N):
        a, b = int(cu[d]), int(cu[d + 1])
        t = torch.arange(b - a, device="cuda", dtype=torch.float64)
        apart = t[:, None] - t
        A = torch.einsum("rhd,chd->hrc", q[a:b], k[a:b]) * torch.exp(decay.double()[:, None, None] * apart.clamp(min=0)) * (apart >= 0)
        out.append(SCALE * torch.einsum("hrc,chd->rhd", A, v[a:b]))
    want = torch.cat(out)
    ((want * do.view(T, HV, 128).double()).sum() + (hd * along.double()).sum()).backward()
    # By the 2-norm: y is rounded (once, and enters q, k and v), then P and S, then the outputs; each rounding is R / sqrt(3) of
    # what it rounds on average, and in a product of three rounded rows they add up: five of them, with as much again to spare.
    for name, got, ref in (("o", o, want.detach()), ("dx", dx, hd.grad), ("dw", dw, wd.grad)):
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel <= 2 * np.sqrt(5) * R / np.sqrt(3), (name, rel)
