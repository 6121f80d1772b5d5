"""A gated-delta-rule layer from training to generation, through the library's entry points.

The layer's core, between its projections: the causal convolution over packed q, k, v rows, the norm of q and k per head
with the position rotation, and the rule.

    python examples/generate.py

prefills a ragged batch of prompts (gdn_conv1d_fwd, gdn_qk_norm_rope_fwd, gdn_fwd_states), generates from there one
token at a time on pools of windows and states (gdn_conv1d_step, gdn_qk_norm_rope_fwd, gdn_step, captured once in a CUDA
graph), and compares the outputs with one prefill over prompts and generated tokens together; then takes the
gradients of the whole (gdn_bwd, gdn_qk_norm_rope_bwd, gdn_conv1d_bwd).  Random weights, random rows in place of the
projections' outputs.
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import linear_attention_gdn_gb300 as gdn  # noqa: E402

D = 128


class Layer:
    """Weights of the layer's core, and its two ways through the library."""

    def __init__(self, H=4, HV=12, W=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.H, self.HV, self.W, self.C = H, HV, W, (2 * H + HV) * D
        self.w, self.b = 0.5 * rnd(self.C, W), 0.1 * rnd(self.C)
        self.wq, self.wk = 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D)
        self.norm = gdn.NORM_L2   # unit keys times weights near one: what the rule wants
        freq, self.m = gdn.gdn_rope_frequencies(D // 2, scaling=gdn.ROPE_PARTS, factor=4.0, original=4096)
        self.freq = torch.from_numpy(freq).cuda()

    def heads(self, rows):
        """Views of q, k, v [T, heads, D] of packed rows [T, C]."""
        x = rows.unflatten(1, (self.C // D, D))
        return x[:, :self.H], x[:, self.H:2 * self.H], x[:, 2 * self.H:]

    def qk_problem(self, T, N=0):
        return gdn.qk_problem(T, self.H, self.H, rot=D // 2, layout=gdn.ROPE_HALF, norm=self.norm, mscale=self.m, N=N,
                              q_strides=(self.C, D), k_strides=(self.C, D))

    def prefill(self, rows, g, beta, cu, states=None):
        """Outputs of packed documents; `states` [N, HV, D, D] receives the state after each.  Keeps what backward()
        needs."""
        T, N, H, HV = rows.shape[0], len(cu) - 1, self.H, self.HV
        cu_dev = torch.from_numpy(cu).cuda()
        y = torch.empty_like(rows)
        gdn.gdn_conv1d_fwd(gdn.conv_problem(T, N, self.C, self.W), rows, self.w, self.b, cu_dev, cu, y)
        q, k, v = self.heads(y)
        qn, kn = (torch.empty((T, H, D), dtype=rows.dtype, device="cuda") for _ in range(2))
        gdn.gdn_qk_norm_rope_fwd(self.qk_problem(T, N), q, k, self.wq, self.wk, self.freq, None, cu_dev, qn, kn)
        v = v.contiguous()
        prob = gdn.problem(T, N, H, HV, l2norm=False)
        buf = gdn.Buffers(prob, cu)
        o = torch.empty((T, HV, D), dtype=rows.dtype, device="cuda")
        gdn.gdn_fwd_states(prob, qn, kn, v, g, beta, cu_dev, cu, None, o, states, buf.saved, buf.workspace)
        self.kept = (rows, g, beta, cu, cu_dev, y, qn, kn, v, prob, buf)
        return o

    def backward(self, do):
        """Gradients of the last prefill: of the rows, the gates, and the weights."""
        rows, g, beta, cu, cu_dev, y, qn, kn, v, prob, buf = self.kept
        T, N = rows.shape[0], len(cu) - 1
        dq, dk, dv = (torch.empty_like(t) for t in (qn, kn, v))
        dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
        gdn.gdn_bwd(prob, qn, kn, v, g, beta, cu_dev, cu, do, buf.saved, dq, dk, dv, dg, dbeta, buf.workspace)
        dy = torch.empty_like(y)   # q's and k's gradients go straight into its rows
        yq, yk, _ = self.heads(y)
        gq, gk, gv = self.heads(dy)
        gv.copy_(dv)
        dwq, dwk = torch.empty_like(self.wq), torch.empty_like(self.wk)
        qk = self.qk_problem(T, N)
        ws = torch.empty(gdn.gdn_qk_workspace_bytes(qk), dtype=torch.uint8, device="cuda")
        gdn.gdn_qk_norm_rope_bwd(qk, yq, yk, self.wq, self.wk, self.freq, None, cu_dev, dq, dk, gq, gk, dwq, dwk, ws)
        conv = gdn.conv_problem(T, N, self.C, self.W)
        dx, dw, db = torch.empty_like(rows), torch.empty_like(self.w), torch.empty_like(self.b)
        ws = torch.empty(gdn.gdn_conv1d_workspace_bytes(conv, cu), dtype=torch.uint8, device="cuda")
        gdn.gdn_conv1d_bwd(conv, rows, self.w, self.b, cu_dev, cu, dy, dx, dw, db, ws)
        return dict(rows=dx, g=dg, beta=dbeta, w=dw, b=db, wq=dwq, wk=dwk)


class Generator:
    """A batch's pools and the captured step of one token for each sequence."""

    def __init__(self, layer, N, slots):
        H, HV, C = layer.H, layer.HV, layer.C
        new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.layer, self.N = layer, N
        self.window, self.states = new(slots, layer.W - 1, C), new(slots, HV, D, D, dtype=torch.float32)
        self.rows, self.y, self.o = new(N, C), new(N, C), new(N, HV, D)
        self.qn, self.kn = new(N, H, D), new(N, H, D)
        self.g, self.beta = new(N, HV, dtype=torch.float32), new(N, HV, dtype=torch.float32)
        self.slot, self.position = new(N, dtype=torch.int32), new(N, dtype=torch.int32)
        self.err = new(1, dtype=torch.int32)
        self.conv = gdn.conv_step_problem(N, N, C, slots, W=layer.W)
        self.qk = layer.qk_problem(N)
        self.rule = gdn.step_problem(N, N, H, HV, slots, l2norm=False, strides=(0, 0, C))   # v stays in y's rows
        self.graph = None

    def launch(self):
        la = self.layer
        gdn.gdn_conv1d_step(self.conv, self.rows, la.w, la.b, self.window, self.y, self.err, slot_in=self.slot,
                            slot_out=self.slot)
        q, k, v = la.heads(self.y)
        gdn.gdn_qk_norm_rope_fwd(self.qk, q, k, la.wq, la.wk, la.freq, self.position, None, self.qn, self.kn)
        gdn.gdn_step(self.rule, self.qn, self.kn, v, self.g, self.beta, self.states, self.o, self.err, slot_in=self.slot,
                     slot_out=self.slot)
        self.position += 1

    def capture(self):
        """Call before the pools are filled: the launches that load the kernels run on them."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.launch()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.launch()

    def step(self, rows, g, beta):
        self.rows.copy_(rows)
        self.g.copy_(g)
        self.beta.copy_(beta)
        self.graph.replay()
        return self.o


def run(lens=(130, 1, 700, 64, 333), new=24, seed=0, say=lambda *a: None):
    """(relative difference of the generated outputs from the prefill of everything, gradients)."""
    layer, N = Layer(seed=seed), len(lens)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    total = [n + new for n in lens]
    ends = np.concatenate([[0], np.cumsum(total)]).astype(np.int32)
    T = int(ends[-1])
    rows = torch.randn((T, layer.C), generator=gen, device="cuda").to(torch.bfloat16)
    g = torch.nn.functional.logsigmoid(2 + 4 * torch.rand((T, layer.HV), generator=gen, device="cuda"))
    beta = torch.rand((T, layer.HV), generator=gen, device="cuda")

    # everything at once
    whole = layer.prefill(rows, g, beta, ends)
    grads = layer.backward(torch.randn(whole.shape, generator=gen, device="cuda").to(torch.bfloat16))

    # the prompts, then token by token; a scheduler hands out slots in any order
    slots = N + 3
    batch = Generator(layer, N, slots)
    batch.capture()
    slot = torch.randperm(slots, generator=gen, device="cuda")[:N]
    prompt = torch.cat([torch.arange(int(a), int(a) + n) for a, n in zip(ends[:-1], lens)]).cuda()
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    states = torch.empty((N, layer.HV, D, D), device="cuda")
    layer.prefill(rows[prompt], g[prompt], beta[prompt], cu, states)
    batch.states[slot] = states
    batch.slot.copy_(slot)
    batch.position.copy_(torch.tensor(lens))
    batch.window.zero_()
    for n, a, s in zip(lens, ends[:-1], slot.tolist()):
        keep = min(n, layer.W - 1)
        batch.window[s, layer.W - 1 - keep:] = rows[int(a) + n - keep:int(a) + n]
    outs = []
    for j in range(new):
        at = torch.tensor([int(a) + n + j for a, n in zip(ends[:-1], lens)], device="cuda")
        outs.append(batch.step(rows[at], g[at], beta[at]).clone())
    status = gdn.gdn_device_status(batch.err)
    if status != 0:
        raise RuntimeError(gdn.gdn_status_string(status))
    at = torch.cat([torch.arange(int(a) + n, int(a) + n + new) for a, n in zip(ends[:-1], lens)]).cuda()
    want, got = whole[at].double(), torch.stack(outs, 1).flatten(0, 1).double()
    off = float((got - want).norm() / want.norm())
    say(f"{N} sequences, {new} tokens each after prompts of {list(lens)}: generated against prefilled, relative "
        f"difference {off:.2e}")
    say("gradient norms: " + ", ".join(f"{n} {float(t.double().norm()):.3g}" for n, t in grads.items()))
    return off, grads


if __name__ == "__main__":
    run(say=print)
