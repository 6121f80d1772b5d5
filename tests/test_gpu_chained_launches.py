"""Chained kernels (those of the steps and of the norm with rotation, which may be placed while the one before ends) among
kernels of any other kind: every order gives the bits of the same calls with a wait after each."""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
N, H, HV, W, D = 24, 2, 6, 4, 128
C = (2 * H + HV) * D


class Chain:
    """Operations that feed one another over shared buffers: whoever starts too early reads what is not yet there, whoever
    writes too early changes what is still read."""

    def __init__(self):
        import linear_attention_gdn_gb300 as gdn
        self.gdn = gdn
        gen = torch.Generator(device="cuda").manual_seed(1)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        # (tables and the error word as views that do not start on 16 bytes)
        table = lambda a: torch.tensor([0] + a, dtype=torch.int32, device="cuda")[1:]  # noqa: E731
        self.rows, self.y = rnd(N, C).bfloat16(), rnd(N, C).bfloat16()
        self.w, self.b, self.wq = 0.5 * rnd(C, W), 0.1 * rnd(C), 1 + 0.1 * rnd(D)
        self.window, self.states = rnd(N, W - 1, C).bfloat16(), 0.5 * rnd(N, HV, D, D)
        self.g, self.beta = -rnd(N, HV).abs(), torch.sigmoid(rnd(N, HV))
        self.gk = -rnd(N, HV, D).abs()
        self.qn, self.kn = (rnd(N, H, D).bfloat16() for _ in range(2))
        self.dy = rnd(N, C).bfloat16()
        self.o = rnd(N, HV, D).bfloat16()
        self.dwq, self.dwk = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
        self.slot, self.slots_out = table(list(range(N - 1, -1, -1))), table(list(range(N - 1, -1, -1)))
        self.cu1, self.cu3 = table(list(range(N + 1))), table([0, 10, 11, N])
        self.pos, self.err = table(list(range(100, 100 + N))), torch.zeros(2, dtype=torch.int32, device="cuda")[1:]
        freq, _ = gdn.gdn_rope_frequencies(64)
        self.freq = torch.from_numpy(freq).cuda()
        self.conv, self.conv3 = (gdn.conv_step_problem(N, n, C, N, W=W) for n in (N, 3))
        self.rule, self.rule3 = (gdn.step_problem(N, n, H, HV, N, l2norm=True, strides=(0, 0, C)) for n in (N, 3))
        self.qk = gdn.qk_problem(N, H, H, rot=64, norm=gdn.NORM_L2, q_strides=(C, D), k_strides=(C, D))
        self.ws = torch.empty(gdn.gdn_qk_workspace_bytes(self.qk), dtype=torch.uint8, device="cuda")
        self.cu = np.array([0, 10, 11, N], np.int32)
        self.train = gdn.conv_problem(N, 3, C, W)
        self.big = torch.zeros(1 << 24, device="cuda")
        self.pinned = torch.zeros(N, dtype=torch.int32).pin_memory()

    def heads(self, rows):
        x = rows.unflatten(1, (C // D, D))
        return x[:, :H], x[:, H:2 * H], x[:, 2 * H:]

    def op(self, name):
        g = self.gdn
        q, k, v = self.heads(self.y)
        if name == "conv":
            g.gdn_conv1d_step(self.conv, self.rows, self.w, self.b, self.window, self.y, self.err, slot_in=self.slot,
                              slot_out=self.slots_out)
        elif name == "conv_short":
            g.gdn_conv1d_step(self.conv, self.rows, self.w, self.b, self.window, self.y, self.err, cu_seqlens_dev=self.cu1)
        elif name == "conv_ranges":
            g.gdn_conv1d_step(self.conv3, self.rows, self.w, self.b, self.window, self.y, self.err, cu_seqlens_dev=self.cu3)
        elif name == "qk":
            g.gdn_qk_norm_rope_fwd(self.qk, q, k, self.wq, None, self.freq, self.pos, None, self.qn, self.kn)
        elif name == "qk_bwd":
            g.gdn_qk_norm_rope_bwd(self.qk, q, k, self.wq, None, self.freq, self.pos, None, self.qn, self.kn,
                                   *self.heads(self.dy)[:2], self.dwq, self.dwk, self.ws)
        elif name == "step":
            g.gdn_step(self.rule, self.qn, self.kn, v, self.g, self.beta, self.states, self.o, self.err, slot_in=self.slot)
        elif name == "kda_few":
            g.gdn_kda_step(self.rule3, self.qn, self.kn, v, self.gk, self.beta, self.states, self.o, self.err,
                           cu_seqlens_dev=self.cu3)
        elif name == "train":   # a kernel launched as always
            g.gdn_conv1d_fwd(self.train, self.rows, self.w, self.b, self.cu3.clone(), self.cu, self.y)
        elif name == "feed":
            self.rows.copy_((0.5 * self.rows.float() + 0.1 * self.dy.float() + self.o.flatten(1).float().repeat(1, 2)[:, :C]).bfloat16())
        elif name == "gates":
            self.beta.mul_(0.999).add_(5e-4)
            self.wq.add_(0.01 * self.dwq.tanh())
        elif name == "long":   # what follows waits for something
            self.big.add_(1)
            self.rows.add_((self.big[0] * 1e-3).bfloat16())
        elif name == "clear":
            self.qn.zero_()
        elif name == "copy":
            self.pos.add_(1)
            self.pinned.copy_(self.pos, non_blocking=True)
            self.pos.copy_(self.pinned, non_blocking=True)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.rows, self.y, self.window, self.states, self.qn, self.kn, self.o, self.dy, self.dwq, self.dwk,
                                    self.wq, self.pos, self.err)]


OPS = ["conv", "conv_short", "conv_ranges", "qk", "qk_bwd", "step", "kda_few", "train", "feed", "gates", "long", "clear", "copy"]


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("graph", [False, True])
def test_any_order_gives_the_same_bits(seed, graph):
    rng = random.Random(seed)
    order = [rng.choice(OPS) for _ in range(60)]
    if graph:
        order = [n for n in order if n not in ("copy", "train")]
    a, b = Chain(), Chain()
    for name in order:
        a.op(name)
        torch.cuda.synchronize()
    if graph:
        b.op("conv"), b.op("conv_short"), b.op("conv_ranges"), b.op("qk"), b.op("qk_bwd"), b.op("step"), b.op("kda_few")
        b = Chain()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for name in order:
                b.op(name)
        g.replay()
    else:
        for name in order:
            b.op(name)
    want, got = a.results(), b.results()
    assert int(want[-1]) == 0
    for i, (x, y) in enumerate(zip(want, got)):
        assert torch.equal(x, y) and torch.isfinite(x.float()).all(), i
