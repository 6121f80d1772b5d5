"""Measured cases of the operators around the gated delta rule for generation and training:

  step        the recurrent form over a pool of states, one decay per head (kda=0) or per key channel (kda=1)
  conv_step   the causal conv1d + SiLU over a pool of windows
  qk_fwd      the norm of q and k per head with the position rotation in the same pass
  qk_bwd      its gradients

`run` computes a case in its plain form, or, where `own` is set, by the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

D = 128            # head size of the recurrent rule
EPS = 1e-6         # under the root of the norms
BASE = 10000.0     # base of the rotation's frequencies
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _step(name, N, lo=1, hi=1, H=16, HV=48, kda=0, dtype="bf16", keep="last", fresh=0, shape_seed=1):
    """N sequences of lo..hi tokens. keep "last": the state goes back to its own slot; "all": the state after every
    token goes to a slot of that token. fresh: how many sequences start from no state."""
    return dict(name=name, op="step", N=N, lo=lo, hi=hi, H=H, HV=HV, kda=kda, dtype=dtype, keep=keep, fresh=fresh,
                shape_seed=shape_seed)


def _conv(name, N, lo=1, hi=1, C=10240, W=4, dtype="bf16", fresh=0, shape_seed=1):
    return dict(name=name, op="conv_step", N=N, lo=lo, hi=hi, C=C, W=W, dtype=dtype, fresh=fresh, shape_seed=shape_seed)


def _qk(name, op, T, docs, HQ=16, HK=16, dim=128, rot=128, layout="half", norm="rms", dtype="bf16", packed=0, start=0,
        stretch=1.0, shape_seed=1):
    """docs 0: a position for each token is an input (drawn up to `start`); else so many packed documents. packed: q and
    k are views of one projection's rows, `packed` heads wide. stretch: how much longer than trained the context is."""
    return dict(name=name, op=op, T=T, docs=docs, HQ=HQ, HK=HK, dim=dim, rot=rot, layout=layout, norm=norm, dtype=dtype,
                packed=packed, start=start, stretch=stretch, shape_seed=shape_seed)


def listed():
    return [
        # one user's next token in one layer: nothing but latency
        _step("step_1", 1),
        # an ordinary serving batch, one token each
        _step("step_64", 64, fresh=3),
        # a large serving batch: the states' bandwidth
        _step("step_512", 512),
        # drafts of 1 to 8 tokens to verify, the state after each kept so that a rejected tail can be dropped
        _step("step_verify", 24, lo=1, hi=8, keep="all", dtype="fp16"),
        # the per-channel rule, an odd batch, one head of q and k to each value head
        _step("kda_step_37", 37, H=32, HV=32, kda=1),
        # the per-channel rule on the ragged rest of prompts: some empty, the longest 160 tokens
        _step("kda_step_ragged", 6, lo=0, hi=160, kda=1, fresh=2, shape_seed=3),
        # the convolution in front of a batch's single tokens
        _conv("conv_step_64", 64, fresh=3),
        # the convolution over packed pieces of prompts that go on from a window
        _conv("conv_step_ragged", 12, lo=0, hi=4096, fresh=4, shape_seed=5),
        # a batch's single tokens deep in their contexts; rows of the packed q, k, v projection
        _qk("qk_fwd_64", "qk_fwd", 64, 0, packed=80, start=500000, stretch=8.0),
        # the packed training batch of four documents
        _qk("qk_fwd_262k", "qk_fwd", 262144, 4, packed=80),
        # the same batch's gradients
        _qk("qk_bwd_262k", "qk_bwd", 262144, 4, packed=80),
        # an odd length, shared k heads, part of the head rotated in adjacent pairs, 32-bit values
        _qk("qk_bwd_5001", "qk_bwd", 5001, 7, HQ=24, HK=3, dim=96, rot=48, layout="pairs", norm="l2", dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("step", "step", "conv_step", "qk_fwd", "qk_bwd"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    seed = rng.randrange(1 << 20)
    if op == "step":
        H = rng.choice((1, 2, 4, 8, 16))
        HV = H * rng.choice((1, 2, 3, 4))
        kda = rng.randrange(2)
        way = rng.choice(("one", "verify", "ragged"))
        if way == "one":
            c = _step("", _log(rng, 1, max(1, 24000 // HV)), H=H, HV=HV, kda=kda, dtype=dtype, shape_seed=seed)
        elif way == "verify":
            c = _step("", _log(rng, 1, max(1, min(256, 3000 // HV))), 1, rng.randint(2, 8), H=H, HV=HV, kda=kda,
                      dtype=dtype, keep="all", shape_seed=seed)
        else:
            c = _step("", _log(rng, 1, 32), 0, _log(rng, 9, 160), H=H, HV=HV, kda=kda, dtype=dtype, shape_seed=seed)
        c["fresh"] = rng.randint(0, c["N"] // 2)
    elif op == "conv_step":
        C, W = 8 * _log(rng, 16, 1536), rng.randint(2, 4)
        if rng.random() < 0.5:
            c = _conv("", _log(rng, 1, 512), 1, rng.choice((1, 1, 4)), C, W, dtype, shape_seed=seed)
        else:
            c = _conv("", _log(rng, 1, 32), 0, _log(rng, 9, 2048), C, W, dtype, shape_seed=seed)
        c["fresh"] = rng.randint(0, c["N"] // 2)
    else:
        dim = rng.choice((64, 80, 96, 128, 128, 192, 256))
        rot = rng.choice((dim, dim, dim // 2, dim // 4))
        HK = rng.choice((1, 2, 3, 4, 8, 16))
        HQ = HK * rng.choice((1, 2, 4, 8))
        docs = rng.choice((0, 1, 3, 8, 50))
        most = min(262144, int(4e8 / ((HQ + HK) * dim)))
        c = _qk("", op, _log(rng, 1, most), docs, HQ, HK, dim, rot, rng.choice(("half", "pairs")),
                rng.choice(("rms", "rms", "l2", "none")), dtype, rng.choice((0, HQ + 2 * HK)),
                0 if docs else _log(rng, 100, 1000000), rng.choice((1.0, 1.0, 4.0)), seed)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------
def _lengths(case):
    """Tokens of each sequence: a property of the case, not of the inputs' seed."""
    r = np.random.RandomState(case["shape_seed"])
    n = r.randint(case["lo"], case["hi"] + 1, case["N"])
    n[r.randint(case["N"])] = case["hi"]
    return n


def _documents(case):
    """Starts of the packed documents, cu[0] = 0 to cu[docs] = T (some may be empty)."""
    r = np.random.RandomState(case["shape_seed"])
    cuts = np.sort(r.randint(0, case["T"] + 1, case["docs"] - 1))
    return np.concatenate([[0], cuts, [case["T"]]]).astype(np.int32)


def _slots(case, n, seed):
    """(slots, slot_in [N], slot_out [T]) as a scheduler hands them out, in no order; -1: no state, none kept."""
    r = np.random.RandomState(seed % (1 << 31))
    N, T = case["N"], int(n.sum())
    every = case.get("keep") == "all"
    slots = N + (T if every else 0) + 3
    order = r.permutation(slots).astype(np.int32)
    home = order[:N]
    slot_in = home.copy()
    slot_in[r.permutation(N)[:case["fresh"]]] = -1
    slot_out = np.full(T, -1, np.int32)
    last = np.cumsum(n) - 1
    if every:
        slot_out[:] = order[N:N + T]
    else:
        slot_out[last[n > 0]] = home[n > 0]
    return slots, slot_in, slot_out


def _rows(n):
    """For the j-th token of every sequence: (sequences, tokens), the plan by which a plain form walks them together."""
    cu = np.concatenate([[0], np.cumsum(n)])
    plan = []
    for j in range(int(n.max()) if len(n) else 0):
        seqs = np.nonzero(n > j)[0]
        plan.append((torch.from_numpy(seqs).cuda(), torch.from_numpy(cu[seqs] + j).cuda()))
    return plan


def _frequencies(rot, stretch):
    """Radians per position of each rotated pair, and the factor on cos and sin; stretched contexts go by YaRN's
    interpolation by parts (arXiv:2309.00071) from a trained length of 4096."""
    f = BASE ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if stretch == 1.0:
        return f, 1.0
    at = [rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(BASE)) for turns in (32.0, 1.0)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    ramp = np.clip((np.arange(rot // 2) - low) / max(high - low, 0.001), 0, 1)
    return f * (1 - ramp) + f / stretch * ramp, 0.1 * math.log(stretch) + 1


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)

    if case["op"] in ("step", "conv_step"):
        n = _lengths(case)
        T = int(n.sum())
        slots, slot_in, slot_out = _slots(case, n, seed)
        x = dict(T=T, slots=slots, n=n, slot_in_host=slot_in, slot_out_host=slot_out,
                 cu=torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda(),
                 slot_in=torch.from_numpy(slot_in).cuda(), slot_out=torch.from_numpy(slot_out).cuda())
    if case["op"] == "step":
        H, HV = case["H"], case["HV"]
        qkv = normal(T, 2 * H + HV, D).to(dt)   # the convolution's output: q, k and v are views of its rows
        shape = (T, HV, D) if case["kda"] else (T, HV)
        x.update(q=qkv[:, :H], k=qkv[:, H:2 * H], v=qkv[:, 2 * H:],
                 g=torch.nn.functional.logsigmoid(2.0 + 4.0 * uniform(*shape)), beta=torch.sigmoid(normal(T, HV)),
                 states=normal(slots, HV, D, D).mul_(0.5))
    elif case["op"] == "conv_step":
        C, W = case["C"], case["W"]
        x.update(x=normal(T, C).to(dt), w=0.5 * normal(C, W), b=0.1 * normal(C), window=normal(slots, W - 1, C).to(dt))
    else:
        T, HQ, HK, dim = case["T"], case["HQ"], case["HK"], case["dim"]
        if case["packed"]:
            qkv = torch.empty((T, case["packed"], dim), dtype=dt, device="cuda")
            q, k = qkv[:, :HQ], qkv[:, HQ:HQ + HK]
        else:
            q, k = (torch.empty((T, h, dim), dtype=dt, device="cuda") for h in (HQ, HK))
        q.copy_(normal(T, HQ, dim).mul_(0.5 + uniform(dim)))   # channels of unlike size
        k.copy_(normal(T, HK, dim).mul_(0.5 + uniform(dim)))
        f, m = _frequencies(case["rot"], case["stretch"])
        x = dict(q=q, k=k, wq=1 + 0.1 * normal(dim), wk=1 + 0.1 * normal(dim), freq=torch.from_numpy(f).cuda(), m=m,
                 cu=None, pos=None)
        if case["docs"]:
            x["cu"] = torch.from_numpy(_documents(case)).cuda()
        else:
            x["pos"] = torch.randint(0, case["start"] + 1, (T,), generator=gen, device="cuda", dtype=torch.int32)
        if case["op"] == "qk_bwd":
            x.update(gq=normal(T, HQ, dim).to(dt), gk=normal(T, HK, dim).to(dt))
    return x


def prepare(case, seed):
    s = _inputs(case, seed)
    s.update(case=case, dt=TYPES[case["dtype"]])
    if case["op"] == "step":
        s["plan"] = _rows(s["n"])
        s["o"] = torch.empty((s["T"], case["HV"], D), dtype=s["dt"], device="cuda")
    elif case["op"] == "conv_step":
        s["y"] = torch.empty_like(s["x"])
    elif case["op"] == "qk_fwd":
        s["yq"], s["yk"] = (torch.empty(s[n].shape, dtype=s["dt"], device="cuda") for n in ("q", "k"))
    if case["op"] == "qk_bwd":
        s["dwq"], s["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
        if case["packed"]:   # the gradients go where the projection's backward reads them
            rows = torch.empty((case["T"], case["packed"], case["dim"]), dtype=s["dt"], device="cuda")
            s["dq"], s["dk"] = rows[:, :case["HQ"]], rows[:, case["HQ"]:case["HQ"] + case["HK"]]
        else:
            s["dq"], s["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    s["err"] = torch.zeros(64, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _plain_step(s):
    c = s["case"]
    G = c["HV"] // c["H"]
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + EPS) * D ** -0.5
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + EPS)
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    a = torch.exp(s["g"])[..., None] if c["kda"] else torch.exp(s["g"])[..., None, None]
    pool, slot_in, slot_out = s["states"], s["slot_in"].long(), s["slot_out"].long()
    S = pool[slot_in.clamp(min=0)]
    S.mul_((slot_in >= 0)[:, None, None, None])
    # the rule is a recurrence: this loop walks the tokens of all sequences together
    for seqs, t in s["plan"]:
        whole = len(seqs) == len(S)
        Z = (S if whole else S[seqs]).mul_(a[t])
        kt = k[t][..., None]
        d = s["beta"][t][..., None] * (v[t] - (Z * kt).sum(-2))
        Z += kt * d[..., None, :]
        s["o"][t] = (Z * q[t][..., None]).sum(-2).to(s["dt"])
        if not whole:
            S[seqs] = Z
        if c["keep"] == "all":
            pool[slot_out[t]] = Z
    if c["keep"] != "all":
        some = s["cu"][1:] > s["cu"][:-1]
        last = (s["cu"][1:].long() - 1)[some]
        pool[slot_out[last]] = S[some]
    return {"o": s["o"], "states": pool}


def _plain_conv_step(s):
    c = s["case"]
    W, T, N = c["W"], s["T"], c["N"]
    cu = s["cu"].long()
    seq = torch.repeat_interleave(torch.arange(N, device="cuda"), cu[1:] - cu[:-1], output_size=T)
    # every row with what went before it: the sequences' windows lie in front of the tokens
    slot = s["slot_in"].long()
    old = s["window"][slot.clamp(min=0)].float() * (slot >= 0)[:, None, None]
    rows = torch.cat([old.reshape(N * (W - 1), -1), s["x"].float()])
    back = torch.arange(W - 1, -1, -1, device="cuda")
    at = torch.arange(T, device="cuda")[:, None] - back
    first = cu[:-1][seq][:, None]
    at = torch.where(at >= first, N * (W - 1) + at, seq[:, None] * (W - 1) + (W - 1) + at - first)
    z = (rows[at] * s["w"].t()).sum(1) + s["b"]
    y = (z / (1 + torch.exp(-z))).to(s["dt"])
    some = cu[1:] > cu[:-1]
    last = (cu[1:] - 1)[some]
    s["window"][s["slot_out"].long()[last]] = rows[at[last][:, 1:]].to(s["dt"])
    return {"y": y, "window": s["window"]}


def _turn(s):
    """cos and sin [T, 1, rot / 2] of each token's angles, in 32 bits; turns are counted in whole parts of 2^-32, so that
    far positions keep their angle."""
    if s["pos"] is None:
        T = s["q"].shape[0]
        cu = s["cu"].long()
        at = torch.arange(T, device="cuda")
        pos = at - cu[torch.searchsorted(cu, at, right=True) - 1]
    else:
        pos = s["pos"].long()
    part = torch.round(s["freq"] / (2 * math.pi) * 2.0 ** 52).long()
    part = (pos[:, None] * part) & ((1 << 52) - 1)
    angle = (part >> 20).float() * (2 * math.pi * 2.0 ** -32)
    return (torch.cos(angle) * s["m"])[:, None], (torch.sin(angle) * s["m"])[:, None]


def _pairs(c, x):
    """The two halves of the rotated part, and the rest."""
    r = c["rot"]
    return (x[..., :r // 2], x[..., r // 2:r], x[..., r:]) if c["layout"] == "half" else (x[..., 0:r:2], x[..., 1:r:2], x[..., r:])


def _joined(c, a, b, rest):
    pair = torch.cat([a, b], -1) if c["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([pair, rest], -1)


def _inverse_norm(c, x):
    ss = (x * x).sum(-1, keepdim=True)
    if c["norm"] == "none":
        return torch.ones_like(ss)
    return torch.rsqrt(ss / c["dim"] + EPS) if c["norm"] == "rms" else torch.rsqrt(ss + EPS)


def _plain_qk_fwd(s, x, w, cos, sin):
    c = s["case"]
    x = x.float()
    a, b, rest = _pairs(c, x * _inverse_norm(c, x) * w)
    return _joined(c, a * cos - b * sin, b * cos + a * sin, rest).to(s["dt"])


def _plain_qk_bwd(s, x, w, g, cos, sin):
    c = s["case"]
    a, b, rest = _pairs(c, g.float())
    g = _joined(c, a * cos + b * sin, b * cos - a * sin, rest)
    x = x.float()
    r = _inverse_norm(c, x)
    xhat = x * r
    dw = (g * xhat).sum((0, 1))
    g = g * w
    if c["norm"] != "none":
        part = (g * xhat).sum(-1, keepdim=True)
        g = g - xhat * (part / c["dim"] if c["norm"] == "rms" else part)
    return (g * r).to(s["dt"]), dw


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _problem(s):
    """The framework's description of the case, which a user's program keeps; made at the first pass of a state."""
    if "prob" not in s:
        import linear_attention_gdn_gb300 as gdn
        c = s["case"]
        if c["op"] == "step":
            s["prob"] = gdn.step_problem(s["T"], c["N"], c["H"], c["HV"], s["slots"], scale=D ** -0.5, l2norm=True, dtype=s["dt"],
                                         strides=tuple(s[n].stride(0) for n in ("q", "k", "v")))
        elif c["op"] == "conv_step":
            s["prob"] = gdn.conv_step_problem(s["T"], c["N"], c["C"], s["slots"], W=c["W"], dtype=s["dt"])
        else:
            s["prob"] = gdn.qk_problem(
                c["T"], c["HQ"], c["HK"], D=c["dim"], rot=c["rot"], N=c["docs"],
                layout=gdn.ROPE_HALF if c["layout"] == "half" else gdn.ROPE_PAIRS,
                norm={"none": gdn.NORM_NONE, "rms": gdn.NORM_RMS, "l2": gdn.NORM_L2}[c["norm"]], eps=EPS, mscale=s["m"],
                dtype=s["dt"], q_strides=s["q"].stride()[:2], k_strides=s["k"].stride()[:2])
            if c["op"] == "qk_bwd":
                s["ws"] = torch.empty(gdn.gdn_qk_workspace_bytes(s["prob"]), dtype=torch.uint8, device="cuda")
        s["gdn"] = gdn
    return s["gdn"], s["prob"]


def run(s):
    op = s["case"]["op"]
    if own:
        gdn, prob = _problem(s)
        cu = None if s["case"].get("hi") == 1 else s["cu"]   # one token each: no starts are needed
        if op == "step":
            step = gdn.gdn_kda_step if s["case"]["kda"] else gdn.gdn_step
            step(prob, s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["o"], s["err"], cu_seqlens_dev=cu,
                 slot_in=s["slot_in"], slot_out=s["slot_out"])
            return {"o": s["o"], "states": s["states"]}
        if op == "conv_step":
            gdn.gdn_conv1d_step(prob, s["x"], s["w"], s["b"], s["window"], s["y"], s["err"], cu_seqlens_dev=cu,
                                slot_in=s["slot_in"], slot_out=s["slot_out"])
            return {"y": s["y"], "window": s["window"]}
        if op == "qk_fwd":
            gdn.gdn_qk_norm_rope_fwd(prob, s["q"], s["k"], s["wq"], s["wk"], s["freq"], s["pos"], s["cu"], s["yq"], s["yk"])
            return {"q": s["yq"], "k": s["yk"]}
        gdn.gdn_qk_norm_rope_bwd(prob, s["q"], s["k"], s["wq"], s["wk"], s["freq"], s["pos"], s["cu"], s["gq"], s["gk"],
                                 s["dq"], s["dk"], s["dwq"], s["dwk"], s["ws"])
        return {"dq": s["dq"], "dk": s["dk"], "dwq": s["dwq"], "dwk": s["dwk"]}
    if op == "step":
        return _plain_step(s)
    if op == "conv_step":
        return _plain_conv_step(s)
    cos, sin = _turn(s)
    if op == "qk_fwd":
        return {"q": _plain_qk_fwd(s, s["q"], s["wq"], cos, sin), "k": _plain_qk_fwd(s, s["k"], s["wk"], cos, sin)}
    dq, dwq = _plain_qk_bwd(s, s["q"], s["wq"], s["gq"], cos, sin)
    dk, dwk = _plain_qk_bwd(s, s["k"], s["wk"], s["gk"], cos, sin)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------
def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "step":
        n = _lengths(case)
        T, live, HV, H = int(n.sum()), int((n > 0).sum()), case["HV"], case["H"]
        _, slot_in, slot_out = _slots(case, n, 0)
        reads = int(((slot_in >= 0) & (n > 0)).sum())
        writes = int((slot_out >= 0).sum())
        state = HV * D * D * 4
        gate = HV * 4 * (D if case["kda"] else 1)
        return {"bytes": (reads + writes) * state + T * ((2 * H + 2 * HV) * D * e + gate + HV * 4 + 4) + 8 * live,
                "flops": T * HV * D * D * 7}
    if case["op"] == "conv_step":
        n = _lengths(case)
        T, C, W = int(n.sum()), case["C"], case["W"]
        _, slot_in, slot_out = _slots(case, n, 0)
        rows = (int(((slot_in >= 0) & (n > 0)).sum()) + int((slot_out >= 0).sum())) * (W - 1)
        return {"bytes": (2 * T + rows) * C * e + C * (W + 1) * 4 + 4 * T, "flops": T * C * (2 * W + 5)}
    rows = case["T"] * (case["HQ"] + case["HK"])
    back = case["op"] == "qk_bwd"
    small = 2 * case["dim"] * 4 * (2 if back else 1) + case["rot"] // 2 * 8 + 4 * (case["docs"] or case["T"])
    return {"bytes": rows * case["dim"] * e * (3 if back else 2) + small, "flops": rows * case["dim"] * (14 if back else 7)}


def _exact_step(c, x):
    G = c["HV"] // c["H"]
    o = torch.zeros((x["T"], c["HV"], D), dtype=torch.float64, device="cuda")
    pool = x["states"].double()
    first = 0
    begin = pool.clone()
    spread = lambda h: h.double().repeat_interleave(G, 0)  # noqa: E731
    groups = {}
    for i, m in enumerate(x["n"]):
        groups.setdefault(int(m), []).append((i, first))
        first += int(m)
    for m, members in groups.items():   # sequences of one length go together
        idx = [i for i, _ in members]
        at = torch.tensor([f for _, f in members], device="cuda")
        S = torch.stack([begin[x["slot_in_host"][i]] if x["slot_in_host"][i] >= 0 else torch.zeros_like(begin[0]) for i in idx])
        for j in range(m):
            t = at + j
            q, k, v = (x[n][t].double() for n in ("q", "k", "v"))
            q, k = (torch.stack([spread(h) for h in y / torch.sqrt(torch.einsum("nhd,nhd->nh", y, y)[..., None] + EPS)]) for y in (q, k))
            decay = torch.exp(x["g"][t].double())
            S = torch.einsum("nhij,nhi->nhij", S, decay) if c["kda"] else torch.einsum("nhij,nh->nhij", S, decay)
            miss = v - torch.einsum("nhij,nhi->nhj", S, k)
            S = S + torch.einsum("nhi,nhj,nh->nhij", k, miss, x["beta"][t].double())
            o[t] = torch.einsum("nhij,nhi->nhj", S, q) / math.sqrt(D)
            for r, tok in enumerate(t.tolist()):
                if x["slot_out_host"][tok] >= 0:
                    pool[x["slot_out_host"][tok]] = S[r]
    return {"o": o, "states": pool}


def _exact_conv_step(c, x):
    W, first = c["W"], 0
    y = torch.zeros((x["T"], c["C"]), dtype=torch.float64, device="cuda")
    window, w = x["window"].double(), x["w"].double()
    new = window.clone()
    for i, m in enumerate(x["n"].tolist()):
        slot = x["slot_in_host"][i]
        old = window[slot] if slot >= 0 else torch.zeros_like(window[0])
        line = torch.cat([old, x["x"][first:first + m].double()])
        z = x["b"].double() + sum(w[:, j] * line[j:j + m] for j in range(W))
        y[first:first + m] = z * torch.sigmoid(z)
        for j in range(m):
            if (slot := x["slot_out_host"][first + j]) >= 0:
                new[slot] = line[j + 1:j + W]
        first += m
    return {"y": y, "window": new}


def _exact_qk(c, x):
    T, r = c["T"], c["rot"]
    if x["pos"] is None:
        starts = _documents(c)
        pos = np.concatenate([np.arange(n) for n in np.diff(starts)])
    else:
        pos = x["pos"].cpu().numpy()
    angle = torch.from_numpy(pos.astype(np.float64)).cuda()[:, None] * x["freq"]
    turn = torch.polar(torch.full_like(angle, x["m"]), angle)[:, None]
    out = {}

    def rotated(y, by):
        pair = y[..., :r].reshape(*y.shape[:-1], 2, r // 2).transpose(-1, -2) if c["layout"] == "half" else y[..., :r].reshape(*y.shape[:-1], r // 2, 2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * by)
        z = z.transpose(-1, -2) if c["layout"] == "half" else z
        return torch.cat([z.reshape(*y.shape[:-1], r), y[..., r:]], -1)

    for n in ("q", "k"):
        w, parts, dw = x["w" + n].double(), [], 0
        H, dim = x[n].shape[1:]
        step = max(1, (1 << 27) // (H * dim))
        for a in range(0, T, step):
            y = x[n][a:a + step].double()
            norm = torch.linalg.vector_norm(y, dim=-1, keepdim=True)
            inv = {"none": torch.ones_like(norm), "rms": (norm ** 2 / dim + EPS) ** -0.5, "l2": (norm ** 2 + EPS) ** -0.5}[c["norm"]]
            if c["op"] == "qk_fwd":
                parts.append(rotated(y * inv * w, turn[a:a + step]))
                continue
            g = rotated(x["g" + n][a:a + step].double(), turn[a:a + step].conj())
            dw = dw + torch.einsum("thd,thd->d", g, y * inv)
            g = g * w
            share = {"none": 0.0, "rms": 1.0 / dim, "l2": 1.0}[c["norm"]]
            parts.append((g * inv - y * inv ** 3 * share * torch.einsum("thd,thd->th", g, y)[..., None]))
        if c["op"] == "qk_fwd":
            out[n] = torch.cat(parts)
        else:
            out["d" + n], out["dw" + n] = torch.cat(parts), dw
    return out


def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "step":
        return _exact_step(case, x)
    if case["op"] == "conv_step":
        return _exact_conv_step(case, x)
    return _exact_qk(case, x)
