"""Measured cases of the operators beside the gated delta rule:

  la_fwd, la_bwd   linear attention with a fixed decay per head over packed documents, and its gradients
  la_step          its recurrent form over a pool of states
  norm_fwd         the root-mean-square norm with the residual's addition, with an output in 8 bits where wanted
  norm_bwd         its gradients
  tables           the tables of a generation step from the requests' lengths, blocks handed out on the way

`run` computes a case in its plain form, or, where `own` is set, by the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

D = 128            # head size of the linear attention
EPS = 1e-6         # under the root of the norm
CHUNK = 64         # tokens that the plain form of the attention takes at a time
E4M3 = 448.0       # the largest value of the 8-bit type
LEAST = 2.0 ** -100  # the least scale
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _la(name, op, N, lo, hi, H=16, HV=48, states="both", packed=1, shape_seed=1):
    """N documents of lo..hi tokens. states: "both": each goes on from a state and leaves one (backward: their
    gradients); "out": none to start from; "none". packed: q, k and v are views of the convolution's rows."""
    return dict(name=name, op=op, N=N, lo=lo, hi=hi, H=H, HV=HV, states=states, packed=packed, shape_seed=shape_seed)


def _step(name, N, lo=1, hi=1, H=16, HV=48, dtype="bf16", keep="last", fresh=0, shape_seed=1):
    """N sequences of lo..hi tokens. keep "last": the state goes back to its own slot; "all": the state after every
    token goes to a slot of that token. fresh: how many sequences start from no state."""
    return dict(name=name, op="la_step", N=N, lo=lo, hi=hi, H=H, HV=HV, dtype=dtype, keep=keep, fresh=fresh,
                shape_seed=shape_seed)


def _norm(name, op, T, C, dtype="bf16", residual=1, plain=1, group=-1):
    """T rows of C values. residual: x is added to a stream that goes on (backward: a gradient arrives along it). plain:
    the norm is wanted in `dtype`. group: it is wanted in 8 bits, one scale to so many values (0: to a row; -1: not)."""
    return dict(name=name, op=op, T=T, C=C, dtype=dtype, residual=residual, plain=plain, group=group)


def _tables(name, N, lo, hi, block=64, context=4096, done=0, short=0, shape_seed=1):
    """N requests that take lo..hi new tokens, with up to `context` before them, a state kept every `block` tokens.
    done: how many have ended and give their blocks back. short: the tables are too small for the last ones."""
    return dict(name=name, op="tables", N=N, lo=lo, hi=hi, block=block, context=context, done=done, short=short,
                shape_seed=shape_seed)


def listed():
    return [
        # a short prompt in one layer: nothing but latency
        _la("la_fwd_200", "la_fwd", 1, 200, 200, states="out"),
        # pieces of twelve prompts that go on from their states
        _la("la_fwd_ragged", "la_fwd", 12, 1, 4096, shape_seed=2),
        # one long prompt, a head of q and k to each of v
        _la("la_fwd_32k", "la_fwd", 1, 32768, 32768, H=16, HV=16, states="out", packed=0),
        # a ragged training pack with an empty document, states at its ends
        _la("la_bwd_ragged", "la_bwd", 7, 0, 3001, H=8, HV=24, packed=0, shape_seed=3),
        # the packed training batch of documents of 8,192 tokens
        _la("la_bwd_65k", "la_bwd", 8, 8192, 8192, states="none"),
        # one user's next token in one layer
        _step("la_step_1", 1),
        # a serving batch with drafts of 1 to 4 tokens to verify, three requests just begun
        _step("la_step_verify", 96, lo=1, hi=4, H=32, HV=32, dtype="fp16", keep="all", fresh=3),
        # a batch's single tokens in front of an 8-bit projection
        _norm("norm_fwd_64", "norm_fwd", 64, 4096, plain=0, group=128),
        # the packed batch's rows, the norm in both types
        _norm("norm_fwd_65k", "norm_fwd", 65536, 4096, group=0),
        # and its gradients
        _norm("norm_bwd_65k", "norm_bwd", 65536, 4096),
        # a decoding batch: a token each
        _tables("tables_64", 64, 1, 1),
        # a large batch of prompts' pieces and single tokens, some requests at their end, the pool nearly empty
        _tables("tables_2000", 2000, 0, 64, context=32768, done=40, short=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("la_fwd", "la_fwd", "la_bwd", "la_step", "norm_fwd", "norm_bwd", "tables"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    seed = rng.randrange(1 << 20)
    if op in ("la_fwd", "la_bwd", "la_step"):
        H = rng.choice((1, 2, 4, 8, 16, 32))
        HV = min(64, H * rng.choice((1, 1, 2, 3, 4, 8)))
        HV -= HV % H
    if op in ("la_fwd", "la_bwd"):
        N = _log(rng, 1, 64)
        most = max(1, (65536 if op == "la_fwd" else 40000) * 24 // (N * max(HV, 2 * H)))
        hi = _log(rng, 1, min(most, 32768))
        lo = rng.choice((0, 1, hi // 2 + 1, hi))
        c = _la("", op, N, min(lo, hi), hi, H, HV, rng.choice(("both", "out", "none")), rng.randrange(2), seed)
    elif op == "la_step":
        hi = rng.choice((1, 1, 1, rng.randint(2, 8), rng.randint(9, 40)))
        N = _log(rng, 1, max(1, 12000 // (HV * (1 if hi == 1 else 2 if hi > 8 else 6))))
        lo = 1 if hi == 1 else rng.choice((0, 1))
        c = _step("", N, lo, hi, H, HV, dtype, "all" if 1 < hi <= 8 and rng.random() < 0.7 else "last",
                  rng.randint(0, N // 2), seed)
    elif op in ("norm_fwd", "norm_bwd"):
        C = rng.choice((rng.randint(1, 40), 8 * _log(rng, 8, 2048), 128 * _log(rng, 1, 128)))
        T = _log(rng, 1, min(65536, int(2.5e8 / C)))
        group = rng.choice((-1, 0, 32, 64, 128)) if op == "norm_fwd" else -1
        if group > 0 and C % group:
            group = 0
        c = _norm("", op, T, C, dtype, rng.randrange(2), 1 if group < 0 else rng.randrange(2), group)
    else:
        N = _log(rng, 1, 4096)
        hi = rng.choice((1, 1, rng.randint(2, 8), _log(rng, 9, 2048)))
        hi = max(1, min(hi, 131072 // N))
        c = _tables("", N, rng.choice((0, 1)), hi, rng.choice((1, 16, 64, 100, 256)), _log(rng, 1, 32768),
                    rng.randint(0, N // 4), rng.randrange(2), seed)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------
def _lengths(case):
    """Tokens of each document or sequence: a property of the case, not of the inputs' seed."""
    r = np.random.RandomState(case["shape_seed"])
    n = r.randint(case["lo"], case["hi"] + 1, case["N"])
    n[r.randint(case["N"])] = case["hi"]
    if case["op"] == "la_bwd" and case["N"] > 1 and case["lo"] == 0:
        n[(int(np.argmax(n)) + 1) % case["N"]] = 0
    return n


def _slots(case, n, seed):
    """(slots, slot_in [N], slot_out [T]) as a scheduler hands them out, in no order; -1: no state, none kept."""
    r = np.random.RandomState(seed % (1 << 31))
    N, T = case["N"], int(n.sum())
    every = case["keep"] == "all"
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


def _requests(case, seed):
    """A scheduler's books on the host: new tokens and tokens before them, which are the case's, and the blocks' slots and
    the free ones, in the inputs' order."""
    r = np.random.RandomState(case["shape_seed"])
    N, B = case["N"], case["block"]
    length = r.randint(case["lo"], case["hi"] + 1, N)
    context = np.floor(np.exp(r.uniform(0, math.log(case["context"] + 1), N))).astype(np.int64) - 1
    length[r.permutation(N)[:case["done"]]] = -1
    held = -(-context // B)
    after = -(-(context + np.maximum(length, 0)) // B)
    most = -(-(case["context"] + case["hi"]) // B) + 1
    new = np.where(length >= 0, after - held, 0)
    back = int(held[length < 0].sum())
    need, T = int(new.sum()), int(np.maximum(length, 0).sum())
    free = max(0, need - back + 5)
    if case["short"]:   # about the last tenth of the requests has to wait
        free = max(0, int(0.9 * need) - back)
    slots = int(held.sum()) + free + back
    order = np.random.RandomState(seed % (1 << 31)).permutation(slots).astype(np.int32)
    table = np.full((N, most), -1, np.int32)
    at = 0
    for i in range(N):
        table[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
    stack = np.full(slots, -1, np.int32)
    stack[:free] = order[at:at + free]
    return dict(T=max(1, T + 7), most=most, slots=slots, free=free, length=length.astype(np.int32), table=table,
                context=context.astype(np.int32), stack=stack)


def _grid(n):
    """The chunks of all documents, by place in their document: (tokens [NC, CHUNK], which of them there are, and for
    the j-th chunk of every document the documents and the chunks)."""
    cu = np.concatenate([[0], np.cumsum(n)])
    per = -(-n // CHUNK)
    first = np.concatenate([[0], np.cumsum(per)])
    doc = np.repeat(np.arange(len(n)), per)
    j = np.arange(first[-1]) - first[doc]
    tok = (cu[doc] + j * CHUNK)[:, None] + np.arange(CHUNK)
    real = tok < cu[doc + 1][:, None]
    walk = []
    for i in range(int(per.max()) if len(per) else 0):
        d = np.nonzero(per > i)[0]
        walk.append((torch.from_numpy(d).cuda(), torch.from_numpy(first[d] + i).cuda()))
    return dict(tok=torch.from_numpy(np.where(real, tok, 0)).cuda(), real=torch.from_numpy(real).cuda(), walk=walk)


def _rows(n):
    """For the j-th token of every sequence: (sequences, tokens)."""
    cu = np.concatenate([[0], np.cumsum(n)])
    plan = []
    for j in range(int(n.max()) if len(n) else 0):
        seqs = np.nonzero(n > j)[0]
        plan.append((torch.from_numpy(seqs).cuda(), torch.from_numpy(cu[seqs] + j).cuda()))
    return plan


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    if op == "tables":
        x = _requests(case, seed)
        x.update(lengths=torch.from_numpy(x["length"]).cuda(), before=torch.from_numpy(x["context"]).cuda(),
                 blocks=torch.from_numpy(x["table"]).cuda(), free_list=torch.from_numpy(x["stack"]).cuda(),
                 free_count=torch.tensor([x["free"]], dtype=torch.int32, device="cuda"))
        return x
    if op in ("norm_fwd", "norm_bwd"):
        T, C, dt = case["T"], case["C"], TYPES[case["dtype"]]
        x = dict(w=1 + 0.1 * normal(C))
        if op == "norm_fwd":
            x["x"] = normal(T, C).to(dt)
            x["r"] = (3 * normal(T, C)).to(dt) if case["residual"] else None
        else:
            x["h"], x["dy"] = (3 * normal(T, C)).to(dt), normal(T, C).to(dt)
            x["along"] = normal(T, C).to(dt) if case["residual"] else None
        return x
    H, HV, N = case["H"], case["HV"], case["N"]
    n = _lengths(case)
    T = int(n.sum())
    dt = TYPES[case.get("dtype", "bf16")]
    if case.get("packed", 1):
        qkv = torch.empty((T, 2 * H + HV, D), dtype=dt, device="cuda")
        q, k, v = qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:]
    else:
        q, k, v = (torch.empty((T, h, D), dtype=dt, device="cuda") for h in (H, H, HV))
    q.copy_(normal(T, H, D))
    k.copy_(normal(T, H, D).mul_(0.3))
    v.copy_(normal(T, HV, D))
    # decays as such layers fix them: from one head to the next by a constant factor, 0.5 to 1 - 1 / 512 a token
    g = torch.log1p(-torch.pow(2.0, -1 - 8 * torch.arange(HV, dtype=torch.float64) / max(HV - 1, 1))).float().cuda()
    x = dict(n=n, T=T, q=q, k=k, v=v, g=g, cu_host=np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
    x["cu"] = torch.from_numpy(x["cu_host"]).cuda()
    if op == "la_step":
        slots, slot_in, slot_out = _slots(case, n, seed)
        x.update(slots=slots, slot_in_host=slot_in, slot_out_host=slot_out, slot_in=torch.from_numpy(slot_in).cuda(),
                 slot_out=torch.from_numpy(slot_out).cuda(), states=normal(slots, HV, D, D))
    else:
        both = case["states"] == "both"
        x["s_in"] = normal(N, HV, D, D) if both else None
        if op == "la_bwd":
            x["do"] = normal(T, HV, D).to(dt)
            x["ds_out"] = normal(N, HV, D, D).mul_(0.3) if case["states"] != "none" else None
    return x


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"], op = case, case["op"]
    s["err"] = torch.zeros(64, dtype=torch.int32, device="cuda")
    if op == "tables":
        N, T = case["N"], s["T"]
        new = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        s.update(after=new(N), left=new(1), cu=new(N + 1), positions=new(T), slot_in=new(N), slot_out=new(T))
    elif op == "norm_fwd":
        T, C, dt = case["T"], case["C"], TYPES[case["dtype"]]
        s["h"] = torch.empty((T, C), dtype=dt, device="cuda") if case["residual"] else None
        s["y"] = torch.empty((T, C), dtype=dt, device="cuda") if case["plain"] else None
        s["y8"] = s["scales"] = None
        if case["group"] >= 0:
            s["y8"] = torch.empty((T, C), dtype=torch.float8_e4m3fn, device="cuda")
            s["scales"] = torch.empty((T, C // (case["group"] or C)), dtype=torch.float32, device="cuda")
    elif op == "norm_bwd":
        s["dx"], s["dw"] = torch.empty_like(s["h"]), torch.empty_like(s["w"])
    elif op == "la_step":
        s["plan"] = _rows(s["n"])
        s["o"] = torch.empty((s["T"], case["HV"], D), dtype=s["q"].dtype, device="cuda")
    else:
        N, H, HV, T = case["N"], case["H"], case["HV"], s["T"]
        s["grid"] = _grid(s["n"])
        pool = lambda want: torch.empty((N, HV, D, D), dtype=torch.float32, device="cuda") if want else None  # noqa: E731
        if op == "la_fwd":
            s["o"] = torch.empty((T, HV, D), dtype=torch.bfloat16, device="cuda")
            s["s_out"] = pool(case["states"] != "none")
        else:
            if case["packed"]:   # the gradients go where the convolution's backward reads them
                rows = torch.empty((T, 2 * H + HV, D), dtype=torch.bfloat16, device="cuda")
                s["dq"], s["dk"], s["dv"] = rows[:, :H], rows[:, H:2 * H], rows[:, 2 * H:]
            else:
                s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[m]) for m in "qkv")
            s["ds_in"] = pool(case["states"] == "both")
    return s


# ---------------------------------------------------------------------------
# the plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _chunks(s, x, groups=1):
    """[NC, heads, CHUNK, D] in 32 bits, zeros past a document's end; each head `groups` times."""
    y = x[s["grid"]["tok"]].float() * s["grid"]["real"][..., None, None]
    return y.transpose(1, 2).repeat_interleave(groups, 1)


def _tokens(s, y):
    """Back from chunks to [T, heads, D], rounded."""
    return y.transpose(1, 2)[s["grid"]["real"]].to(torch.bfloat16)


def _states(s, add, first, back):
    """The state before each chunk (back: the gradient of the state after it) and what the last leaves, from what each
    chunk adds. The rule is a recurrence: this loop walks the chunks of all documents together."""
    c, grid = s["case"], s["grid"]
    count = grid["real"].sum(1).float()
    whole = torch.exp(s["g"] * count[:, None])[..., None, None]
    S = torch.zeros((c["N"], c["HV"], D, D), device="cuda") if first is None else first.clone()
    at = torch.empty_like(add)
    for docs, chunks in (reversed(grid["walk"]) if back else grid["walk"]):
        at[chunks] = S[docs]
        S[docs] = S[docs] * whole[chunks] + add[chunks]
    return at, S


def _powers(s):
    """Decays inside a chunk: from token c to r [HV, CHUNK, CHUNK], to r from the state before [HV, CHUNK, 1], and from
    c to the chunk's end [NC, HV, CHUNK, 1]."""
    i = torch.arange(CHUNK, device="cuda")
    apart = i[:, None] - i
    inside = torch.exp(s["g"][:, None, None] * apart.clamp(min=0)) * (apart >= 0)
    before = torch.exp(s["g"][:, None] * (i + 1))[..., None]
    left = (s["grid"]["real"].sum(1)[:, None] - 1 - i).clamp(min=0)
    return inside, before, torch.exp(s["g"][:, None] * left[:, None, :])[..., None]


def _plain_la_fwd(s):
    c, scale = s["case"], D ** -0.5
    G = c["HV"] // c["H"]
    q, k, v = _chunks(s, s["q"], G), _chunks(s, s["k"], G), _chunks(s, s["v"])
    inside, before, after = _powers(s)
    S, last = _states(s, (k * after).transpose(-1, -2) @ v, s["s_in"], False)
    o = ((q @ k.transpose(-1, -2)) * inside) @ v + before * (q @ S)
    s["o"].copy_(_tokens(s, scale * o))
    if s["s_out"] is not None:
        s["s_out"].copy_(last)
    return _la_outputs(s)


def _plain_la_bwd(s):
    c, scale = s["case"], D ** -0.5
    H, G = c["H"], c["HV"] // c["H"]
    q, k, v, do = _chunks(s, s["q"], G), _chunks(s, s["k"], G), _chunks(s, s["v"]), scale * _chunks(s, s["do"])
    inside, before, after = _powers(s)
    S, _ = _states(s, (k * after).transpose(-1, -2) @ v, s["s_in"], False)
    W, first = _states(s, (q * before).transpose(-1, -2) @ do, s["ds_out"], True)
    A = ((q @ k.transpose(-1, -2)) * inside).transpose(-1, -2)
    B = (do @ v.transpose(-1, -2)) * inside
    dv = A @ do + after * (k @ W)
    dq = B @ k + before * (do @ S.transpose(-1, -2))
    dk = B.transpose(-1, -2) @ q + after * (v @ W.transpose(-1, -2))
    s["dv"].copy_(_tokens(s, dv))
    for name, y in (("dq", dq), ("dk", dk)):
        s[name].copy_(_tokens(s, y.unflatten(1, (H, G)).sum(2)))
    if s["ds_in"] is not None:
        s["ds_in"].copy_(first)
    return _la_outputs(s)


def _plain_la_step(s):
    c = s["case"]
    G = c["HV"] // c["H"]
    q, k, v = (s[m].float() for m in "qkv")
    q, k = (q * D ** -0.5).repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    a = torch.exp(s["g"])[:, None, None]
    pool, slot_in, slot_out = s["states"], s["slot_in"].long(), s["slot_out"].long()
    S = pool[slot_in.clamp(min=0)]
    S.mul_((slot_in >= 0)[:, None, None, None])
    # the rule is a recurrence: this loop walks the tokens of all sequences together
    for seqs, t in s["plan"]:
        whole = len(seqs) == len(S)
        Z = (S if whole else S[seqs]).mul_(a)
        Z += k[t][..., None] * v[t][..., None, :]
        s["o"][t] = (Z * q[t][..., None]).sum(-2).to(s["o"].dtype)
        if not whole:
            S[seqs] = Z
        if c["keep"] == "all":
            pool[slot_out[t]] = Z
    if c["keep"] != "all":
        some = s["cu"][1:] > s["cu"][:-1]
        pool[slot_out[(s["cu"][1:].long() - 1)[some]]] = S[some]
    return {"o": s["o"], "states": pool}


def _plain_norm_fwd(s):
    c = s["case"]
    h = s["x"]
    if s["r"] is not None:
        s["h"].copy_(s["x"].float() + s["r"].float())
        h = s["h"]
    h = h.float()
    z = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
    if s["y"] is not None:
        s["y"].copy_(z)
    if s["y8"] is not None:
        z = z.unflatten(-1, (-1, c["group"] or c["C"]))
        most = z.abs().amax(-1, keepdim=True).clamp(min=LEAST * E4M3)
        s["scales"].copy_((most / E4M3)[..., 0])
        s["y8"].copy_((z * (E4M3 / most)).flatten(-2).to(torch.float8_e4m3fn))
    return _norm_outputs(s)


def _plain_norm_bwd(s):
    h, g = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    xhat = h * r
    s["dw"].copy_((g * xhat).sum(0))
    g = g * s["w"]
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["along"] is not None:
        dx = dx + s["along"].float()
    s["dx"].copy_(dx)
    return {"dx": s["dx"], "dw": s["dw"]}


def _plain_tables(s):
    c, T = s["case"], s["T"]
    B, N = c["block"], c["N"]
    length, context = s["lengths"].long(), s["before"].long()
    held = (context + B - 1) // B
    done = length < 0
    # blocks of ended requests come back, in order, on top of the free ones
    count, back = s["free_count"].long(), torch.where(done, held, 0)
    total = s["blocks"].shape[1]
    given = (torch.arange(total, device="cuda") < back[:, None])
    spot = (torch.cumsum(back, 0) - back)[:, None] + torch.arange(total, device="cuda") + count
    s["free_list"][spot[given]] = s["blocks"][given]
    count = count + back.sum()
    # the requests that fit, in order
    want = length.clamp(min=0)
    new = torch.where(done, 0, (context + want + B - 1) // B - held)
    fits = (torch.cumsum(want, 0) <= T) & (torch.cumsum(new, 0) <= count)
    want, new = want * fits, new * fits
    # new blocks from the top of the free ones
    j = torch.arange(total, device="cuda")
    taken = (j >= held[:, None]) & (j < (held + new)[:, None])
    rank = (torch.cumsum(new, 0) - new)[:, None] + j - held[:, None]
    s["blocks"][taken] = s["free_list"][(count - 1 - rank)[taken]]
    s["left"].copy_(count - new.sum())
    s["after"].copy_(torch.where(done, 0, context + want))
    s["cu"][0] = 0
    s["cu"][1:] = torch.cumsum(want, 0)
    start = ((context - 1) // B).clamp(min=0)
    s["slot_in"].copy_(torch.where(done | (context == 0), -1, torch.gather(s["blocks"], 1, start[:, None])[:, 0]))
    # tokens
    cu, t = s["cu"].long(), torch.arange(T, device="cuda")
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=N - 1)
    pos = context[seq] + t - cu[seq]
    inside = t < cu[N]
    keep = inside & (((pos + 1) % B == 0) | (t == cu[seq + 1] - 1))
    s["positions"].copy_(torch.where(inside, pos, 0))
    s["slot_out"].copy_(torch.where(keep, s["blocks"][seq, (pos // B).clamp(max=total - 1)], -1))
    return _table_outputs(s)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _la_outputs(s):
    names = ("o", "s_out") if s["case"]["op"] == "la_fwd" else ("dq", "dk", "dv", "ds_in")
    return {m: s[m] for m in names if s[m] is not None}


def _norm_outputs(s):
    return {m: s[m] for m in ("h", "y", "y8", "scales") if s[m] is not None}


def _table_outputs(s):
    names = ("after", "left", "cu", "positions", "slot_in", "slot_out", "blocks", "free_list")
    return {m: s[m] for m in names}


def _problem(s):
    """The framework's description of the case, which a user's program keeps; made at the first pass of a state."""
    if "prob" not in s:
        import linear_attention_gdn_gb300 as gdn
        c = s["case"]
        if c["op"] in ("la_fwd", "la_bwd"):
            s["prob"] = gdn.la_problem(s["T"], c["N"], c["H"], c["HV"], scale=D ** -0.5,
                                       strides=tuple(s[m].stride(0) for m in "qkv"))
            need = gdn.gdn_la_workspace_bytes(s["prob"], s["cu_host"])[c["op"] == "la_bwd"]
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        elif c["op"] == "la_step":
            s["prob"] = gdn.step_problem(s["T"], c["N"], c["H"], c["HV"], s["slots"], scale=D ** -0.5, l2norm=False,
                                         dtype=s["q"].dtype, strides=tuple(s[m].stride(0) for m in "qkv"))
        elif c["op"] == "tables":
            s["prob"] = gdn.tables_problem(c["N"], s["T"], c["block"], s["most"], s["slots"])
        else:
            s["prob"] = gdn.norm_problem(c["T"], c["C"], eps=EPS, dtype=TYPES[c["dtype"]], group=max(c["group"], 0))
            if c["op"] == "norm_bwd":
                s["ws"] = torch.empty(max(gdn.gdn_add_norm_workspace_bytes(s["prob"]), 16), dtype=torch.uint8,
                                      device="cuda")
        s["gdn"] = gdn
    return s["gdn"], s["prob"]


def _own(s):
    gdn, prob = _problem(s)
    op = s["case"]["op"]
    if op == "la_fwd":
        gdn.gdn_la_fwd(prob, s["q"], s["k"], s["v"], s["g"], s["cu"], s["cu_host"], s["s_in"], s["o"], s["s_out"],
                       s["err"], s["ws"])
        return _la_outputs(s)
    if op == "la_bwd":
        gdn.gdn_la_bwd(prob, s["q"], s["k"], s["v"], s["g"], s["cu"], s["cu_host"], s["s_in"], s["do"], s["ds_out"],
                       s["dq"], s["dk"], s["dv"], s["ds_in"], s["err"], s["ws"])
        return _la_outputs(s)
    if op == "la_step":
        cu = None if s["case"]["hi"] == 1 else s["cu"]   # one token each: no starts are needed
        gdn.gdn_la_step(prob, s["q"], s["k"], s["v"], s["g"], s["states"], s["o"], s["err"], cu_seqlens_dev=cu,
                        slot_in=s["slot_in"], slot_out=s["slot_out"])
        return {"o": s["o"], "states": s["states"]}
    if op == "norm_fwd":
        gdn.gdn_add_norm_fwd(prob, s["x"], s["r"], s["w"], s["h"], s["y"], s["y8"], s["scales"])
        return _norm_outputs(s)
    if op == "norm_bwd":
        gdn.gdn_add_norm_bwd(prob, s["h"], s["w"], s["dy"], s["along"], s["dx"], s["dw"], s["ws"])
        return {"dx": s["dx"], "dw": s["dw"]}
    gdn.gdn_step_tables(prob, s["lengths"], s["before"], s["after"], s["blocks"], s["free_list"], s["free_count"],
                        s["left"], s["cu"], s["positions"], s["slot_in"], s["slot_out"], s["err"])
    return _table_outputs(s)


def run(s):
    if own:
        return _own(s)
    return {"la_fwd": _plain_la_fwd, "la_bwd": _plain_la_bwd, "la_step": _plain_la_step, "norm_fwd": _plain_norm_fwd,
            "norm_bwd": _plain_norm_bwd, "tables": _plain_tables}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "tables":
        x = _requests(case, 0)
        N, T = case["N"], x["T"]
        held = -(-x["context"].astype(np.int64) // case["block"])
        new = -(-(x["context"] + np.maximum(x["length"], 0).astype(np.int64)) // case["block"]) - held
        moved = int(held[x["length"] < 0].sum()) + int(new.sum())
        return {"bytes": 4 * (2 * T + 5 * N + 2 * moved), "flops": 0}
    if op in ("norm_fwd", "norm_bwd"):
        T, C, e = case["T"], case["C"], SIZE[case["dtype"]]
        if op == "norm_fwd":
            per = e * (1 + 2 * case["residual"] + case["plain"]) + (1 if case["group"] >= 0 else 0)
            scales = T * (C // (case["group"] or C)) * 4 if case["group"] >= 0 else 0
            return {"bytes": T * C * per + scales + 4 * C, "flops": 6 * T * C}
        return {"bytes": T * C * e * (3 + case["residual"]) + 8 * C, "flops": 11 * T * C}
    n = _lengths(case)
    T, live, HV, H = int(n.sum()), int((n > 0).sum()), case["HV"], case["H"]
    state = HV * D * D * 4
    if op == "la_step":
        _, slot_in, slot_out = _slots(case, n, 0)
        moved = int(((slot_in >= 0) & (n > 0)).sum()) + int((slot_out >= 0).sum())
        return {"bytes": moved * state + T * ((2 * H + 2 * HV) * D * SIZE[case["dtype"]] + 4) + 8 * live,
                "flops": T * HV * D * D * 5}
    small = case["N"] * 4 + HV * 4
    if op == "la_fwd":
        moved = case["N"] * state * {"both": 2, "out": 1, "none": 0}[case["states"]]
        return {"bytes": max(T * (2 * H + 2 * HV) * D * 2 + moved + small, 1), "flops": T * HV * D * D * 4}
    moved = case["N"] * state * {"both": 3, "out": 1, "none": 0}[case["states"]]
    return {"bytes": max(T * (4 * H + 3 * HV) * D * 2 + moved + small, 1), "flops": T * HV * D * D * 10}


def _exact_la(c, x):
    """The rule document by document in blocks of 256 tokens, in 64 bits; gradients by differentiating that."""
    G, back = c["HV"] // c["H"], c["op"] == "la_bwd"
    leaves = {m: x[m].double() for m in "qkv"}
    if back:
        leaves = {m: t.requires_grad_() for m, t in leaves.items()}
    q, k, v = leaves["q"], leaves["k"], leaves["v"]
    g = x["g"].double()
    start = torch.zeros((c["N"], c["HV"], D, D), dtype=torch.float64, device="cuda") if x["s_in"] is None else x["s_in"].double()
    if back:
        start.requires_grad_()
    outs, ends = [], []
    for d in range(c["N"]):
        S = start[d]
        for a in range(int(x["cu_host"][d]), int(x["cu_host"][d + 1]), 256):
            b = min(a + 256, int(x["cu_host"][d + 1]))
            Q, K, V = q[a:b].repeat_interleave(G, 1), k[a:b].repeat_interleave(G, 1), v[a:b]
            i = torch.arange(b - a, dtype=torch.float64, device="cuda")
            apart = i[:, None] - i
            decay = torch.where(apart >= 0, torch.exp(g[:, None, None] * apart.clamp(min=0)), 0.0)
            A = torch.einsum("rhd,chd->hrc", Q, K) * decay
            outs.append(torch.einsum("hrc,chd->rhd", A, V) + torch.einsum("rhi,hij,hr->rhj", Q, S, torch.exp(g[:, None] * (i + 1))))
            S = S * torch.exp(g * (b - a))[:, None, None] + torch.einsum("chi,chj,hc->hij", K, V, torch.exp(g[:, None] * (b - a - 1 - i)))
        ends.append(S)
    o = torch.cat(outs) / math.sqrt(D) if outs else torch.zeros((0, c["HV"], D), dtype=torch.float64, device="cuda")
    end = torch.stack(ends)
    if not back:
        return {"o": o, "s_out": end} if c["states"] != "none" else {"o": o}
    loss = (o * x["do"].double()).sum()
    if x["ds_out"] is not None:
        loss = loss + (end * x["ds_out"].double()).sum()
    if not loss.requires_grad:
        return None
    loss.backward()
    got = {"d" + m: t.grad if t.grad is not None else torch.zeros_like(t) for m, t in leaves.items()}
    if c["states"] == "both":
        got["ds_in"] = start.grad
    return got


def _exact_la_step(c, x):
    G, first = c["HV"] // c["H"], 0
    pool = x["states"].double()
    begin = pool.clone()
    o = torch.zeros((x["T"], c["HV"], D), dtype=torch.float64, device="cuda")
    a = torch.exp(x["g"].double())
    for i, m in enumerate(x["n"].tolist()):
        S = begin[x["slot_in_host"][i]] if x["slot_in_host"][i] >= 0 else torch.zeros_like(begin[0])
        for t in range(first, first + m):
            q, k = (x[y][t].double().repeat_interleave(G, 0) for y in ("q", "k"))
            S = torch.einsum("h,hij->hij", a, S) + torch.einsum("hi,hj->hij", k, x["v"][t].double())
            o[t] = torch.einsum("hij,hi->hj", S, q) / math.sqrt(D)
            if x["slot_out_host"][t] >= 0:
                pool[x["slot_out_host"][t]] = S
        first += m
    return {"o": o, "states": pool}


def _exact_norm(c, x):
    outs = {}
    if c["op"] == "norm_fwd":
        h = x["x"].double()
        if x["r"] is not None:
            h = h + x["r"].double()
            outs["h"] = h
            h = h.to(x["x"].dtype).double()   # the stream is held in its type, and the norm is of what is held
        z = h / torch.sqrt(torch.linalg.vector_norm(h, dim=-1, keepdim=True) ** 2 / c["C"] + EPS) * x["w"].double()
        if c["plain"]:
            outs["y"] = z
        if c["group"] >= 0:
            z = z.reshape(c["T"], -1, c["group"] or c["C"])
            outs["scales"] = torch.linalg.vector_norm(z, ord=math.inf, dim=-1).clamp(min=E4M3 * LEAST) / E4M3
            outs["y8"] = (z / outs["scales"][..., None]).reshape(c["T"], c["C"])
        return outs
    h, w = x["h"].double().requires_grad_(), x["w"].double().requires_grad_()
    y = h / torch.sqrt((h ** 2).mean(-1, keepdim=True) + EPS) * w
    y.backward(x["dy"].double())
    return {"dx": h.grad if x["along"] is None else h.grad + x["along"].double(), "dw": w.grad}


def exact(case, seed):
    if case["op"] == "tables":
        return None   # whole numbers
    x = _inputs(case, seed)
    if case["op"] in ("la_fwd", "la_bwd"):
        return _exact_la(case, x)
    if case["op"] == "la_step":
        return _exact_la_step(case, x)
    return _exact_norm(case, x)
