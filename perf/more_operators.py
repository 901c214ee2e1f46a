"""Decay-gated linear attention over sequences and in decode, and rotary positions: cases, plain forms and exact values.

Four operators, each reached through ``gdnspec`` where ``own`` is true and computed by elementary torch operations
where it is false:

* ``forward``  linear attention with a decay for each head over packed sequences (prefill): outputs and final states
* ``train``    the same with its gradient: one training step's forward and backward
* ``step``     one token for each sequence, the states of a pool updated in place (decode)
* ``rotary``   rotary positions of q and k, or (inverse) of their gradients

The recurrence for each (sequence, head), S being d_v x d_k:

    S_t = exp(log_alpha_t) S_{t-1} + beta_t v_t k_t^T,  o_t = S_t q_t

A rotary pair (x, y) at position p with frequency f becomes, for the angle a = p f,

    scale (x cos a - y sin a, x sin a + y cos a)
"""
import math
import random

import numpy as np
import torch
import torch.nn.functional as F

own = False

CHUNK = 64
ELEM = {"bf16": (torch.bfloat16, 2), "f32": (torch.float32, 4)}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    # decay "token": a gate of each token and head; "head": a constant of each head, slow, with write strength one
    seq = dict(dtype="bf16", n=1, H=8, Hk=8, dk=256, dv=256, ragged=False, decay="token")
    rot = dict(op="rotary", dtype="bf16", n=1, H=8, Hk=8, d=256, rot=256, layout="half", inverse=False, far=0, factor=1.0)
    return [
        # a long prompt of one user: the state before the first draft is verified
        dict(seq, name="prompt", op="forward", total=8192, decay="head"),
        # prompts of many users packed behind one another, q and k heads shared by two value heads
        dict(seq, name="prompts packed", op="forward", n=24, total=16000, Hk=4, dk=128, dv=128, ragged=True),
        # a follow-up turn: where the call's latency counts
        dict(seq, name="prompt short", op="forward", total=77),
        # training, equal lengths
        dict(seq, name="train", op="train", n=4, total=8192),
        # training on packed documents of odd lengths, q and k heads shared by four value heads
        dict(seq, name="train packed", op="train", n=9, total=6001, Hk=2, dk=128, dv=128, ragged=True, decay="head"),
        # a small model or a check run in single precision
        dict(seq, name="train f32", op="train", dtype="f32", n=2, total=301, H=4, Hk=4, dk=64, dv=64, ragged=True),
        # decode of one sequence
        dict(name="step one", op="step", dtype="bf16", B=1, slots=4, H=8, Hk=8, dk=256, dv=256),
        # decode of a full batch, with rows left empty by the batch's padding
        dict(name="step batch", op="step", dtype="bf16", B=64, slots=80, H=8, Hk=8, dk=256, dv=256),
        # q and k of 64 sequences' next tokens, deep in long contexts
        dict(rot, name="rotary decode", n=64, total=64, far=120000, factor=8.0),
        # q and k of a long prompt
        dict(rot, name="rotary prompt", total=8192),
        # gradients of packed documents, half of each head rotated, pairs side by side
        dict(rot, name="rotary gradient", n=9, total=6001, Hk=2, d=128, rot=64, layout="interleaved", inverse=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "train", "train", "step", "rotary", "rotary"])
    if op in ("forward", "train"):
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        Hk = rng.choice([1, 2, 4, 8])
        H = Hk * rng.choice([g for g in (1, 2, 4, 8) if Hk * g <= 8])
        dk, dv = rng.choice([(256, 256), (128, 128), (64, 64), (128, 256), (256, 128), (64, 128), (96, 96), (16, 48), (192, 80)])
        total = _log_int(rng, 1, 600 if dtype == "f32" else 8000)
        ragged = rng.random() < 0.6
        n = _log_int(rng, 1, 24 if dk * dv < 256 * 256 else 4) if ragged else rng.choice([1, 2, 3, 4])
        total = total if ragged else -(-total // n) * n
        return dict(op=op, dtype=dtype, n=n, total=total, H=H, Hk=Hk, dk=dk, dv=dv, ragged=ragged,
                    decay=rng.choice(["token", "head"]))
    if op == "step":
        Hk = rng.choice([1, 2, 4, 8])
        dk, dv = rng.choice([(256, 256), (128, 128), (64, 64), (128, 256), (96, 96), (16, 48), (192, 80)])
        B = _log_int(rng, 1, 64)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, slots=B + rng.randint(0, 16),
                    H=8, Hk=Hk, dk=dk, dv=dv)
    d = rng.choice([16, 48, 64, 96, 128, 192, 256])
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), n=rng.randint(1, 16), total=_log_int(rng, 16, 8000),
                H=rng.choice([1, 2, 4, 8]), Hk=rng.choice([1, 2, 4, 8]), d=d,
                rot=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]), layout=rng.choice(["half", "interleaved"]),
                inverse=rng.random() < 0.4, far=rng.choice([0, 0, 30000, 1000000]), factor=rng.choice([1.0, 1.0, 4.0, 32.0]))


def work(case):
    c = dict(case)
    if c["op"] in ("forward", "train"):
        e, tok = ELEM[c["dtype"]][1], c["total"]
        qk, vo = tok * c["Hk"] * c["dk"] * e, tok * c["H"] * c["dv"] * e
        gates, state = tok * c["H"] * 4, c["n"] * c["H"] * c["dk"] * c["dv"] * 4
        # the state updated and read for each token
        flops = 4 * tok * c["H"] * c["dk"] * c["dv"]
        nbytes = 2 * qk + 2 * vo + 2 * gates + 2 * state
        if c["op"] == "train":      # + dO, dS_T read; dq, dk, dv, two gate gradients, dS_0 written
            nbytes += 2 * qk + 2 * vo + 2 * gates + 2 * state
            flops *= 3
        return {"bytes": nbytes, "flops": flops}
    if c["op"] == "step":
        e = ELEM[c["dtype"]][1]
        live = len([i for i in _slots(c, 0) if i >= 0])
        state = live * c["H"] * c["dk"] * c["dv"]
        return {"bytes": 8 * state + c["B"] * e * (2 * c["Hk"] * c["dk"] + 2 * c["H"] * c["dv"]) + 8 * c["B"] * c["H"],
                "flops": 5 * state}
    heads = c["total"] * (c["H"] + c["Hk"])
    return {"bytes": 2 * heads * c["d"] * ELEM[c["dtype"]][1] + 4 * c["total"], "flops": 4 * heads * c["rot"]}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _lengths(case, seed):
    """Lengths of the packed sequences: equal, or cut at random places (empty sequences among them)."""
    if not case.get("ragged", True):
        return [case["total"] // case["n"]] * case["n"]
    r = random.Random(seed * 7919 + 13)
    cuts = sorted(r.randint(0, case["total"]) for _ in range(case["n"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["total"]])]


def _slots(case, seed):
    """Each row's place in the pool of states; -1 for a row that the batch's padding leaves empty (one in eight)."""
    r = random.Random(seed * 104729 + 7)
    at = r.sample(range(case["slots"]), case["B"])
    return [-1 if i % 8 == 5 else s for i, s in enumerate(at)]


def _frequencies(rot, base, factor, original):
    """Frequencies of the pairs, those that turn less than 32 times in the original context slowed by up to `factor`."""
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    turns = original * f / (2 * math.pi)
    kept = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return (f * kept + f / factor * (1.0 - kept)).float()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _unit(shape, g):
    x = torch.randn(shape, generator=g, device="cuda")
    return x / x.norm(dim=-1, keepdim=True)


def _gates(shape, g, decay):
    if decay == "head":
        # constant decays 1 - 2^-u, u from 3 to 9
        u = torch.linspace(3, 9, shape[-1], device="cuda")
        return (-torch.pow(2.0, -u)).log1p().expand(shape).contiguous(), torch.ones(shape, device="cuda")
    # decay exp(-softplus(u)) from slow (0.998 a token) to fast (0.27), write strength sigmoid(u)
    la = -F.softplus(torch.rand(shape, generator=g, device="cuda") * 7 - 6)
    beta = torch.sigmoid(torch.rand(shape, generator=g, device="cuda") * 4 - 2)
    return la, beta


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    dev, t = "cuda", ELEM[c["dtype"]][0]
    s = dict(case=c)
    if c["op"] in ("forward", "train"):
        n, tok, H, Hk, dk, dv = (c[x] for x in ("n", "total", "H", "Hk", "dk", "dv"))
        lead = (tok,) if c["ragged"] else (n, tok // n)
        s["q"], s["k"] = _unit((*lead, Hk, dk), g).to(t), _unit((*lead, Hk, dk), g).to(t)
        s["v"] = torch.randn((*lead, H, dv), generator=g, device=dev).to(t)
        s["log_alpha"], s["beta"] = _gates((*lead, H), g, c["decay"])
        s["S0"] = torch.randn((n, H, dv, dk), generator=g, device=dev) * 0.1
        s["lengths"] = _lengths(c, seed)
        s["offsets"] = torch.tensor(np.cumsum([0] + s["lengths"]), dtype=torch.int32, device=dev) if c["ragged"] else None
        s["out"], s["S_T"] = torch.empty_like(s["v"]), torch.empty_like(s["S0"])
        if c["op"] == "train":
            s["dout"] = torch.randn((*lead, H, dv), generator=g, device=dev).to(t)
            s["dS_T"] = torch.randn((n, H, dv, dk), generator=g, device=dev) * 0.1
            for x in ("q", "k", "v", "log_alpha", "beta", "S0"):
                s["d" + x] = torch.empty_like(s[x])
        return s
    if c["op"] == "step":
        B, H, Hk, dk, dv = (c[x] for x in ("B", "H", "Hk", "dk", "dv"))
        s["q"], s["k"] = _unit((B, Hk, dk), g).to(t), _unit((B, Hk, dk), g).to(t)
        s["v"] = torch.randn((B, H, dv), generator=g, device=dev).to(t)
        s["log_alpha"], s["beta"] = _gates((B, H), g, "token")
        s["S"] = torch.randn((c["slots"], H, dv, dk), generator=g, device=dev) * 0.1
        at = _slots(c, seed)
        s["index"] = torch.tensor(at, dtype=torch.int32, device=dev)
        s["rows"] = torch.tensor([i for i, x in enumerate(at) if x >= 0], device=dev)
        s["at"] = torch.tensor([x for x in at if x >= 0], device=dev)
        s["out"] = torch.empty_like(s["v"])
        return s
    lengths = _lengths(c, seed)
    r = random.Random(seed * 15485863 + 3)
    starts = [r.randint(0, c["far"]) for _ in lengths]
    s["positions"] = torch.from_numpy(np.concatenate([np.arange(p, p + m) for p, m in zip(starts, lengths)])).to(torch.int32).to(dev)
    s["inv_freq"] = _frequencies(c["rot"], 10000.0, c["factor"], 4096.0).to(dev)
    s["scale"] = 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0
    s["q"] = torch.randn((c["total"], c["H"], c["d"]), generator=g, device=dev).to(t)
    s["k"] = torch.randn((c["total"], c["Hk"], c["d"]), generator=g, device=dev).to(t)
    s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    return {"forward": _forward, "train": _train, "step": _step, "rotary": _rotary}[c["op"]](s, c)


def _lib():
    from speculative_decoding_linear_gb300 import gdnspec
    return gdnspec


def _forward(s, c):
    if own:
        G = _lib()
        if "workspace" not in s:
            s["workspace"] = G.empty_linear_seq_workspace(c["n"], c["total"], c["H"], c["Hk"], c["dk"], c["dv"], s["q"].dtype,
                                                          backward=False)
        G.gdn_linear_seq_forward(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["S0"], s["out"], s["S_T"],
                                 s["workspace"], offsets=s["offsets"])
        return {"out": s["out"], "S_T": s["S_T"]}
    x = _padded(s, c, torch.float32)
    o, S = _chunked(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], s["S0"], c["H"] // c["Hk"])
    return {"out": _packed(o, s, c).to(s["q"].dtype), "S_T": S}


def _train(s, c):
    if own:
        G = _lib()
        if "workspace" not in s:
            dims = (c["n"], c["total"], c["H"], c["Hk"], c["dk"], c["dv"], s["q"].dtype)
            s["workspace"], s["record"] = G.empty_linear_seq_workspace(*dims), G.empty_linear_seq_record(*dims)
        G.gdn_linear_seq_forward(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["S0"], s["out"], s["S_T"],
                                 s["workspace"], offsets=s["offsets"], record=s["record"])
        G.gdn_linear_seq_backward(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["dout"], s["dS_T"], s["record"],
                                  s["dq"], s["dk"], s["dv"], s["dlog_alpha"], s["dbeta"], s["dS0"], s["workspace"],
                                  offsets=s["offsets"])
        return {x: s[x] for x in ("out", "S_T", "dq", "dk", "dv", "dlog_alpha", "dbeta", "dS0")}
    x = _padded(s, c, torch.float32)
    names = ("q", "k", "v", "log_alpha", "beta")
    leaf = {m: x[m].requires_grad_() for m in names}
    leaf["S0"] = s["S0"].detach().clone().requires_grad_()
    with torch.enable_grad():
        o, S = _chunked(*(leaf[m] for m in names), leaf["S0"], c["H"] // c["Hk"])
    grads = torch.autograd.grad((o, S), [*leaf.values()], (x["dout"], s["dS_T"]))
    got = {"out": _packed(o.detach(), s, c).to(s["q"].dtype), "S_T": S.detach()}
    got.update({"d" + m: d if m == "S0" else _packed(d, s, c).to(s[m].dtype) for m, d in zip(leaf, grads)})
    return got


def _step(s, c):
    if own:
        _lib().gdn_linear_seq_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["S"], s["out"], state_index=s["index"])
        return {"out": s["out"], "S": s["S"]}
    r, rep = s["rows"], c["H"] // c["Hk"]
    q, k = (s[m][r].float().repeat_interleave(rep, 1) for m in ("q", "k"))
    S = s["S"][s["at"]] * s["log_alpha"][r].exp()[..., None, None]
    S = S + (s["beta"][r][..., None] * s["v"][r].float())[..., None] * k[:, :, None, :]
    out = torch.zeros_like(s["v"])
    out[r] = (S * q[:, :, None, :]).sum(-1).to(out.dtype)
    s["S"][s["at"]] = S
    return {"out": out, "S": s["S"]}


def _rotary(s, c):
    if own:
        _lib().gdn_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"], scale=s["scale"],
                          interleaved=c["layout"] == "interleaved", inverse=c["inverse"])
        return {"q": s["q_out"], "k": s["k_out"]}
    # angles of far positions in 64 bits
    a = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = (a.cos() * s["scale"]).float(), (a.sin() * (-s["scale"] if c["inverse"] else s["scale"])).float()

    def turned(x):
        y = x[..., : c["rot"]].float()
        if c["layout"] == "half":
            u, w = y.chunk(2, -1)
            y = torch.cat([u * cos - w * sin, u * sin + w * cos], -1)
        else:
            u, w = y[..., 0::2], y[..., 1::2]
            y = torch.stack([u * cos - w * sin, u * sin + w * cos], -1).flatten(-2)
        return torch.cat([y.to(x.dtype), x[..., c["rot"]:]], -1)

    return {"q": turned(s["q"]), "k": turned(s["k"])}


# ---------------------------------------------------------------------------------------------------------------
# plain linear attention: chunks of 64 tokens, and products over all chunks for the states between them
# ---------------------------------------------------------------------------------------------------------------
def _place(s, c):
    """Row of each packed token in the padded batch [n, longest]."""
    longest = max(1, max(s["lengths"]))
    return torch.cat([torch.arange(m, device="cuda") + i * longest for i, m in enumerate(s["lengths"])]), longest


def _padded(s, c, dtype):
    """The call's tensors as [n, longest, ...]: a token with k = q = v = 0, log_alpha = 0, beta = 0 changes nothing."""
    names = [m for m in ("q", "k", "v", "log_alpha", "beta", "dout") if m in s]
    if not c["ragged"]:
        return {m: s[m].detach().to(dtype, copy=True) for m in names}
    at, longest = _place(s, c)

    def padded(x):
        y = torch.zeros((c["n"] * longest, *x.shape[1:]), dtype=dtype, device="cuda")
        y[at] = x.detach().to(dtype)
        return y.view(c["n"], longest, *x.shape[1:])

    return {m: padded(s[m]) for m in names}


def _packed(x, s, c):
    if not c["ragged"]:
        return x
    return x.flatten(0, 1)[_place(s, c)[0]]


def _chunked(q, k, v, log_alpha, beta, S0, rep):
    n, T, H, dv = v.shape
    N = max(1, -(-T // CHUNK))

    def cut(x):      # [n, T, heads, ...] -> [n, heads, N, 64, ...], its end filled with tokens that change nothing
        x = torch.cat([x, x.new_zeros((n, N * CHUNK - T, *x.shape[2:]))], 1)
        return x.unflatten(1, (N, CHUNK)).movedim(3, 1)

    def below(g, first):      # exp(g_i - g_j) for j <= i - first, else 0; differences of long sums in 64 bits
        at = torch.arange(g.shape[-1], device=g.device)
        seen = at[:, None] - first >= at[None, :]
        return (g[..., :, None] - g[..., None, :]).masked_fill(~seen, -math.inf).exp().float()

    q, k, v, beta = cut(q), cut(k), cut(v), cut(beta)
    g = cut(log_alpha).double().cumsum(-1)
    qk = q @ k.transpose(-1, -2)
    if rep > 1:
        q, k, qk = (x.repeat_interleave(rep, 1) for x in (q, k, qk))
    w = beta[..., None] * v
    end = g[..., -1]
    into = end.cumsum(-1)                                        # decay of all chunks so far
    # what each chunk adds to the state, and the state behind each chunk: S0 and the chunks up to it, decayed
    added = k.transpose(-1, -2) @ ((end[..., None] - g).exp().float()[..., None] * w)
    S0 = S0.transpose(-1, -2)
    behind = (below(into, 0) @ added.flatten(-2)).view_as(added) + into.exp().float()[..., None, None] * S0[:, :, None]
    before = torch.cat([S0[:, :, None], behind[:, :, :-1]], 2)
    o = g.exp().float()[..., None] * (q @ before) + (qk * below(g, 0)) @ w
    return o.flatten(2, 3)[:, :, :T].movedim(1, 2), behind[:, :, -1].transpose(-1, -2).contiguous()


# ---------------------------------------------------------------------------------------------------------------
# exact values: the definition in 64 bits, token by token
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    return {"forward": _exact_seq, "train": _exact_seq, "step": _exact_step, "rotary": _exact_rotary}[c["op"]](s, c)


def _outer(x, y):
    return x[..., :, None] * y[..., None, :]


def _exact_seq(s, c):
    x, rep = _padded(s, c, torch.float64), c["H"] // c["Hk"]
    q, k = (x[m].repeat_interleave(rep, 2) for m in ("q", "k"))
    v, la, b = x["v"], x["log_alpha"], x["beta"]
    T, S, o, kept = v.shape[1], s["S0"].double(), torch.zeros_like(v), []
    for t in range(T):
        if t % CHUNK == 0 and c["op"] == "train":
            kept.append(S)
        S = S * la[:, t].exp()[..., None, None] + _outer(b[:, t, :, None] * v[:, t], k[:, t])
        o[:, t] = (S @ q[:, t, :, :, None])[..., 0]
    got = {"out": _packed(o, s, c), "S_T": S}
    if c["op"] != "train":
        return got
    do, dS = x["dout"], s["dS_T"].double()
    dq, dk, dv, dla, db = (torch.zeros_like(y) for y in (q, k, v, la, b))
    for first in reversed(range(0, T, CHUNK)):
        S, seen = kept[first // CHUNK], []
        for t in range(first, min(T, first + CHUNK)):
            D = S * la[:, t].exp()[..., None, None]
            S = D + _outer(b[:, t, :, None] * v[:, t], k[:, t])
            seen.append((t, S, D))
        for t, St, D in reversed(seen):
            dq[:, t] = (do[:, t, :, None, :] @ St)[..., 0, :]
            dS = dS + _outer(do[:, t], q[:, t])
            dw = (dS @ k[:, t, :, :, None])[..., 0]
            db[:, t], dv[:, t] = (dw * v[:, t]).sum(-1), b[:, t, :, None] * dw
            dk[:, t] = b[:, t, :, None] * (v[:, t, :, None, :] @ dS)[..., 0, :]
            dla[:, t] = (dS * D).sum((-1, -2))
            dS = dS * la[:, t].exp()[..., None, None]
    dq, dk = (y.unflatten(2, (c["Hk"], rep)).sum(3) for y in (dq, dk))
    for m, y in (("q", dq), ("k", dk), ("v", dv), ("log_alpha", dla), ("beta", db)):
        got["d" + m] = _packed(y, s, c)
    got["dS0"] = dS
    return got


def _exact_step(s, c):
    pool, out, rep = s["S"].double(), torch.zeros_like(s["v"], dtype=torch.float64), c["H"] // c["Hk"]
    for row, at in zip(s["rows"].tolist(), s["at"].tolist()):
        q, k = (s[m][row].double().repeat_interleave(rep, 0) for m in ("q", "k"))
        decay = torch.exp(s["log_alpha"][row].double())
        pool[at] = torch.einsum("h,hvk->hvk", decay, pool[at]) + torch.einsum("h,hv,hk->hvk", s["beta"][row].double(), s["v"][row].double(), k)
        out[row] = torch.einsum("hvk,hk->hv", pool[at], q)
    return {"out": out, "S": pool}


def _exact_rotary(s, c):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    turn = torch.polar(torch.full_like(angle, s["scale"]), -angle if c["inverse"] else angle)[:, None, :]
    m = c["rot"] // 2
    got = {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        first, second = (slice(0, m), slice(m, 2 * m)) if c["layout"] == "half" else (slice(0, 2 * m, 2), slice(1, 2 * m, 2))
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        x[..., first], x[..., second] = z.real, z.imag
        got[name] = x
    return got
