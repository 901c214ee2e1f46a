"""Sequence, single-token and norm operators of a Gated DeltaNet block: their cases, plain forms and exact values.

Four operators, each reached through ``gdnspec`` where ``own`` is true and computed by elementary torch operations
where it is false:

* ``forward``     the gated delta rule over packed sequences (prefill): outputs and final states
* ``train``       the same with its gradient: one training step's forward and backward
* ``step``        one token for each sequence, the states of a pool updated in place (decode)
* ``gated_norm``  y = RMSNorm(o) * w * SiLU(z) for each head, and its gradient
* ``block_norm``  x' = rho x + gamma * (RMSNorm(z) * w_post), h = RMSNorm(x') * w_pre, and its gradient

The recurrence for each (sequence, head), S being d_v x d_k:

    S' = exp(log_alpha_t) S_{t-1},  e_t = v_t - S' k_t,  S_t = S' + beta_t e_t k_t^T,  o_t = S_t q_t
"""
import math
import random

import numpy as np
import torch
import torch.nn.functional as F

own = False

EPS = 1e-6
CHUNK = 64
ELEM = {"bf16": (torch.bfloat16, 2), "f32": (torch.float32, 4)}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    seq = dict(dtype="bf16", n=1, H=8, Hk=8, dk=256, dv=256, ragged=False)
    return [
        # a long prompt of one user: the state before the first draft is verified
        dict(seq, name="prompt", op="forward", total=8192),
        # prompts of many users packed behind one another, q and k heads shared by two value heads
        dict(seq, name="prompts packed", op="forward", n=24, total=16000, Hk=4, dk=128, dv=128, ragged=True),
        # a follow-up turn: little more than a chunk, where the call's latency counts
        dict(seq, name="prompt short", op="forward", total=77),
        # training, equal lengths
        dict(seq, name="train", op="train", n=4, total=8192),
        # training on packed documents of odd lengths, q and k heads shared by four value heads
        dict(seq, name="train packed", op="train", n=9, total=6001, Hk=2, dk=128, dv=128, ragged=True),
        # a small model or a check run in single precision
        dict(seq, name="train f32", op="train", dtype="f32", n=2, total=301, H=4, Hk=4, dk=64, dv=64, ragged=True),
        # decode of one sequence
        dict(name="step one", op="step", dtype="bf16", B=1, slots=4, H=8, Hk=8, dk=256, dv=256),
        # decode of a full batch, with rows left empty by the batch's padding
        dict(name="step batch", op="step", dtype="bf16", B=64, slots=80, H=8, Hk=8, dk=256, dv=256),
        # output norm and gate of a verified tree (fp32 outputs of the verifier)
        dict(name="gated norm verify", op="gated_norm", back=False, odtype="f32", dtype="bf16", rows=64, H=8, d=256),
        # the same in training
        dict(name="gated norm train", op="gated_norm", back=True, odtype="bf16", dtype="bf16", rows=8192, H=8, d=256),
        # residual, post-norm and the next layer's pre-norm in decode
        dict(name="block norm decode", op="block_norm", back=False, post=True, dtype="bf16", rows=64, D=2048),
        # the same in training
        dict(name="block norm train", op="block_norm", back=True, post=True, dtype="bf16", rows=8192, D=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "train", "train", "step", "gated_norm", "block_norm"])
    if op in ("forward", "train"):
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        Hk = rng.choice([1, 2, 4, 8])
        H = Hk * rng.choice([g for g in (1, 2, 4, 8) if Hk * g <= 8])
        dk, dv = rng.choice([(256, 256), (128, 128), (64, 64), (128, 256), (256, 128), (64, 128), (96, 96), (16, 48), (192, 80)])
        total = _log_int(rng, 1, 600 if dtype == "f32" else 8000)
        ragged = rng.random() < 0.6
        n = _log_int(rng, 1, 24) if ragged else rng.choice([1, 2, 3, 4])
        total = total if ragged else -(-total // n) * n
        return dict(op=op, dtype=dtype, n=n, total=total, H=H, Hk=Hk, dk=dk, dv=dv, ragged=ragged)
    if op == "step":
        Hk = rng.choice([1, 2, 4, 8])
        dk, dv = rng.choice([(256, 256), (128, 128), (64, 64), (128, 256), (96, 96), (16, 48), (192, 80)])
        B = _log_int(rng, 1, 64)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, slots=B + rng.randint(0, 16),
                    H=8, Hk=Hk, dk=dk, dv=dv)
    if op == "gated_norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, back=rng.random() < 0.5, odtype="f32" if dtype == "f32" or rng.random() < 0.4 else "bf16",
                    dtype=dtype, rows=_log_int(rng, 1, 8192), H=rng.choice([1, 2, 4, 8]),
                    d=rng.choice([16, 48, 64, 96, 128, 192, 256]))
    return dict(op=op, back=rng.random() < 0.5, post=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "f32"]),
                rows=_log_int(rng, 1, 4096), D=rng.choice([64, 264, 1000, 2048, 2560, 4096]))


def work(case):
    c = dict(case)
    if c["op"] in ("forward", "train"):
        e, tok = ELEM[c["dtype"]][1], c["total"]
        qk, vo = tok * c["Hk"] * c["dk"] * e, tok * c["H"] * c["dv"] * e
        gates, state = tok * c["H"] * 4, c["n"] * c["H"] * c["dk"] * c["dv"] * 4
        # K S, Q S and K^T delta for each token, and the products inside a chunk (half of each is masked)
        flops = 2 * tok * c["H"] * (3 * c["dk"] * c["dv"] + CHUNK // 2 * (2 * c["dk"] + 2 * c["dv"]))
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
                "flops": 7 * state}
    if c["op"] == "gated_norm":
        n, e, eo = c["rows"] * c["H"] * c["d"], ELEM[c["dtype"]][1], ELEM[c["odtype"]][1]
        return {"bytes": n * (2 * eo + 3 * e) if c["back"] else n * (eo + 2 * e), "flops": n * (20 if c["back"] else 8)}
    n, e = c["rows"] * c["D"], ELEM[c["dtype"]][1]
    streams = (6 if c["post"] else 4) if c["back"] else (4 if c["post"] else 2)
    return {"bytes": streams * n * e, "flops": n * (24 if c["back"] else 10)}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _lengths(case, seed):
    """Lengths of the packed sequences: equal, or cut at random places (empty sequences among them)."""
    if not case["ragged"]:
        return [case["total"] // case["n"]] * case["n"]
    r = random.Random(seed * 7919 + 13)
    cuts = sorted(r.randint(0, case["total"]) for _ in range(case["n"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["total"]])]


def _slots(case, seed):
    """Each row's place in the pool of states; -1 for a row that the batch's padding leaves empty (one in eight)."""
    r = random.Random(seed * 104729 + 7)
    at = r.sample(range(case["slots"]), case["B"])
    return [-1 if i % 8 == 5 else s for i, s in enumerate(at)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _unit(shape, g):
    x = torch.randn(shape, generator=g, device="cuda")
    return x / x.norm(dim=-1, keepdim=True)


def _gates(shape, g):
    # decay exp(-softplus(u)) from slow (0.998 a token) to fast (0.27), write strength sigmoid(u)
    la = -F.softplus(torch.rand(shape, generator=g, device="cuda") * 7 - 6)
    beta = torch.sigmoid(torch.rand(shape, generator=g, device="cuda") * 4 - 2)
    return la, beta


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    dev = "cuda"
    s = dict(case=c)
    if c["op"] in ("forward", "train"):
        t = ELEM[c["dtype"]][0]
        n, tok, H, Hk, dk, dv = (c[x] for x in ("n", "total", "H", "Hk", "dk", "dv"))
        lead = (tok,) if c["ragged"] else (n, tok // n)
        s["q"], s["k"] = _unit((*lead, Hk, dk), g).to(t), _unit((*lead, Hk, dk), g).to(t)
        s["v"] = torch.randn((*lead, H, dv), generator=g, device=dev).to(t)
        s["log_alpha"], s["beta"] = _gates((*lead, H), g)
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
        t = ELEM[c["dtype"]][0]
        B, H, Hk, dk, dv = (c[x] for x in ("B", "H", "Hk", "dk", "dv"))
        s["q"], s["k"] = _unit((B, Hk, dk), g).to(t), _unit((B, Hk, dk), g).to(t)
        s["v"] = torch.randn((B, H, dv), generator=g, device=dev).to(t)
        s["log_alpha"], s["beta"] = _gates((B, H), g)
        s["S"] = torch.randn((c["slots"], H, dv, dk), generator=g, device=dev) * 0.1
        at = _slots(c, seed)
        s["index"] = torch.tensor(at, dtype=torch.int32, device=dev)
        s["rows"] = torch.tensor([i for i, x in enumerate(at) if x >= 0], device=dev)
        s["at"] = torch.tensor([x for x in at if x >= 0], device=dev)
        s["out"] = torch.empty_like(s["v"])
        return s
    t = ELEM[c["dtype"]][0]

    def rand(*shape, std=1.0, mean=0.0, dtype=None):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype or t)

    if c["op"] == "gated_norm":
        shape = (c["rows"], c["H"], c["d"])
        s["o"], s["z"] = rand(*shape, std=0.3, dtype=ELEM[c["odtype"]][0]), rand(*shape)
        s["w"] = rand(c["d"], std=0.1, mean=1.0)
        s["y"] = torch.empty_like(s["z"])
        if c["back"]:
            s["dy"] = rand(*shape)
            s["do"], s["dz"] = torch.empty_like(s["o"]), torch.empty_like(s["z"])
            s["dw"] = torch.empty(c["d"], device=dev)
        return s
    rows, D = c["rows"], c["D"]
    s["x"], s["w"] = rand(rows, D), rand(D, std=0.1, mean=1.0)
    s["z"] = rand(rows, D, std=0.5) if c["post"] else None
    s["wp"] = rand(D, std=0.1, mean=1.0) if c["post"] else None
    s["gate"] = rand(D, std=0.1, mean=0.5) if c["post"] else None
    s["rho"] = 0.9 if c["post"] else 1.0
    s["h"], s["x2"] = torch.empty_like(s["x"]), torch.empty_like(s["x"]) if c["post"] else None
    if c["back"]:
        s["dh"], s["dx2"] = rand(rows, D), rand(rows, D)
        s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty(D, device=dev)
        if c["post"]:
            s["dz"], s["dwp"], s["dgate"] = torch.empty_like(s["x"]), torch.empty(D, device=dev), torch.empty(D, device=dev)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    return {"forward": _forward, "train": _train, "step": _step, "gated_norm": _gated_norm,
            "block_norm": _block_norm}[c["op"]](s, c)


def _lib():
    from speculative_decoding_linear_gb300 import gdnspec
    return gdnspec


def _forward(s, c):
    if own:
        G = _lib()
        if "workspace" not in s:
            s["workspace"] = G.empty_seq_workspace(c["n"], c["total"], c["H"], c["Hk"], c["dk"], c["dv"], s["q"].dtype)
        G.gdn_seq_forward(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["S0"], s["out"], s["S_T"],
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
            s["workspace"], s["record"] = G.empty_seq_workspace(*dims), G.empty_seq_record(*dims)
        G.gdn_seq_forward(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["S0"], s["out"], s["S_T"],
                          s["workspace"], offsets=s["offsets"], record=s["record"])
        G.gdn_seq_backward(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["dout"], s["dS_T"], s["record"],
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
    for m, d in zip(leaf, grads):
        got["d" + m] = d if m == "S0" else _packed(d, s, c).to(s[m].dtype)
    return got


def _step(s, c):
    if own:
        _lib().gdn_seq_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["S"], s["out"], state_index=s["index"])
        return {"out": s["out"], "S": s["S"]}
    r, rep = s["rows"], c["H"] // c["Hk"]
    q, k = (s[m][r].float().repeat_interleave(rep, 1) for m in ("q", "k"))
    S = s["S"][s["at"]] * s["log_alpha"][r].exp()[..., None, None]
    e = s["v"][r].float() - (S * k[:, :, None, :]).sum(-1)
    S = S + (s["beta"][r][..., None] * e)[..., None] * k[:, :, None, :]
    out = torch.zeros_like(s["v"])
    out[r] = (S * q[:, :, None, :]).sum(-1).to(out.dtype)
    s["S"][s["at"]] = S
    return {"out": out, "S": s["S"]}


def _gated_norm(s, c):
    if own:
        G = _lib()
        if not c["back"]:
            G.gdn_gated_norm(s["o"], s["z"], s["w"], s["y"], eps=EPS)
            return s["y"]
        if "workspace" not in s:
            s["workspace"] = G.empty_norm_workspace(c["rows"] * c["H"], c["d"])
        G.gdn_gated_norm_backward(s["o"], s["z"], s["w"], s["dy"], s["do"], s["dz"], s["dw"], s["workspace"], eps=EPS)
        return {m: s[m] for m in ("do", "dz", "dw")}
    o, z, w = s["o"].float(), s["z"].float(), s["w"].float()
    r = (o.square().mean(-1, keepdim=True) + EPS).rsqrt()
    sg = 1 / (1 + (-z).exp())
    if not c["back"]:
        return (o * r * w * (z * sg)).to(s["z"].dtype)
    dy, n = s["dy"].float(), o * r
    dn = dy * w * (z * sg)
    return {"do": (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(s["o"].dtype),
            "dz": (dy * n * w * sg * (1 + z * (1 - sg))).to(s["z"].dtype),
            "dw": (dy * n * (z * sg)).double().sum((0, 1)).float()}


def _block_norm(s, c):
    if own:
        G = _lib()
        if not c["back"]:
            G.gdn_block_norm(s["x"], s["z"], s["wp"], s["gate"], s["w"], s["x2"], s["h"], eps=EPS, res_scale=s["rho"])
            return {"h": s["h"], "x2": s["x2"]}
        if "workspace" not in s:
            s["workspace"] = G.empty_norm_workspace(c["rows"], c["D"])
        G.gdn_block_norm_backward(s["x"], s["z"], s["wp"], s["gate"], s["w"], s["dh"], s["dx2"], s["dx"], s.get("dz"),
                                  s.get("dwp"), s.get("dgate"), s["dw"], s["workspace"], eps=EPS, res_scale=s["rho"])
        return {m: s.get(m) for m in ("dx", "dz", "dw", "dwp", "dgate")}
    t, x, w, rho = s["x"].dtype, s["x"].float(), s["w"].float(), s["rho"]

    def unit(u):
        r = (u.square().mean(-1, keepdim=True) + EPS).rsqrt()
        return u * r, r

    if not c["back"]:
        if c["post"]:
            x = rho * x + s["gate"].float() * (unit(s["z"].float())[0] * s["wp"].float())
        return {"h": (unit(x)[0] * w).to(t), "x2": x.to(t) if c["post"] else None}
    # backward takes the new residual stream, which the forward pass gave, as its x
    dh, (n, r) = s["dh"].float(), unit(x)
    dn = dh * w
    d = s["dx2"].float() + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    got = {"dx": (rho * d).to(t), "dw": (dh * n).double().sum(0).float(), "dz": None, "dwp": None, "dgate": None}
    if c["post"]:
        m, r = unit(s["z"].float())
        gate, wp = s["gate"].float(), s["wp"].float()
        dm = d * gate * wp
        got["dz"] = (r * (dm - m * (dm * m).mean(-1, keepdim=True))).to(t)
        got["dwp"] = (d * gate * m).double().sum(0).float()
        got["dgate"] = (d * m * wp).double().sum(0).float()
    return got


# ---------------------------------------------------------------------------------------------------------------
# the plain gated delta rule: chunks of 64 tokens, one matrix product for all chunks where the state is not needed
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
    got = {}
    for m in names:
        x = torch.zeros((c["n"] * longest, *s[m].shape[1:]), dtype=dtype, device="cuda")
        x[at] = s[m].detach().to(dtype)
        got[m] = x.view(c["n"], longest, *s[m].shape[1:])
    return got


def _packed(x, s, c):
    if not c["ragged"]:
        return x
    return x.flatten(0, 1)[_place(s, c)[0]]


def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower A [..., 64, 64], by blocks of 1, 2, 4, ... on the diagonal."""
    m = A.shape[-1]
    inv = torch.ones((*A.shape[:-2], m, 1, 1), dtype=A.dtype, device=A.device)
    b = 1
    while b < m:
        k = m // (2 * b)
        blocks = A.unflatten(-1, (m // b, b)).unflatten(-3, (m // b, b)).movedim(-2, -3)   # [..., row, col, b, b]
        at = torch.arange(k, device=A.device)
        low = blocks[..., 2 * at + 1, 2 * at, :, :]
        a, d = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
        top = torch.cat([a, torch.zeros_like(a)], -1)
        inv = torch.cat([top, torch.cat([-(d @ (low @ a)), d], -1)], -2)
        b *= 2
    return inv[..., 0, :, :]


def _chunked(q, k, v, log_alpha, beta, S0, rep):
    n, T, H, dv = v.shape
    N = max(1, -(-T // CHUNK))

    def cut(x):      # [n, T, heads, ...] -> [n, heads, N, 64, ...], its end filled with tokens that change nothing
        x = torch.cat([x, x.new_zeros((n, N * CHUNK - T, *x.shape[2:]))], 1)
        return x.unflatten(1, (N, CHUNK)).movedim(3, 1)

    q, k, v, beta = cut(q), cut(k), cut(v), cut(beta)
    g = cut(log_alpha).double().cumsum(-1)               # differences of long sums: 64 bits
    row = torch.arange(CHUNK, device=v.device)
    seen = row[:, None] >= row[None, :]
    decay = (g[..., :, None] - g[..., None, :]).masked_fill(~seen, -math.inf).exp().float()
    kk, qk = k @ k.transpose(-1, -2), q @ k.transpose(-1, -2)
    if rep > 1:
        q, k, kk, qk = (x.repeat_interleave(rep, 1) for x in (q, k, kk, qk))
    inv = _unit_lower_inverse((kk * decay).masked_fill(row[:, None] == row[None, :], 0.0) * beta[..., None, :])
    P = qk * decay
    eg, end = g.exp().float()[..., None], g[..., -1:]
    tail, last = (end - g).exp().float()[..., None], end.exp().float()[..., None]
    S, out = S0.transpose(-1, -2), []
    for i in range(N):
        r = v[:, :, i] - eg[:, :, i] * (k[:, :, i] @ S)
        delta = beta[:, :, i, :, None] * (inv[:, :, i] @ r)
        out.append(eg[:, :, i] * (q[:, :, i] @ S) + P[:, :, i] @ delta)
        S = last[:, :, i] * S + k[:, :, i].transpose(-1, -2) @ (tail[:, :, i] * delta)
    o = torch.stack(out, 2).flatten(2, 3)[:, :, :T].movedim(1, 2)
    return o, S.transpose(-1, -2).contiguous()


# ---------------------------------------------------------------------------------------------------------------
# exact values: the definition in 64 bits, token by token
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    return {"forward": _exact_seq, "train": _exact_seq, "step": _exact_step, "gated_norm": _exact_gated_norm,
            "block_norm": _exact_block_norm}[c["op"]](s, c)


def _token(S, q, k, v, la, b):
    """One token of the recurrence: (S_t, decayed state, error, output)."""
    D = S * la.exp()[..., None, None]
    e = v - torch.einsum("nhvk,nhk->nhv", D, k)
    S = D + torch.einsum("nhv,nhk->nhvk", b[..., None] * e, k)
    return S, D, e, torch.einsum("nhvk,nhk->nhv", S, q)


def _exact_seq(s, c):
    x, rep = _padded(s, c, torch.float64), c["H"] // c["Hk"]
    q, k = (x[m].repeat_interleave(rep, 2) for m in ("q", "k"))
    v, la, b = x["v"], x["log_alpha"], x["beta"]
    T, S, o, kept = v.shape[1], s["S0"].double(), torch.zeros_like(v), []
    for t in range(T):
        if t % CHUNK == 0 and c["op"] == "train":
            kept.append(S)
        S, _, _, o[:, t] = _token(S, q[:, t], k[:, t], v[:, t], la[:, t], b[:, t])
    got = {"out": _packed(o, s, c), "S_T": S}
    if c["op"] != "train":
        return got
    do, dS = x["dout"], s["dS_T"].double()
    dq, dk, dv, dla, db = (torch.zeros_like(y) for y in (q, k, v, la, b))
    for first in reversed(range(0, T, CHUNK)):
        S, seen = kept[first // CHUNK], []
        for t in range(first, min(T, first + CHUNK)):
            S, D, e, _ = _token(S, q[:, t], k[:, t], v[:, t], la[:, t], b[:, t])
            seen.append((t, S, D, e))
        for t, St, D, e in reversed(seen):
            dq[:, t] = torch.einsum("nhvk,nhv->nhk", St, do[:, t])
            dS = dS + torch.einsum("nhv,nhk->nhvk", do[:, t], q[:, t])
            w = torch.einsum("nhvk,nhk->nhv", dS, k[:, t])
            bt = b[:, t, :, None]
            db[:, t], de = (w * e).sum(-1), bt * w
            dv[:, t] = de
            dk[:, t] = torch.einsum("nhvk,nhv->nhk", dS, bt * e) - torch.einsum("nhvk,nhv->nhk", D, de)
            dS = dS - torch.einsum("nhv,nhk->nhvk", de, k[:, t])
            dla[:, t] = (dS * D).sum((-1, -2))
            dS = dS * la[:, t].exp()[..., None, None]
    dq, dk = (y.unflatten(2, (c["Hk"], rep)).sum(3) for y in (dq, dk))
    for m, y in (("q", dq), ("k", dk), ("v", dv), ("log_alpha", dla), ("beta", db)):
        got["d" + m] = _packed(y, s, c)
    got["dS0"] = dS
    return got


def _exact_step(s, c):
    r, rep = s["rows"], c["H"] // c["Hk"]
    q, k = (s[m][r].double().repeat_interleave(rep, 1) for m in ("q", "k"))
    pool, out = s["S"].double(), torch.zeros_like(s["v"], dtype=torch.float64)
    S, _, _, out[r] = _token(pool[s["at"]], q, k, s["v"][r].double(), s["log_alpha"][r].double(), s["beta"][r].double())
    pool[s["at"]] = S
    return {"out": out, "S": pool}


def _rms_grad(u, du):
    """Gradient of u / sqrt(mean u^2 + eps) for the incoming du."""
    m = u.shape[-1]
    root = torch.sqrt((u * u).sum(-1, keepdim=True) / m + EPS)
    return du / root - u * (u * du).sum(-1, keepdim=True) / (m * root ** 3)


def _rms(u):
    return u / torch.sqrt((u * u).sum(-1, keepdim=True) / u.shape[-1] + EPS)


def _exact_gated_norm(s, c):
    o, z, w = (s[m].double() for m in ("o", "z", "w"))
    silu = z * torch.sigmoid(z)
    if not c["back"]:
        return _rms(o) * w * silu
    dy = s["dy"].double()
    sg = torch.sigmoid(z)
    return {"do": _rms_grad(o, dy * w * silu), "dz": dy * _rms(o) * w * (sg + z * sg * (1 - sg)),
            "dw": (dy * _rms(o) * silu).sum((0, 1))}


def _exact_block_norm(s, c):
    x, w = s["x"].double(), s["w"].double()
    if c["post"]:
        z, wp, gate = (s[m].double() for m in ("z", "wp", "gate"))
    if not c["back"]:
        x = s["rho"] * x + gate * wp * _rms(z) if c["post"] else x
        return {"h": _rms(x) * w, "x2": x if c["post"] else None}
    dh = s["dh"].double()
    d = s["dx2"].double() + _rms_grad(x, dh * w)
    got = {"dx": s["rho"] * d, "dw": (dh * _rms(x)).sum(0), "dz": None, "dwp": None, "dgate": None}
    if c["post"]:
        got.update(dz=_rms_grad(z, d * gate * wp), dwp=(d * gate * _rms(z)).sum(0), dgate=(d * wp * _rms(z)).sum(0))
    return got
