"""Two Gated DeltaNet blocks: a training step, prefill of packed prompts, single-token decode, and a draft tree.

Run on a GB300:  python examples/gdn_blocks.py

Each block is  x -> x + gate * post_norm(W_o gated_norm(gdn(q, k, v), z))  with its pre-norm in front; between two
blocks the residual, the post-norm and the next pre-norm are one call (``gdn_block_norm``).  The dense projections are
torch products; there is no convolution.  Everything else runs in the library:

* ``train_step``   forward and backward over packed sequences, and an update of the weights
* ``prefill``      the same forward pass, keeping each layer's state
* ``decode``       one token for each sequence, states updated in place
* ``verify``       a draft tree from a prefilled state, as the verifier of a speculative decoder sees it
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_linear_gb300 import gdnspec  # noqa: E402

HID, H, HK, DK, DV, LAYERS, EPS = 512, 4, 2, 128, 128, 2, 1e-6
BF16 = torch.bfloat16


def weights(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s, std=0.02, mean=0.0: (torch.randn(s, generator=g, device="cuda") * std + mean).to(BF16)  # noqa: E731
    rows = 2 * HK * DK + 2 * H * DV + 2 * H
    one = lambda d: rand(d, std=0.05, mean=1.0)  # noqa: E731
    layers = [dict(w_in=rand(HID, rows, std=HID ** -0.5), w_o=rand(H * DV, HID, std=(H * DV) ** -0.5), pre=one(HID), post=one(HID),
                   gate=rand(HID, std=0.05, mean=0.5), out=one(DV)) for _ in range(LAYERS)]
    return layers, one(HID)


def split(y):
    """q, k (unit rows), v, z, log decay and write strength of projected rows [n, .]."""
    q, k, v, z, a, b = y.split([HK * DK, HK * DK, H * DV, H * DV, H, H], dim=1)
    unit = lambda x: F.normalize(x.float().view(-1, HK, DK), dim=-1).to(BF16)  # noqa: E731
    return (unit(q), unit(k), v.reshape(-1, H, DV).contiguous(), z.reshape(-1, H, DV).contiguous(), -F.softplus(a.float()).contiguous(),
            torch.sigmoid(b.float()).contiguous())


def norm_in(x, w):
    h = torch.empty_like(x)
    gdnspec.gdn_block_norm(x, None, None, None, w, None, h, eps=EPS)
    return h


def between(x, z, p, next_w):
    x2, h = torch.empty_like(x), torch.empty_like(x)
    gdnspec.gdn_block_norm(x, z, p["post"], p["gate"], next_w, x2, h, eps=EPS)
    return x2, h


def gated(o, z, w):
    y = torch.empty_like(z)
    gdnspec.gdn_gated_norm(o, z, w, y, eps=EPS)
    return y


def forward(params, x, offsets, states=None, keep=False):
    """Rows x [total, HID] of packed sequences through all blocks: (h after the last norm, states, what backward needs)."""
    layers, last = params
    n, total = offsets.numel() - 1, x.shape[0]
    dims = (n, total, H, HK, DK, DV, BF16)
    ws = gdnspec.empty_seq_workspace(*dims, backward=keep)
    h, out_states, kept = norm_in(x, layers[0]["pre"]), [], []
    for i, p in enumerate(layers):
        q, k, v, z, la, b = split(h @ p["w_in"])
        o, S = torch.empty_like(v), torch.empty(n, H, DV, DK, device="cuda")
        rec = gdnspec.empty_seq_record(*dims) if keep else None
        gdnspec.gdn_seq_forward(q, k, v, la, b, None if states is None else states[i], o, S, ws, offsets=offsets, record=rec)
        m = gated(o, z, p["out"]).flatten(1) @ p["w_o"]
        next_w = layers[i + 1]["pre"] if i + 1 < LAYERS else last
        x2, h2 = between(x, m, p, next_w)
        kept.append(dict(h=h, q=q, k=k, v=v, z=z, la=la, b=b, o=o, rec=rec, m=m, x2=x2, next_w=next_w))
        out_states.append(S)
        x, h = x2, h2
    return h, out_states, (kept, ws)


def backward(params, x, offsets, kept_ws, dh):
    """Gradients of all weights for the gradient dh of forward's result: one dict a layer, and the last norm's."""
    layers, _ = params
    kept, ws = kept_ws
    total = x.shape[0]
    f32 = lambda d: torch.empty(d, device="cuda")  # noqa: E731
    nws, gws = gdnspec.empty_norm_workspace(total, HID), gdnspec.empty_norm_workspace(total * H, DV)
    grads, dx2, last = [None] * LAYERS, None, None
    for i in reversed(range(LAYERS)):
        p, s = layers[i], kept[i]
        dx, dm, g = torch.empty_like(s["x2"]), torch.empty_like(s["m"]), {}
        dnext = f32(HID)
        g["post"], g["gate"] = f32(HID), f32(HID)
        gdnspec.gdn_block_norm_backward(s["x2"], s["m"], p["post"], p["gate"], s["next_w"], dh, dx2, dx, dm, g["post"], g["gate"], dnext,
                                        nws, eps=EPS)
        if i + 1 < LAYERS:
            grads[i + 1]["pre"] = dnext
        else:
            last = dnext
        y = gated(s["o"], s["z"], p["out"]).flatten(1)
        g["w_o"] = y.T @ dm
        do, dz, g["out"] = torch.empty_like(s["o"]), torch.empty_like(s["z"]), f32(DV)
        gdnspec.gdn_gated_norm_backward(s["o"], s["z"], p["out"], (dm @ p["w_o"].T).view(total, H, DV), do, dz, g["out"], gws, eps=EPS)
        d = {m: torch.empty_like(s[m]) for m in ("q", "k", "v", "la", "b")}
        gdnspec.gdn_seq_backward(s["q"], s["k"], s["v"], s["la"], s["b"], do, None, s["rec"], d["q"], d["k"], d["v"], d["la"], d["b"], None,
                                 ws, offsets=offsets)
        # through the unit rows and the gates' functions, which torch differentiates
        yin = (s["h"] @ p["w_in"]).detach().requires_grad_()
        with torch.enable_grad():
            outs = split(yin)
        dy, = torch.autograd.grad(outs, yin, (d["q"], d["k"], d["v"], dz, d["la"], d["b"]))
        g["w_in"] = s["h"].T @ dy
        grads[i], dh, dx2 = g, dy @ p["w_in"].T, dx
    dpre, dfirst = torch.empty_like(x), f32(HID)
    gdnspec.gdn_block_norm_backward(x, None, None, None, layers[0]["pre"], dh, None, dpre, None, None, None, dfirst, nws, eps=EPS)
    grads[0]["pre"] = dfirst
    return grads, last


def loss_of(h, target):
    return ((h.float() - target.float()) ** 2).mean()


def train_step(params, x, offsets, target, lr):
    h, _, kept = forward(params, x, offsets, keep=True)
    loss = loss_of(h, target)
    dh = ((h.float() - target.float()) * (2.0 / h.numel())).to(BF16)
    grads, last = backward(params, x, offsets, kept, dh)
    for p, g in zip(params[0], grads):
        for name in g:
            p[name].copy_((p[name].float() - lr * g[name].float()).to(BF16))
    params[1].copy_((params[1].float() - lr * last).to(BF16))
    return loss.item()


def decode(params, x, states, index):
    """One token a sequence, rows x [B, HID]; states: each layer's pool, updated in place at `index`."""
    layers, last = params
    h = norm_in(x, layers[0]["pre"])
    for i, p in enumerate(layers):
        q, k, v, z, la, b = split(h @ p["w_in"])
        o = torch.empty_like(v)
        gdnspec.gdn_seq_step(q, k, v, la, b, states[i], o, state_index=index)
        x, h = between(x, gated(o, z, p["out"]).flatten(1) @ p["w_o"], p, layers[i + 1]["pre"] if i + 1 < LAYERS else last)
    return h


def verify(params, x, parent, state):
    """The first block's recurrence for a draft tree's rows x [N, HID] from one sequence's state: outputs [N, H, DV] fp32."""
    N = x.shape[0]
    q, k, v, _, la, b = split(norm_in(x, params[0][0]["pre"]) @ params[0][0]["w_in"])
    spread = lambda t: t.repeat_interleave(H // HK, 1)[None].contiguous()  # noqa: E731
    out = torch.empty(1, N, H, DV, device="cuda")
    fac = gdnspec.empty_factors(1, N, H, DK, DV, BF16)
    ws = gdnspec.empty_workspace(1, N, H, DK, DV)
    gdnspec.gdn_tree_verify(spread(q), spread(k), v[None].contiguous(), la.exp()[None].contiguous(), b[None].contiguous(), parent[None], state, out,
                            fac, ws)
    return out[0]


@torch.no_grad()
def main():
    torch.manual_seed(0)
    params = weights()
    lengths = [300, 0, 77, 451]
    offsets = torch.tensor([0, 300, 300, 377, 828], dtype=torch.int32, device="cuda")
    x = torch.randn(828, HID, device="cuda").to(BF16)
    target = torch.randn(828, HID, device="cuda").to(BF16) * 0.5
    losses = [train_step(params, x, offsets, target, lr=20.0) for _ in range(6)]
    print("training: loss " + " ".join("%.4f" % v for v in losses))

    # prompts without their last three tokens, then those one by one: the whole prompts' results
    whole, states, _ = forward(params, x, offsets)
    ends = [e for e, n in zip(offsets[1:].tolist(), lengths) if n]
    keep = torch.cat([torch.arange(e - n, e - 3, device="cuda") for e, n in zip(offsets[1:].tolist(), lengths) if n])
    short = torch.tensor([0, 297, 371, 819], dtype=torch.int32, device="cuda")
    _, pool, _ = forward(params, x[keep].contiguous(), short)
    index = torch.arange(3, dtype=torch.int32, device="cuda")
    for t in range(3, 0, -1):
        h = decode(params, x[torch.tensor([e - t for e in ends], device="cuda")].contiguous(), pool, index)
    step_err = ((h - whole[torch.tensor([e - 1 for e in ends], device="cuda")]).float().norm() / h.float().norm()).item()
    state_err = max(((a - b[[0, 2, 3]]).norm() / a.norm()).item() for a, b in zip(pool, states))
    print("decode after prefill: outputs %.1e, states %.1e from the whole prompts'" % (step_err, state_err))

    # a chain of drafts verified from the first prompt's state, and the same tokens as a prompt
    drafts = torch.randn(5, HID, device="cuda").to(BF16)
    o = verify(params, drafts, torch.arange(-1, 4, dtype=torch.int32, device="cuda"), states[0][:1].contiguous())
    q, k, v, _, la, b = split(norm_in(drafts, params[0][0]["pre"]) @ params[0][0]["w_in"])
    o2 = torch.empty_like(v)
    ws = gdnspec.empty_seq_workspace(1, 5, H, HK, DK, DV, BF16)
    gdnspec.gdn_seq_forward(q, k, v, la, b, states[0][:1].contiguous(), o2, None, ws)
    tree_err = ((o - o2.float()).norm() / o.norm()).item()
    print("draft chain verified from a prefilled state: %.1e from the sequence operator" % tree_err)
    assert gdnspec.gdn_last_error() == 0
    return losses, step_err, state_err, tree_err


if __name__ == "__main__":
    main()
