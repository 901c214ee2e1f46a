"""The gated delta rule over sequences, one token of it, and the block's norms in fp64 -- TEST INFRASTRUCTURE ONLY.

Written from the definitions, token by token, in numpy; shares no code with the CUDA library.

    S' = exp(log_alpha_t) S_{t-1},  e_t = v_t - S' k_t,  S_t = S' + beta_t e_t k_t^T,  o_t = S_t q_t

Value head h reads q/k head h // (H // Hk).  Sequences are packed; ``lengths`` gives their tokens.
"""
from __future__ import annotations

import numpy as np


def _spread(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def seq_forward(q, k, v, log_alpha, beta, S0, lengths):
    """(out [total, H, dv], S_T [n, H, dv, dk]); fp64 arrays."""
    H = v.shape[1]
    qh, kh = _spread(q, H), _spread(k, H)
    out, S_T, t = np.zeros_like(v), S0.copy(), 0
    for s, n in enumerate(lengths):
        S = S0[s].copy()
        for _ in range(n):
            S = S * np.exp(log_alpha[t])[:, None, None]
            e = v[t] - np.einsum("hvk,hk->hv", S, kh[t])
            S = S + np.einsum("hv,hk->hvk", beta[t][:, None] * e, kh[t])
            out[t] = np.einsum("hvk,hk->hv", S, qh[t])
            t += 1
        S_T[s] = S
    return out, S_T


def seq_backward(q, k, v, log_alpha, beta, S0, lengths, dout, dS_T):
    """Gradients of sum(out * dout) + sum(S_T * dS_T): dict of q, k, v, log_alpha, beta, S0."""
    H, Hk = v.shape[1], q.shape[1]
    qh, kh = _spread(q, H), _spread(k, H)
    dq, dk, dv = np.zeros_like(qh), np.zeros_like(kh), np.zeros_like(v)
    dla, db, dS0 = np.zeros_like(log_alpha), np.zeros_like(beta), dS_T.copy()
    first = 0
    for s, n in enumerate(lengths):
        kept, S = [], S0[s].copy()
        for t in range(first, first + n):
            D = S * np.exp(log_alpha[t])[:, None, None]
            e = v[t] - np.einsum("hvk,hk->hv", D, kh[t])
            S = D + np.einsum("hv,hk->hvk", beta[t][:, None] * e, kh[t])
            kept.append((D, e, S))
        dS = dS_T[s].copy()
        for t in reversed(range(first, first + n)):
            D, e, S = kept[t - first]
            dq[t] = np.einsum("hvk,hv->hk", S, dout[t])
            dS = dS + np.einsum("hv,hk->hvk", dout[t], qh[t])
            w = np.einsum("hvk,hk->hv", dS, kh[t])
            db[t] = (w * e).sum(-1)
            de = beta[t][:, None] * w
            dv[t] = de
            dk[t] = np.einsum("hvk,hv->hk", dS, beta[t][:, None] * e) - np.einsum("hvk,hv->hk", D, de)
            dS = dS - np.einsum("hv,hk->hvk", de, kh[t])
            dla[t] = (dS * D).sum((-1, -2))
            dS = dS * np.exp(log_alpha[t])[:, None, None]
        dS0[s] = dS
        first += n
    fold = lambda x: x.reshape(x.shape[0], Hk, H // Hk, x.shape[-1]).sum(2)  # noqa: E731
    return dict(q=fold(dq), k=fold(dk), v=dv, log_alpha=dla, beta=db, S0=dS0)


def _rms(x, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def _rms_back(x, dy, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return r * dy - x * r ** 3 * (x * dy).mean(-1, keepdims=True)


def gated_norm(o, gate, weight, eps):
    return weight * _rms(o, eps) * gate / (1.0 + np.exp(-gate))


def gated_norm_backward(o, gate, weight, dy, eps):
    sg = 1.0 / (1.0 + np.exp(-gate))
    d_o = _rms_back(o, dy * weight * gate * sg, eps)
    dgate = dy * weight * _rms(o, eps) * (sg + gate * sg * (1.0 - sg))
    return d_o, dgate, (dy * _rms(o, eps) * gate * sg).reshape(-1, o.shape[-1]).sum(0)


def block_norm(x, z, post_weight, gate, weight, eps, res_scale):
    if z is not None:
        x = res_scale * x + gate * post_weight * _rms(z, eps)
    return x, weight * _rms(x, eps)


def block_norm_backward(x_out, z, post_weight, gate, weight, dh, dx_out, eps, res_scale):
    """(dx, dz, dpost_weight, dgate, dweight); dz, dpost_weight, dgate None without z."""
    d = dx_out + _rms_back(x_out, dh * weight, eps)
    dw = (dh * _rms(x_out, eps)).sum(0)
    if z is None:
        return d, None, None, None, dw
    n = _rms(z, eps)
    return (res_scale * d, _rms_back(z, d * gate * post_weight, eps), (d * gate * n).sum(0), (d * post_weight * n).sum(0), dw)
