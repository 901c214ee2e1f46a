"""Decay-gated linear attention over sequences, one token of it, and rotary positions in fp64 -- TEST INFRASTRUCTURE ONLY.

Written from the definitions, token by token, in numpy; shares no code with the CUDA library.

    S_t = exp(log_alpha_t) S_{t-1} + beta_t v_t k_t^T,  o_t = S_t q_t

Value head h reads q/k head h // (H // Hk).  Sequences are packed; ``lengths`` gives their tokens.
"""
from __future__ import annotations

import numpy as np


def _spread(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def forward(q, k, v, log_alpha, beta, S0, lengths):
    """(out [total, H, dv], S_T [n, H, dv, dk]); fp64 arrays."""
    H = v.shape[1]
    qh, kh = _spread(q, H), _spread(k, H)
    out, S_T, t = np.zeros_like(v), S0.copy(), 0
    for s, n in enumerate(lengths):
        S = S0[s].copy()
        for _ in range(n):
            S = S * np.exp(log_alpha[t])[:, None, None] + (beta[t][:, None] * v[t])[:, :, None] * kh[t][:, None, :]
            out[t] = np.matmul(S, qh[t][:, :, None])[:, :, 0]
            t += 1
        S_T[s] = S
    return out, S_T


def backward(q, k, v, log_alpha, beta, S0, lengths, dout, dS_T):
    """Gradients of sum(out * dout) + sum(S_T * dS_T): dict of q, k, v, log_alpha, beta, S0."""
    H, Hk = v.shape[1], q.shape[1]
    qh, kh = _spread(q, H), _spread(k, H)
    dq, dk, dv = np.zeros_like(qh), np.zeros_like(kh), np.zeros_like(v)
    dla, db, dS0 = np.zeros_like(log_alpha), np.zeros_like(beta), dS_T.copy()
    every, first = 32, 0
    for s, n in enumerate(lengths):
        token = lambda S, t: (lambda D: (D, D + (beta[t][:, None] * v[t])[:, :, None] * kh[t][:, None, :]))(  # noqa: E731
            S * np.exp(log_alpha[t])[:, None, None])
        starts, S = [], S0[s].copy()
        for t in range(first, first + n):
            if (t - first) % every == 0:
                starts.append(S)
            S = token(S, t)[1]
        dS = dS_T[s].copy()
        for b in reversed(range(len(starts))):
            S, kept = starts[b], []
            for t in range(first + b * every, min(first + n, first + (b + 1) * every)):
                D, S = token(S, t)
                kept.append((t, D, S))
            for t, D, S in reversed(kept):
                dq[t] = np.matmul(dout[t][:, None, :], S)[:, 0]
                dS = dS + dout[t][:, :, None] * qh[t][:, None, :]
                w = np.matmul(dS, kh[t][:, :, None])[:, :, 0]
                db[t], dv[t] = (w * v[t]).sum(-1), beta[t][:, None] * w
                dk[t] = beta[t][:, None] * np.matmul(v[t][:, None, :], dS)[:, 0]
                dla[t] = (dS * D).sum((-1, -2))
                dS = dS * np.exp(log_alpha[t])[:, None, None]
        dS0[s] = dS
        first += n
    fold = lambda x: x.reshape(x.shape[0], Hk, H // Hk, x.shape[-1]).sum(2)  # noqa: E731
    return dict(q=fold(dq), k=fold(dk), v=dv, log_alpha=dla, beta=db, S0=dS0)


TURN = np.longdouble("6.28318530717958647692528676655900576839")


def rotary(x, positions, inv_freq, scale=1.0, interleaved=False, inverse=False):
    """x [total, heads, d] turned by positions [total] times inv_freq [rot / 2], the frequencies as they are given."""
    rot = 2 * len(inv_freq)
    # whole turns taken off in extended precision: a far position's angle in 64 bits would be off by 1e-16 of itself
    angle = np.longdouble(positions)[:, None] * np.longdouble(inv_freq)[None, :]
    angle = (angle - np.round(angle / TURN) * TURN).astype(np.float64)
    turn = scale * np.exp(1j * (-angle if inverse else angle))[:, None, :]
    y = np.array(x, np.float64)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = (y[..., a] + 1j * y[..., b]) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def rotary_frequencies(rot, base, factor, original, low, high):
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    kept = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0) if original > 0 else np.zeros_like(f)
    return f * kept + f / factor * (1.0 - kept)
