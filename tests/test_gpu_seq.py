"""Sequence and single-token operators on the GPU against the fp64 oracle.

Tolerances, before any run: with u = 2^-24, a product sum of n terms is off by at most n u times the sum of the
terms' sizes, which for a token is d_k, d_v and the 64 tokens of a chunk together; errors of earlier tokens pass
through a recurrence that does not grow them, and a factor 8 covers their sum and the largest element against the
root mean square.  An operand carried as two bf16 terms is off by 2^-16 of itself, below the same allowance.  A bf16
output adds its rounding, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from oracle import seq
from speculative_decoding_linear_gb300 import gdnspec

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
OUT = ("q", "k", "v", "log_alpha", "beta", "S0")


def close(got, ref, what, n):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), what
    if ref.size == 0:
        return
    return got, ref, 8 * n * 2.0 ** -24 * max(np.sqrt(np.mean(ref ** 2)), 1e-30)


def check(got, ref, what, n):
    r = close(got, ref, what, n)
    if r is None:
        return
    g, ref, tol = r
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    bad = np.abs(g - ref) > tol + half * np.abs(ref)
    assert not bad.any(), "%s: %d off, worst %.3g of rms, tolerance %.3g of rms" % (
        what, bad.sum(), np.abs(g - ref).max() / np.sqrt(np.mean(ref ** 2)), tol / np.sqrt(np.mean(ref ** 2)))


def make(lengths, H, Hk, dk, dv, dtype, seed=0, slow=False, wide=False):
    rng = np.random.default_rng(seed)
    total, n = sum(lengths), len(lengths)
    unit = lambda *s: (lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True))(rng.standard_normal(s))  # noqa: E731
    t = TYPES[dtype]
    c = lambda x, d=torch.float32: torch.from_numpy(np.ascontiguousarray(x)).to(d).cuda()  # noqa: E731
    la = -np.logaddexp(0, rng.uniform(-7, -4, (total, H)) if slow else rng.uniform(-6, 1, (total, H)))
    x = dict(q=c(unit(total, Hk, dk), t), k=c(unit(total, Hk, dk), t), v=c(rng.standard_normal((total, H, dv)), t),
             log_alpha=c(la), beta=c(rng.uniform(0.05, 0.95, (total, H))), S0=c(0.1 * rng.standard_normal((n, H, dv, dk))))
    if wide:      # q, k, v as columns of one projection
        both = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1)], 1)
        a, b = Hk * dk, 2 * Hk * dk
        x["q"], x["k"], x["v"] = both[:, :a].view(total, Hk, dk), both[:, a:b].view(total, Hk, dk), both[:, b:].view(total, H, dv)
    off = torch.tensor(np.cumsum([0] + list(lengths)), dtype=torch.int32).cuda()
    return x, off


def wide64(x):
    return {m: y.double().cpu().numpy() for m, y in x.items()}


def forward(x, off, S_T=True, record=False, S0=True):
    total, H, dv = x["v"].shape
    dims = (off.numel() - 1, total, H, x["q"].shape[1], x["q"].shape[2], dv, x["q"].dtype)
    out = torch.full((total, H, dv), float("nan"), dtype=x["q"].dtype, device="cuda")
    S = torch.full_like(x["S0"], float("nan")) if S_T else None
    ws = gdnspec.empty_seq_workspace(*dims)
    ws.fill_(0xFF)
    rec = gdnspec.empty_seq_record(*dims) if record else None
    gdnspec.gdn_seq_forward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["S0"] if S0 else None, out, S, ws,
                            offsets=off, record=rec)
    assert gdnspec.gdn_last_error() == 0
    return out, S, ws, rec


def backward(x, off, dout, dS_T, ws, rec, want_S0=True):
    d = {m: torch.full(x[m].shape, float("nan"), dtype=x[m].dtype, device="cuda") for m in OUT}
    gdnspec.gdn_seq_backward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], dout, dS_T, rec, d["q"], d["k"], d["v"],
                             d["log_alpha"], d["beta"], d["S0"] if want_S0 else None, ws, offsets=off)
    assert gdnspec.gdn_last_error() == 0
    return d


CASES = [  # lengths, H, Hk, dk, dv
    ([1], 1, 1, 256, 256),
    ([63, 64, 65], 2, 2, 256, 256),
    ([0, 5, 0, 200, 128, 0], 2, 1, 256, 256),
    ([130, 1], 4, 2, 128, 128),
    ([77, 190], 4, 1, 64, 64),
    ([100], 2, 1, 128, 256),
    ([100, 31], 2, 2, 256, 128),
    ([70, 3], 2, 2, 64, 128),
    ([90], 3, 1, 96, 96),
    ([2, 66], 2, 1, 16, 48),
    ([67], 2, 2, 192, 80),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_and_backward(case, dtype):
    lengths, H, Hk, dk, dv = CASES[case]
    x, off = make(lengths, H, Hk, dk, dv, dtype, seed=case, wide=case % 2 == 1)
    out, S_T, ws, rec = forward(x, off, record=True)
    y, n = wide64(x), dk + dv + 64
    ref, refS = seq.seq_forward(**y, lengths=lengths)
    check(out, ref, "out", n)
    check(S_T, refS, "S_T", n)
    rng = np.random.default_rng(case + 100)
    dout = torch.from_numpy(rng.standard_normal(out.shape)).to(out.dtype).cuda()
    dS = torch.from_numpy(0.1 * rng.standard_normal(S_T.shape)).float().cuda()
    d = backward(x, off, dout, dS, ws, rec)
    want = seq.seq_backward(**y, lengths=lengths, dout=dout.double().cpu().numpy(), dS_T=dS.double().cpu().numpy())
    for m in OUT:
        check(d[m], want[m], "d" + m, n * (H // Hk))


@pytest.mark.parametrize("dk,dv", [(256, 256), (128, 128), (48, 32)])
def test_long_slow_decay(dk, dv):
    lengths = [700, 333]
    x, off = make(lengths, 2, 1, dk, dv, "bf16", seed=7, slow=True)
    out, S_T, ws, rec = forward(x, off, record=True)
    y, n = wide64(x), dk + dv + 64
    ref, refS = seq.seq_forward(**y, lengths=lengths)
    check(out, ref, "out", n)
    check(S_T, refS, "S_T", n)
    dout = torch.randn_like(out)
    d = backward(x, off, dout, None, ws, rec)
    want = seq.seq_backward(**y, lengths=lengths, dout=dout.double().cpu().numpy(), dS_T=np.zeros_like(y["S0"]))
    for m in OUT:
        check(d[m], want[m], "d" + m, 2 * n)


@pytest.mark.parametrize("dk,dv", [(256, 256), (64, 64), (32, 48)])
def test_gates_at_their_ends(dk, dv):
    """log_alpha -inf (state forgotten), -80 and 0; beta 0 and 1; equal keys; large states."""
    lengths = [150]
    x, off = make(lengths, 2, 2, dk, dv, "bf16", seed=11)
    la, b = x["log_alpha"], x["beta"]
    la[5], la[40], la[64], la[100, 0] = float("-inf"), -80.0, float("-inf"), float("-inf")
    la[101:, 1] = 0.0
    b[::7], b[3::7] = 0.0, 1.0
    x["k"][70:80] = x["k"][70]
    x["S0"].mul_(1e3)
    out, S_T, ws, rec = forward(x, off, record=True)
    y, n = wide64(x), dk + dv + 64
    ref, refS = seq.seq_forward(**y, lengths=lengths)
    check(out, ref, "out", n)
    check(S_T, refS, "S_T", n)
    dout = torch.randn_like(out)
    d = backward(x, off, dout, None, ws, rec)
    y["log_alpha"] = np.maximum(y["log_alpha"], -800.0)       # 0 * inf is not a gradient
    want = seq.seq_backward(**y, lengths=lengths, dout=dout.double().cpu().numpy(), dS_T=np.zeros_like(y["S0"]))
    for m in OUT:
        check(d[m], want[m], "d" + m, n)


@pytest.mark.parametrize("dk,dv", [(256, 256), (32, 48)])
def test_optional_arguments_and_in_place(dk, dv):
    lengths = [65, 20]
    x, off = make(lengths, 2, 1, dk, dv, "bf16", seed=3)
    out, S_T, _, _ = forward(x, off)
    only, none, _, _ = forward(x, off, S_T=False)
    assert none is None and torch.equal(out, only)
    x0 = dict(x, S0=torch.zeros_like(x["S0"]))
    a, Sa, wsa, ra = forward(x0, off, record=True)
    b, Sb, wsb, rb = forward(x, off, S0=False, record=True)
    assert torch.equal(a, b) and torch.equal(Sa, Sb)
    S = x["S0"].clone()
    ws = gdnspec.empty_seq_workspace(2, 85, 2, 1, dk, dv, "bf16")
    o2 = torch.empty_like(out)
    gdnspec.gdn_seq_forward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], S, o2, S, ws, offsets=off)
    assert torch.equal(S, S_T) and torch.equal(o2, out)
    dout = torch.randn_like(out)
    d1 = backward(x, off, dout, torch.zeros_like(S), wsa, ra)
    d2 = backward(x, off, dout, None, wsb, rb, want_S0=False)
    for m in OUT[:-1]:
        assert torch.equal(d1[m], d2[m]), m
    # dS0 over dS_T
    dS = torch.randn_like(S)
    ref = backward(x, off, dout, dS, wsa, ra)
    d = {m: torch.empty_like(x[m]) for m in OUT}
    gdnspec.gdn_seq_backward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], dout, dS, ra, d["q"], d["k"], d["v"],
                             d["log_alpha"], d["beta"], dS, wsa, offsets=off)
    assert torch.equal(dS, ref["S0"])


def test_uniform_batch_is_the_packed_one():
    x, off = make([70] * 3, 2, 1, 128, 128, "bf16", seed=5)
    out, S_T, ws, _ = forward(x, off)
    y = {m: x[m].view(3, 70, *x[m].shape[1:]) for m in ("q", "k", "v", "log_alpha", "beta")}
    o, S = torch.empty_like(y["v"]), torch.empty_like(S_T)
    gdnspec.gdn_seq_forward(y["q"], y["k"], y["v"], y["log_alpha"], y["beta"], x["S0"], o, S, ws)
    assert torch.equal(o.view_as(out), out) and torch.equal(S, S_T)


def test_no_tokens():
    x, off = make([0, 0], 2, 1, 64, 64, "bf16")
    out, S_T, ws, rec = forward(x, off, record=True)
    assert torch.equal(S_T, x["S0"])
    dS = torch.randn_like(S_T)
    d = backward(x, off, out, dS, ws, rec)
    assert torch.equal(d["S0"], dS)


@pytest.mark.parametrize("off", [[0, 70, 60, 100], [0, 50, 101, 100], [-5, 20, 60, 100]])
@pytest.mark.parametrize("d", [64, 48])
def test_bad_offsets_are_reported(off, d):
    x, _ = make([40, 30, 30], 2, 2, d, d, "bf16")
    bad = torch.tensor(off, dtype=torch.int32).cuda()
    ws = gdnspec.empty_seq_workspace(3, 100, 2, 2, d, d, "bf16")
    rec = gdnspec.empty_seq_record(3, 100, 2, 2, d, d, "bf16")
    rec.zero_()
    out, S = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    gdnspec.gdn_seq_forward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["S0"], out, S, ws, offsets=bad, record=rec)
    assert gdnspec.gdn_last_error() == gdnspec.ERR_INDEX
    g = {m: torch.empty_like(x[m]) for m in OUT}
    gdnspec.gdn_seq_backward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], out, None, rec, g["q"], g["k"], g["v"],
                             g["log_alpha"], g["beta"], g["S0"], ws, offsets=bad)
    assert gdnspec.gdn_last_error() == gdnspec.ERR_INDEX
    assert gdnspec.gdn_last_error() == 0


def test_equal_bits_and_other_stream():
    x, off = make([300, 41], 4, 2, 256, 256, "bf16", seed=9)
    out, S, ws, rec = forward(x, off, record=True)
    dout = torch.randn_like(out)
    d = backward(x, off, dout, None, ws, rec)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, S2, ws2, rec2 = forward(x, off, record=True)
        d2 = backward(x, off, dout, None, ws2, rec2)
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(S, S2)
    for m in OUT:
        assert torch.equal(d[m], d2[m]), m


def test_forward_and_backward_in_a_graph():
    x, off = make([130, 60], 2, 1, 256, 256, "bf16", seed=21)
    out, S, ws, rec = forward(x, off, record=True)
    dout = torch.randn_like(out)
    d = backward(x, off, dout, None, ws, rec)
    o2, S2, g2 = torch.zeros_like(out), torch.zeros_like(S), {m: torch.zeros_like(x[m]) for m in OUT}

    def both():
        gdnspec.gdn_seq_forward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["S0"], o2, S2, ws, offsets=off, record=rec)
        gdnspec.gdn_seq_backward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], dout, None, rec, g2["q"], g2["k"], g2["v"],
                                 g2["log_alpha"], g2["beta"], g2["S0"], ws, offsets=off)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    for y in (o2, S2, *g2.values()):
        y.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(S, S2)
    for m in OUT:
        assert torch.equal(d[m], g2[m]), m


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 8, 8, 256, 256), (7, 4, 2, 128, 64), (5, 2, 1, 16, 48), (33, 3, 3, 192, 80)])
def test_step(B, H, Hk, dk, dv, dtype):
    x, _ = make([1] * B, H, Hk, dk, dv, dtype, seed=B)
    rng = np.random.default_rng(B)
    slots = B + 3
    idx = rng.permutation(slots)[:B].astype(np.int32)
    if B > 3:
        idx[2] = -1
    pool = torch.randn((slots, H, dv, dk), device="cuda")
    ref_pool = pool.double().cpu().numpy()
    out = torch.full((B, H, dv), float("nan"), dtype=x["v"].dtype, device="cuda")
    index = torch.from_numpy(idx).cuda()
    gdnspec.gdn_seq_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], pool, out, state_index=index)
    assert gdnspec.gdn_last_error() == 0
    y = wide64(x)
    y["S0"] = ref_pool[np.maximum(idx, 0)]
    ref, S = seq.seq_forward(**y, lengths=[1] * B)
    ref[idx < 0] = 0.0
    for b in range(B):
        if idx[b] >= 0:
            ref_pool[idx[b]] = S[b]
    check(out, ref, "out", dk + 2)
    check(pool, ref_pool, "S", dk + 2)


def test_step_identity_index_and_bad_index():
    x, _ = make([1] * 4, 2, 2, 64, 64, "bf16")
    S = torch.randn((4, 2, 64, 64), device="cuda")
    a, b = S.clone(), S.clone()
    out, o2 = torch.empty_like(x["v"]), torch.empty_like(x["v"])
    gdnspec.gdn_seq_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], a, out)
    gdnspec.gdn_seq_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], b, o2,
                         state_index=torch.arange(4, dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b) and torch.equal(out, o2) and gdnspec.gdn_last_error() == 0
    c = S.clone()
    gdnspec.gdn_seq_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], c, o2,
                         state_index=torch.tensor([0, 4, -2, 3], dtype=torch.int32, device="cuda"))
    assert gdnspec.gdn_last_error() == gdnspec.ERR_INDEX
    assert torch.equal(c[1:3], S[1:3]) and torch.equal(c[0], a[0]) and torch.equal(c[3], a[3])
    assert (o2[1:3] == 0).all()


def test_steps_follow_a_prompt():
    """A prompt and steps behind it give the states and outputs of the whole sequence."""
    x, off = make([70], 2, 1, 256, 256, "bf16", seed=31)
    out, S_T, _, _ = forward(x, off)
    head = {m: (y if m == "S0" else y[:64]) for m, y in x.items()}
    o, S, _, _ = forward(head, torch.tensor([0, 64], dtype=torch.int32).cuda())
    n = 256 + 256 + 64
    y = wide64(x)
    ref, refS = seq.seq_forward(**y, lengths=[70])
    for t in range(64, 70):
        o1 = torch.empty_like(x["v"][:1])
        gdnspec.gdn_seq_step(*(x[m][t:t + 1] for m in ("q", "k", "v", "log_alpha", "beta")), S, o1)
        check(o1, ref[t:t + 1], "step %d" % t, n)
    check(S, refS, "S", n)
    check(S_T, refS, "S_T", n)


def test_long_batch_gives_equal_bits_and_exact_gates():
    """More CTAs than the GPU has SMs, many chunks each: warps and CTAs drift apart, nothing may depend on it."""
    lengths = [1024, 700, 1000, 640]
    x, off = make(lengths, 8, 8, 256, 256, "bf16", seed=41)
    out, S_T, ws, rec = forward(x, off, record=True)
    dout, dS = torch.randn_like(out), 0.1 * torch.randn_like(S_T)
    d = backward(x, off, dout, dS, ws, rec)
    for _ in range(4):
        o2, S2, ws2, rec2 = forward(x, off, record=True)
        d2 = backward(x, off, dout, dS, ws2, rec2)
        assert torch.equal(out, o2) and torch.equal(S_T, S2)
        for m in OUT:
            assert torch.equal(d[m], d2[m]), m
    # one sequence and two heads against fp64
    a, b = sum(lengths[:1]), sum(lengths[:2])
    one = {m: (y[1:2, 2:4] if m == "S0" else y[a:b, 2:4]).double().cpu().numpy() for m, y in x.items()}
    want = seq.seq_backward(**one, lengths=lengths[1:2], dout=dout[a:b, 2:4].double().cpu().numpy(),
                            dS_T=dS[1:2, 2:4].double().cpu().numpy())
    for m in OUT:
        check(d[m][1:2, 2:4] if m == "S0" else d[m][a:b, 2:4], want[m], "d" + m, 256 + 256 + 64)


def test_rows_that_start_on_16_bytes_only():
    """Outputs and inputs whose rows are not 32-byte aligned take the narrower accesses."""
    lengths = [70, 65]
    x, off = make(lengths, 2, 2, 128, 128, "bf16", seed=13)
    out, S_T, ws, rec = forward(x, off, record=True)
    dout = torch.randn_like(out)
    d = backward(x, off, dout, None, ws, rec)

    def shifted(y):
        z = torch.empty(y.numel() + 8, dtype=y.dtype, device="cuda")[8:].view(y.shape)
        return z.copy_(y)
    x2 = dict(x, **{m: shifted(x[m]) for m in ("q", "k", "v")})
    o2, dv2, dq2, dk2 = shifted(out), shifted(out), shifted(x["q"]), shifted(x["k"])
    for y in (o2, dv2, dq2, dk2):
        y.zero_()
    S2 = torch.empty_like(S_T)
    gdnspec.gdn_seq_forward(x2["q"], x2["k"], x2["v"], x["log_alpha"], x["beta"], x["S0"], o2, S2, ws, offsets=off, record=rec)
    assert torch.equal(out, o2) and torch.equal(S_T, S2)
    g = {m: torch.empty_like(x[m]) for m in ("log_alpha", "beta", "S0")}
    gdnspec.gdn_seq_backward(x2["q"], x2["k"], x2["v"], x["log_alpha"], x["beta"], shifted(dout), None, rec, dq2, dk2, dv2, g["log_alpha"],
                             g["beta"], g["S0"], ws, offsets=off)
    assert torch.equal(dv2, d["v"]) and torch.equal(dq2, d["q"]) and torch.equal(dk2, d["k"])
    for m in g:
        assert torch.equal(g[m], d[m])


def test_what_lies_behind_a_sequence_stays_out():
    """NaN and infinities in one sequence's tokens reach no other sequence."""
    lengths = [70, 64, 33]
    x, off = make(lengths, 2, 1, 128, 128, "bf16", seed=17)
    out, S_T, ws, rec = forward(x, off, record=True)
    dout = torch.randn_like(out)
    d = backward(x, off, dout, None, ws, rec)
    y = {m: v.clone() for m, v in x.items()}
    y["q"][70:134], y["k"][70:100], y["v"][80:134] = float("nan"), float("inf"), float("nan")
    y["beta"][70:], y["log_alpha"][70:134] = x["beta"][70:], x["log_alpha"][70:134]
    dout2 = dout.clone()
    dout2[70:134] = float("nan")
    o2, S2, ws2, rec2 = forward(y, off, record=True)
    d2 = backward(y, off, dout2, None, ws2, rec2)
    clean = torch.cat([torch.arange(70), torch.arange(134, 167)]).cuda()
    assert torch.equal(out[clean], o2[clean]) and torch.equal(S_T[[0, 2]], S2[[0, 2]])
    for m in OUT[:-1]:
        assert torch.equal(d[m][clean], d2[m][clean]), m
    assert torch.equal(d["S0"][[0, 2]], d2["S0"][[0, 2]])


def test_order_of_sequences_changes_nothing():
    """More CTAs than run at once: the longest sequences go first, and each comes out as it does alone."""
    lengths = [3, 130, 0, 64, 200, 1, 130, 70, 5, 260, 31, 90]
    x, off = make(lengths, 4, 2, 128, 128, "bf16", seed=23)
    out, S_T, ws, rec = forward(x, off, record=True)
    d = backward(x, off, torch.ones_like(out), torch.ones_like(S_T), ws, rec)
    for s, n in enumerate(lengths):
        a, b = int(off[s]), int(off[s + 1])
        y = {m: (v[s:s + 1] if m == "S0" else v[a:b]).contiguous() for m, v in x.items()}
        o1, S1, ws1, rec1 = forward(y, torch.tensor([0, n], dtype=torch.int32).cuda(), record=True)
        assert torch.equal(out[a:b], o1) and torch.equal(S_T[s:s + 1], S1), s
        if n:
            d1 = backward(y, torch.tensor([0, n], dtype=torch.int32).cuda(), torch.ones_like(o1), torch.ones_like(S1), ws1, rec1)
            assert torch.equal(d["v"][a:b], d1["v"]) and torch.equal(d["S0"][s:s + 1], d1["S0"]), s
