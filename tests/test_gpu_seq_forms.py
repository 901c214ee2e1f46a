"""Forms of the sequence operators that a call's sizes and addresses choose, on the GPU against the fp64 oracle.

Results in fp32 are held to relative root mean squares, derived before any run (u = 2^-24).  Operands of three bf16
terms leave u of themselves, and the fp32 sums of a product, of its terms and of a chunk's step a few u each, which
decays with the state: 16 u for states and their gradients.  dbeta is a dot product of two such vectors: 32 u.
dlog_alpha is a difference of sums that nearly cancel, kept as pairs of floats, of terms each a few u off: 3e-6, a third
of what two terms leave of it.  Without a record S and [That; Phat] have two terms, 3e-6 of them in the mean square: 64 u
for S_T.  A lost term would leave 2^-9, or 2^-17, of an operand.  The fp32 kernels take a token's roundings and those of
64-token sums: 32 u, 64 u for dlog_alpha.
"""
import numpy as np
import pytest
import torch

from oracle import seq
from speculative_decoding_linear_gb300 import gdnspec
from test_gpu_seq import OUT, backward, check, forward, make, wide64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv,n", [(128, 128, 3), (256, 64, 6)])
def test_workspace_that_starts_on_16_bytes(dk, dv, n):
    """32 value columns a CTA (their rows are written by 32 bytes where the place allows it): equal bits either way."""
    lengths = [70, 65, 3, 64, 1, 90][:n]
    x, off = make(lengths, 8, 4, dk, dv, "bf16", seed=51)
    assert n * 8 * dv // 16 > 152
    out, S_T, ws, rec = forward(x, off, record=True)
    dout = torch.randn_like(out)
    d = backward(x, off, dout, None, ws, rec)
    moved = torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:]
    assert moved.data_ptr() % 32 == 16
    o2, S2 = torch.empty_like(out), torch.empty_like(S_T)
    gdnspec.gdn_seq_forward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["S0"], o2, S2, moved, offsets=off)
    plain, S_plain, _, _ = forward(x, off)
    assert torch.equal(o2, plain) and torch.equal(S2, S_plain)
    d2 = backward(x, off, dout, None, moved, rec)
    for m in OUT:
        assert torch.equal(d[m], d2[m]), m


U = 2.0 ** -24
RECORD = dict(S_T=16 * U, S0=16 * U, beta=32 * U, log_alpha=3e-6)
F32 = dict(out=32 * U, S_T=32 * U, q=32 * U, k=32 * U, v=32 * U, S0=32 * U, beta=32 * U, log_alpha=64 * U)


def near(got, ref, bound, what):
    e = np.sqrt(np.mean((got.double().cpu().numpy() - ref) ** 2)) / max(np.sqrt(np.mean(ref ** 2)), 1e-30)
    assert e <= bound, "%s: %.3g of its size off, allowed %.3g" % (what, e, bound)


def both_ways(lengths, H, Hk, dk, dv, dtype, bounds, seed, slow=False):
    x, off = make(lengths, H, Hk, dk, dv, dtype, seed=seed, slow=slow)
    out, S_T, ws, rec = forward(x, off, record=True)
    y, n = wide64(x), dk + dv + 64
    ref, refS = seq.seq_forward(**y, lengths=lengths)
    rng = np.random.default_rng(seed + 1)
    dout = torch.from_numpy(rng.standard_normal(out.shape)).to(out.dtype).cuda()
    dS = torch.from_numpy(0.1 * rng.standard_normal(S_T.shape)).float().cuda()
    d = backward(x, off, dout, dS, ws, rec)
    want = seq.seq_backward(**y, lengths=lengths, dout=dout.double().cpu().numpy(), dS_T=dS.double().cpu().numpy())
    check(out, ref, "out", n)
    for m in OUT:
        check(d[m], want[m], "d" + m, n * (H // Hk if m in ("q", "k") else 1))
    for m, got, r in [("out", out, ref), ("S_T", S_T, refS)] + [(m, d[m], want[m]) for m in OUT]:
        if m in bounds:
            near(got, r, bounds[m], m)


@pytest.mark.parametrize("dk,dv,H,Hk", [(64, 128, 8, 4), (128, 128, 8, 8), (192, 128, 8, 2), (256, 256, 8, 8), (48, 160, 8, 8), (80, 128, 8, 1)])
def test_record_and_gradients_with_32_columns(dk, dv, H, Hk):
    lengths = [130, 70, 0, 64]
    assert len(lengths) * H * dv // 16 > 152
    both_ways(lengths, H, Hk, dk, dv, "bf16", RECORD, seed=61)


@pytest.mark.parametrize("slow", [False, True])
@pytest.mark.parametrize("dk,dv", [(256, 256), (128, 64), (64, 48)])
def test_record_and_gradients_with_16_columns(dk, dv, slow):
    both_ways([330, 65], 2, 2, dk, dv, "bf16", RECORD, seed=63, slow=slow)


@pytest.mark.parametrize("slow", [False, True])
@pytest.mark.parametrize("lengths,H,Hk,dk,dv", [([130, 70, 0, 64], 8, 8, 256, 128), ([130, 70, 0, 64], 8, 4, 192, 128), ([300, 1], 2, 1, 192, 80),
                                                ([130, 70, 0, 64], 8, 2, 128, 128), ([330], 2, 2, 128, 128), ([130, 70, 0, 64], 8, 8, 64, 128),
                                                ([65, 190], 4, 1, 64, 64), ([200], 3, 3, 16, 48), ([400], 1, 1, 256, 256)])
def test_prefill_without_a_record(lengths, H, Hk, dk, dv, slow):
    x, off = make(lengths, H, Hk, dk, dv, "bf16", seed=67, slow=slow)
    out, S_T, _, _ = forward(x, off)
    ref, refS = seq.seq_forward(**wide64(x), lengths=lengths)
    check(out, ref, "out", dk + dv + 64)
    near(S_T, refS, 64 * U, "S_T")


@pytest.mark.parametrize("n,Hk,dk,dv", [(8, 8, 64, 128), (8, 2, 16, 128), (5, 4, 128, 128), (8, 8, 96, 64), (3, 8, 256, 96)])
def test_f32_with_two_rows_a_lane(n, Hk, dk, dv):
    lanes = 8 if dk <= 64 else 16 if dk <= 128 else 32
    lengths = [70, 3, 65, 0, 20, 1, 64, 9][:n]
    assert dv % (256 // lanes) == 0 and n * 8 * dv * lanes // 32 > 12 * 152
    both_ways(lengths, 8, Hk, dk, dv, "f32", F32, seed=71)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,dk,dv", [(4, 2, 128, 128), (2, 2, 64, 48), (8, 1, 256, 256)])
@pytest.mark.parametrize("first,lengths,total", [(5, [70, 0, 31], 140), (0, [66], 100), (64, [64, 1], 129), (7, [0, 0], 20)])
def test_tokens_of_no_sequence(first, lengths, total, H, Hk, dk, dv, dtype):
    """Tokens before the first offset and behind the last: zeros in every output, whatever lies in the inputs there."""
    x, _ = make([total], H, Hk, dk, dv, dtype, seed=73)
    x["S0"] = 0.1 * torch.randn((len(lengths), H, dv, dk), device="cuda")
    a, b = first, first + sum(lengths)
    dout = torch.randn_like(x["v"])
    for m in ("q", "k", "v", "log_alpha", "beta"):
        x[m][:a], x[m][b:] = float("nan"), float("inf")
    dout[:a], dout[b:] = float("inf"), float("nan")
    off = torch.tensor(np.cumsum([first] + lengths), dtype=torch.int32).cuda()
    inside = {m: (y if m == "S0" else y[a:b]).contiguous() for m, y in x.items()}
    y = wide64(inside)
    ref, refS = seq.seq_forward(**y, lengths=lengths)
    want = seq.seq_backward(**y, lengths=lengths, dout=dout[a:b].double().cpu().numpy(), dS_T=np.zeros_like(y["S0"]))
    out, S_T, ws, rec = forward(x, off, record=True)
    plain, _, _, _ = forward(x, off)
    ws.fill_(0xFF)
    d = backward(x, off, dout, None, ws, rec)
    n = dk + dv + 64
    for got, r, what in [(out, ref, "out"), (plain, ref, "out without a record")] + [(d[m], want[m], "d" + m) for m in OUT[:-1]]:
        check(got[a:b], r, what, n * (H // Hk))
        assert (got[:a] == 0).all() and (got[b:] == 0).all(), what
    check(S_T, refS, "S_T", n)
    check(d["S0"], want["S0"], "dS0", n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,H,Hk,dk,dv", [([130, 0, 65], 2, 1, 256, 256), ([70] * 4, 8, 8, 128, 128), ([5], 3, 3, 48, 16), ([0, 0], 2, 1, 64, 64)])
def test_forward_stays_in_its_workspace(lengths, H, Hk, dk, dv, dtype):
    x, off = make(lengths, H, Hk, dk, dv, dtype, seed=79)
    out, S_T, _, _ = forward(x, off)
    dims = (len(lengths), sum(lengths), H, Hk, dk, dv, dtype)
    n = gdnspec.gdn_seq_forward_workspace_bytes(*dims)
    room = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    for record in (None, gdnspec.empty_seq_record(*dims)):
        o2, S2 = torch.empty_like(out), torch.empty_like(S_T)
        gdnspec.gdn_seq_forward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["S0"], o2, S2, room[256:256 + n], offsets=off, record=record)
        assert gdnspec.gdn_last_error() == 0
        assert (room[:256] == 0x5A).all() and (room[256 + n:] == 0x5A).all()
        if record is None:
            assert torch.equal(out, o2) and torch.equal(S_T, S2)
    if dtype == "f32":
        o2, S2 = torch.empty_like(out), torch.empty_like(S_T)
        gdnspec.gdn_seq_forward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["S0"], o2, S2, None, offsets=off)
        assert torch.equal(out, o2) and torch.equal(S_T, S2)


@pytest.mark.parametrize("H,dk,dv", [(8, 256, 256), (2, 256, 256), (4, 128, 64), (4, 64, 48)])
def test_gate_gradients_would_show_a_lost_term(H, dk, dv):
    """Two terms of the state instead of three, everything else in 64 bits, leave 1.7e-6 to 2.6e-6 of dlog_alpha with these
    gates, three 3e-8: 24 u tells them apart (rounding of the dots' terms 8 u, of their sums and of w, o and eps as much each)."""
    both_ways([330, 65], H, H, dk, dv, "bf16", dict(RECORD, log_alpha=24 * U), seed=83)
