"""Decay-gated linear attention over sequences on the GPU: sizes and uses at the edges of its kernels, against 64 bits.

Tolerances, before any run.

bf16 outputs.  Before its own rounding a value is off by what the operands' two bf16 terms leave, 2^-17 of each of its
terms and less in the sum, and by fp32 sums.  A rounding to bf16 is off by at most 2^-8 of the power of two below the
value, evenly spread, so 2^-8 / sqrt(3) of the value in the root mean square at most: the array is held to that and one
per cent for the spread of the sample (at least 10^4 values) and all else.  (Scores or states rounded to bf16 once would
add as much again, sqrt(2) of it where the values are spread evenly over their powers of two.)

fp32 outputs: the array is held to 4e-6 of its norm, 64 x 2^-24: the square root of 4096 terms' roundings.
"""
import numpy as np
import pytest
import torch

from speculative_decoding_linear_gb300 import gdnspec

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "log_alpha", "beta", "S0")


def inputs(lengths, H, Hk, dk, dv, seed, slow=False, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total, n = sum(lengths), len(lengths)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731

    def placed(y):         # 16 bytes behind a 32-byte boundary where shift is 8
        store = torch.empty(y.numel() + 16, dtype=torch.bfloat16, device="cuda")
        z = store[shift:shift + y.numel()].view(y.shape)
        z.copy_(y)
        return z

    unit = lambda y: y / y.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=placed(unit(rand(total, Hk, dk))), k=placed(unit(rand(total, Hk, dk))), v=placed(rand(total, H, dv)))
    u = torch.rand(total, H, generator=g, device="cuda")
    x["log_alpha"] = -(1e-5 + 2e-3 * u) if slow else -torch.nn.functional.softplus(7 * u - 6)
    x["beta"] = 0.05 + 0.95 * torch.rand(total, H, generator=g, device="cuda")
    x["S0"] = 0.1 * rand(n, H, dv, dk)
    return x, torch.tensor(np.cumsum([0] + list(lengths)), dtype=torch.int32, device="cuda"), placed(rand(total, H, dv)), rand(n, H, dv, dk)


def plain(x, lengths, dout=None, dS=None):
    """Each sequence at once: o = e^g S q + (masked, decayed scores) (beta v); gradients by differentiation."""
    p = {m: x[m].double().requires_grad_(dout is not None) for m in NAMES}
    rep = x["v"].shape[1] // x["q"].shape[1]
    outs, ends, b = [], [], 0
    for s, n in enumerate(lengths):
        q, k = (p[m][b:b + n].repeat_interleave(rep, 1).transpose(0, 1) for m in "qk")
        w = (p["beta"][b:b + n, :, None] * p["v"][b:b + n]).transpose(0, 1)
        g = p["log_alpha"][b:b + n].transpose(0, 1).cumsum(1)
        d = g[:, :, None] - g[:, None, :]
        m = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        f = d.masked_fill(~m, 0).exp() * m
        S = p["S0"][s]
        outs.append((g.exp()[..., None] * (q @ S.transpose(1, 2)) + (q @ k.transpose(1, 2) * f) @ w).transpose(0, 1))
        G = g[:, -1] if n else torch.zeros(S.shape[0], dtype=torch.double, device="cuda")
        ends.append(G.exp()[:, None, None] * S + w.transpose(1, 2) @ ((G[:, None] - g).exp()[..., None] * k))
        b += n
    want = {"out": torch.cat(outs), "S_T": torch.stack(ends)}
    if dout is not None:
        ((want["out"] * dout.double()).sum() + (want["S_T"] * dS.double()).sum()).backward()
        want.update({"d" + m: p[m].grad for m in NAMES})
    return {m: y.detach() for m, y in want.items()}


def outputs(x, shift=0):
    def like(y):
        store = torch.full((y.numel() + 16,), float("nan"), dtype=y.dtype, device="cuda")
        at = shift if y.dtype == torch.bfloat16 else 0
        return store[at:at + y.numel()].view(y.shape)

    d = {"out": like(x["v"]), "S_T": like(x["S0"])}
    d.update({"d" + m: like(x[m]) for m in NAMES})
    return d


def both(x, off, dout, dS, d, ws, rec):
    gdnspec.gdn_linear_seq_forward(*(x[m] for m in NAMES), d["out"], d["S_T"], ws, offsets=off, record=rec)
    gdnspec.gdn_linear_seq_backward(*(x[m] for m in NAMES[:-1]), dout, dS, rec, *(d["d" + m] for m in NAMES), ws, offsets=off)


def held(got, want, what):
    rel = ((got.double() - want).norm() / want.norm()).item()
    assert rel <= (1.01 * 2.0 ** -8 / 3 ** 0.5 if got.dtype == torch.bfloat16 else 4e-6), "%s: %.3g of the norm" % (what, rel)


# many turns of the grid: short sequences of all lengths, empty ones among them; whole segments and ragged ones; one long
# sequence with slow decays, whose states add up over 24 segments; one sequence of one head
CASES = [([(37 * i) % 301 for i in range(150)], (8, 4, 64, 64), False), ([512] * 9 + [511, 513, 1024, 130, 1, 0, 640], (8, 2, 128, 128), False),
         ([700, 2100, 90], (4, 4, 256, 256), False), ([12200], (2, 1, 128, 128), True), ([4100], (1, 1, 64, 256), False)]


@pytest.mark.parametrize("shift", [0, 8])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_many_items_in_their_own_rounding(i, shift):
    lengths, dims, slow = CASES[i]
    x, off, dout, dS = inputs(lengths, *dims, seed=i, slow=slow, shift=shift)
    full = (len(lengths), sum(lengths), *dims, torch.bfloat16)
    d, ws, rec = outputs(x, shift), gdnspec.empty_linear_seq_workspace(*full).fill_(0xff), gdnspec.empty_linear_seq_record(*full).fill_(0xff)
    both(x, off, dout, dS, d, ws, rec)
    # and a forward pass that keeps no record
    alone = {"out": torch.empty_like(x["v"]), "S_T": torch.empty_like(x["S0"])}
    ws1 = gdnspec.empty_linear_seq_workspace(*full, backward=False).fill_(0xff)
    gdnspec.gdn_linear_seq_forward(*(x[m] for m in NAMES), alone["out"], alone["S_T"], ws1, offsets=off)
    assert gdnspec.gdn_last_error() == gdnspec.OK
    want = plain(x, lengths, dout, dS)
    for m in want:
        held(d[m], want[m], m)
    held(alone["out"], want["out"], "out, no record")
    assert torch.equal(alone["S_T"], d["S_T"])


def test_two_captured_graphs_share_a_workspace():
    shapes = [([300, 1300], (4, 2, 128, 128)), ([64, 5, 900], (2, 2, 64, 192))]
    sets = [(inputs(*s[:1], *s[1], seed=7 + i), (len(s[0]), sum(s[0]), *s[1], torch.bfloat16)) for i, s in enumerate(shapes)]
    ws = max((gdnspec.empty_linear_seq_workspace(*f) for _, f in sets), key=lambda w: w.numel())
    runs = []
    for (x, off, dout, dS), full in sets:
        rec, d = gdnspec.empty_linear_seq_record(*full), outputs(x)
        both(x, off, dout, dS, d, ws, rec)
        torch.cuda.synchronize()
        want = {m: y.clone() for m, y in d.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both(x, off, dout, dS, d, ws, rec)
        runs.append((graph, d, want, rec))
    for _ in range(3):
        for graph, d, _, _ in runs:
            for y in d.values():
                y.fill_(float("nan"))
            graph.replay()
    torch.cuda.synchronize()
    for _, d, want, _ in runs:
        for m in want:
            assert torch.equal(d[m], want[m]), m


def test_rows_do_not_depend_on_later_tokens():
    """Outputs of a prefix are those of the whole, to the bit: masked scores, however large, weigh nothing."""
    x, off, _, _ = inputs([777], 2, 2, 128, 128, seed=3)
    want = torch.empty_like(x["v"])
    ws = gdnspec.empty_linear_seq_workspace(1, 777, 2, 2, 128, 128, torch.bfloat16, backward=False)
    S_T = torch.empty_like(x["S0"])
    gdnspec.gdn_linear_seq_forward(*(x[m] for m in NAMES), want, S_T, ws, offsets=off)
    for m in "qkv":
        x[m][600:] *= 2.0 ** 40
    x["log_alpha"][600:] = -float("inf")
    got = torch.empty_like(want)
    gdnspec.gdn_linear_seq_forward(*(x[m] for m in NAMES), got, S_T, ws, offsets=off)
    assert torch.equal(got[:600], want[:600])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_decay_of_zero_starts_anew(dtype):
    """log_alpha = -inf at a token: from there on as a sequence of its own from a state of zero, gradients too."""
    lengths, cut = [900], 333
    x, off, dout, dS = inputs(lengths, 2, 1, 64, 64, seed=11)
    x, dout = {m: y.to(dtype) if m in "qkv" else y for m, y in x.items()}, dout.to(dtype)
    x["log_alpha"][cut] = -float("inf")
    full = (1, 900, 2, 1, 64, 64, dtype)
    d = outputs(x)
    both(x, off, dout, dS, d, gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full))
    parts = [{m: (y[:cut] if i == 0 else y[cut:]) if m != "S0" else (y if i == 0 else 0 * y) for m, y in x.items()} for i in range(2)]
    parts[1]["log_alpha"] = parts[1]["log_alpha"].clone()
    parts[1]["log_alpha"][0] = 0.0
    a = plain(parts[0], [cut], dout[:cut], 0 * dS)
    b = plain(parts[1], [900 - cut], dout[cut:], dS)
    for m in ("out", "dq", "dk", "dv", "dbeta"):
        held(d[m], torch.cat([a[m], b[m]]), m)
    held(d["S_T"], b["S_T"], "S_T")
    held(d["dS0"], a["dS0"], "dS0")
    # Nothing passes the cut, so its gradient is zero.  It is formed as sums over the rows from the cut on minus sums over the
    # columns: E_ts of each pair behind it stands in one of either, rounded apart, so the two cancel to their roundings only,
    # as many as any gradient of the array has: sqrt(4096) x 2^-24 of the sums' size, which is that of the largest gradient.
    assert d["dlog_alpha"][cut].abs().max() <= 4e-6 * d["dlog_alpha"].abs().max()
    keep = torch.arange(900, device="cuda") != cut
    held(d["dlog_alpha"][keep], torch.cat([a["dlog_alpha"], b["dlog_alpha"]])[keep], "dlog_alpha")


def test_rows_past_32_bits_of_offsets():
    """The last sequence of a batch whose rows lie beyond 2^31 elements: to the bit what it is alone."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("takes 70 GB")
    dims, lengths = (8, 8, 256, 256), [(1 << 20) + 64, 700]
    total = sum(lengths)
    x = {m: torch.empty(total, 8, 256, dtype=torch.bfloat16, device="cuda").normal_(0, 1 / 16) for m in "qkv"}
    x["log_alpha"] = -torch.rand(total, 8, device="cuda")
    x["beta"] = torch.rand(total, 8, device="cuda")
    x["S0"] = 0.1 * torch.randn(2, 8, 256, 256, device="cuda")
    dout, dS = torch.empty_like(x["v"]).normal_(), torch.randn(2, 8, 256, 256, device="cuda")

    def run(x, lengths, dout, dS):
        full = (len(lengths), sum(lengths), *dims, torch.bfloat16)
        d = {"out": torch.empty_like(x["v"]), "S_T": torch.empty_like(x["S0"])}
        d.update({"d" + m: torch.empty_like(x[m]) for m in NAMES})
        off = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device="cuda")
        both(x, off, dout, dS, d, gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full))
        assert gdnspec.gdn_last_error() == gdnspec.OK
        return d

    got = run(x, lengths, dout, dS)
    want = run({m: (y[1:] if m == "S0" else y[lengths[0]:]).contiguous() for m, y in x.items()}, lengths[1:], dout[lengths[0]:].contiguous(), dS[1:].contiguous())
    for m in want:
        y = got[m][1:] if m in ("S_T", "dS0") else got[m][lengths[0]:]
        assert torch.equal(y, want[m]), m


@pytest.mark.parametrize("dims", [(4, 2, 64, 64), (2, 2, 64, 64)])
def test_rows_of_a_sequence_that_is_not_one_stay(dims):
    """Offsets that leave the batch: reported, and neither outputs nor gradients of those tokens are written."""
    lengths, total = [100, 50, 700], 850
    x, _, dout, dS = inputs(lengths, *dims, seed=5)
    full = (3, total, *dims, torch.bfloat16)
    bad = torch.tensor([0, 100, 850 + 9, 850], dtype=torch.int32, device="cuda")      # the second ends behind the batch, the third before its start
    d, ws, rec = outputs(x), gdnspec.empty_linear_seq_workspace(*full).fill_(0x3f), gdnspec.empty_linear_seq_record(*full).fill_(0x3f)
    both(x, bad, dout, dS, d, ws, rec)
    torch.cuda.synchronize()
    assert gdnspec.gdn_last_error() == gdnspec.ERR_INDEX
    assert gdnspec.gdn_last_error() == gdnspec.OK
    first = {m: (y[:1] if m == "S0" else y[:100]) for m, y in x.items()}
    want = plain(first, [100], dout[:100], dS[:1])
    for m in want:
        one = m in ("S_T", "dS0")
        held(d[m][:1] if one else d[m][:100], want[m], m)
        assert torch.isnan(d[m][1:] if one else d[m][100:]).all(), m
