"""Decay-gated linear attention over sequences and in decode on the GPU against the fp64 oracle.

Tolerances, before any run.

fp32 outputs: a sum of n terms rounded to 24 bits at each step is off by about sqrt(n) 2^-24 of the sum of its terms'
squares' root, and by n 2^-24 of the sum of their sizes at most; a value here is a sum over d_k or d_v and over the
tokens of a segment, and what the segments before it left passes through a decay that does not grow it.  So the
elements are held to 8 n 2^-24 of the root mean square (n = d_k + d_v + 64: the largest element against the root mean
square, and the sum over segments, are in the 8), and the whole array to 4e-6 = 64 x 2^-24 of its norm, the square root
of n = 4096 terms.

bf16 outputs: the scores and the states may be rounded to bf16 once before their products, each term by at most 2^-8 of
itself, and so by 2^-8 / sqrt(3) in the root mean square at most; the output is rounded once.  Independent of one
another the two give sqrt(2 / 3) 2^-8 of the norm: the whole array is held to 2^-8.  An element is off by 2^-8 of
itself and by the sum of its terms' roundings, which have the size of the row's values and a sign each: six times
2^-8 / sqrt(3) of the larger of the row's and the array's root mean square.
"""
import numpy as np
import pytest
import torch

from oracle import linear_seq as ref
from speculative_decoding_linear_gb300 import gdnspec

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("q", "k", "v", "log_alpha", "beta", "S0")


def check(got, want, what, n):
    g = got.double().cpu().numpy()
    assert g.shape == want.shape, what
    assert np.isfinite(g).all(), what
    if want.size == 0:
        return
    d, rms = np.abs(g - want), max(np.sqrt(np.mean(want ** 2)), 1e-30)
    if got.dtype == torch.bfloat16:
        row = np.maximum(np.sqrt(np.mean(want ** 2, -1, keepdims=True)), rms)
        tol, norm = 2.0 ** -8 * (np.abs(want) + 6 / np.sqrt(3) * row), 2.0 ** -8
    else:
        tol, norm = 8 * n * 2.0 ** -24 * rms, 4e-6
    assert not (d > tol).any(), "%s: worst %.3g of rms" % (what, d.max() / rms)
    rel = np.sqrt(np.mean(d ** 2)) / rms
    assert rel <= norm, "%s: %.3g of the norm" % (what, rel)


def make(lengths, H, Hk, dk, dv, dtype, seed=0, gates="mixed", wide=False):
    rng = np.random.default_rng(seed)
    total, n, t = sum(lengths), len(lengths), TYPES[dtype]
    c = lambda x, d=torch.float32: torch.from_numpy(np.ascontiguousarray(x)).to(d).cuda()  # noqa: E731
    unit = lambda *s: (lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True))(rng.standard_normal(s))  # noqa: E731
    la = {"mixed": lambda: -np.logaddexp(0, rng.uniform(-6, 1, (total, H))), "slow": lambda: -rng.uniform(1e-5, 2e-3, (total, H)),
          "none": lambda: np.zeros((total, H)), "fast": lambda: -rng.uniform(2, 30, (total, H))}[gates]()
    x = dict(q=c(unit(total, Hk, dk), t), k=c(unit(total, Hk, dk), t), v=c(rng.standard_normal((total, H, dv)), t),
             log_alpha=c(la), beta=c(rng.uniform(0.05, 1.0, (total, H))), S0=c(0.1 * rng.standard_normal((n, H, dv, dk))))
    if wide:      # q, k, v as columns of one projection
        both = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1)], 1)
        a, b = Hk * dk, 2 * Hk * dk
        x["q"], x["k"], x["v"] = both[:, :a].view(total, Hk, dk), both[:, a:b].view(total, Hk, dk), both[:, b:].view(total, H, dv)
    return x, torch.tensor(np.cumsum([0] + list(lengths)), dtype=torch.int32).cuda()


def wide64(x):
    return {m: y.double().cpu().numpy() for m, y in x.items()}


def poisoned(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def run(x, off, lengths, dims, dtype, back=True, dout=None, dS=None, S0=True, ws=None):
    """Outputs and gradients; every buffer that the calls write starts as NaN."""
    n, total = len(lengths), x["q"].shape[0]
    H, Hk, dk, dv = dims
    t = TYPES[dtype]
    full = (n, total, H, Hk, dk, dv, t)
    if ws is None:
        ws = gdnspec.empty_linear_seq_workspace(*full, backward=back)
    ws.fill_(0xff)
    rec = gdnspec.empty_linear_seq_record(*full).fill_(0xff) if back else None
    got = {"out": poisoned(total, H, dv, dtype=t), "S_T": poisoned(n, H, dv, dk)}
    gdnspec.gdn_linear_seq_forward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["S0"] if S0 else None, got["out"], got["S_T"], ws,
                                   offsets=off, record=rec)
    if back:
        d = {m: poisoned(*x[m].shape, dtype=x[m].dtype) for m in NAMES}
        gdnspec.gdn_linear_seq_backward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], dout, dS, rec, d["q"], d["k"], d["v"],
                                        d["log_alpha"], d["beta"], d["S0"], ws, offsets=off)
        got.update({"d" + m: d[m] for m in NAMES})
    assert gdnspec.gdn_last_error() == gdnspec.OK
    return got


LENGTHS = [[1], [5], [64], [65, 1, 0, 127], [0, 128, 129, 63], [511, 0, 513], [512, 512], [1500]]
DIMS = [(4, 2, 64, 64), (2, 2, 128, 128), (4, 1, 16, 48), (2, 1, 256, 256), (2, 2, 96, 96), (1, 1, 192, 80), (2, 1, 128, 256), (2, 2, 256, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(LENGTHS)))
@pytest.mark.parametrize("gates", ["mixed", "slow"])
def test_forward_and_gradients(dtype, i, gates):
    for j, dims in enumerate((DIMS[i], DIMS[(i + 3) % len(DIMS)])):
        H, Hk, dk, dv = dims
        lengths = LENGTHS[i]
        x, off = make(lengths, *dims, dtype, seed=10 * i + j, gates=gates, wide=j == 1)
        rng = np.random.default_rng(77 + i)
        dout = torch.from_numpy(rng.standard_normal((sum(lengths), H, dv))).to(TYPES[dtype]).cuda()
        dS = torch.from_numpy(0.1 * rng.standard_normal((len(lengths), H, dv, dk))).float().cuda()
        got = run(x, off, lengths, dims, dtype, dout=dout, dS=dS)
        x64 = wide64(x)
        o, S = ref.forward(**x64, lengths=lengths)
        grads = ref.backward(**x64, lengths=lengths, dout=dout.double().cpu().numpy(), dS_T=dS.double().cpu().numpy())
        for name, want in [("out", o), ("S_T", S)] + [("d" + m, grads[m]) for m in NAMES]:
            check(got[name], want, "%s of %s %s" % (name, lengths, dims), dk + dv + 64)
        # without a record: the same, and a smaller workspace
        bare = run(x, off, lengths, dims, dtype, back=False)
        check(bare["out"], o, "out without a record", dk + dv + 64)
        check(bare["S_T"], S, "S_T without a record", dk + dv + 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gates", ["none", "fast"])
def test_decays_of_one_and_close_to_zero(dtype, gates):
    dims, lengths = (2, 2, 64, 64), [700, 90]
    x, off = make(lengths, *dims, dtype, gates=gates)
    if gates == "fast":
        x["log_alpha"][50:60] = -float("inf")        # forgets the state
        x["log_alpha"][600] = -1000.0
    x["beta"][100:140] = 0.0
    rng = np.random.default_rng(5)
    dout = torch.from_numpy(rng.standard_normal((790, 2, 64))).to(TYPES[dtype]).cuda()
    dS = torch.from_numpy(rng.standard_normal((2, 2, 64, 64))).float().cuda()
    got = run(x, off, lengths, dims, dtype, dout=dout, dS=dS)
    x64 = wide64(x)
    o, S = ref.forward(**x64, lengths=lengths)
    grads = ref.backward(**x64, lengths=lengths, dout=dout.double().cpu().numpy(), dS_T=dS.double().cpu().numpy())
    for name, want in [("out", o), ("S_T", S)] + [("d" + m, grads[m]) for m in NAMES]:
        check(got[name], want, name, 192)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_lengths_no_states_and_in_place(dtype):
    H, Hk, dk, dv = dims = (4, 2, 64, 128)
    lengths = [130] * 3
    x, _ = make(lengths, *dims, dtype)
    n = dk + dv + 64
    x64 = wide64(x)
    zero = dict(x64, S0=np.zeros_like(x64["S0"]))
    four = {m: y.view(3, 130, *y.shape[1:]) if m != "S0" else y for m, y in x.items()}
    full = (3, 390, H, Hk, dk, dv, TYPES[dtype])
    ws, rec = gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full)
    out = torch.empty_like(four["v"])
    args = [four[m] for m in ("q", "k", "v", "log_alpha", "beta")]
    gdnspec.gdn_linear_seq_forward(*args, None, out, None, ws, record=rec)                 # no first state, no last one wanted
    check(out.flatten(0, 1), ref.forward(**zero, lengths=lengths)[0], "out", n)
    dout = torch.randn_like(out)
    d = [torch.empty_like(y) for y in args]
    gdnspec.gdn_linear_seq_backward(*args, dout, None, rec, *d, None, ws)
    g = ref.backward(**zero, lengths=lengths, dout=dout.flatten(0, 1).double().cpu().numpy(), dS_T=np.zeros_like(x64["S0"]))
    for m, y in zip(NAMES, d):
        check(y.flatten(0, 1), g[m], "d" + m, n)
    # the states in place
    S = x["S0"].clone()
    gdnspec.gdn_linear_seq_forward(*args, S, out, S, ws)
    o, S_T = ref.forward(**x64, lengths=lengths)
    check(out.flatten(0, 1), o, "out", n)
    check(S, S_T, "S_T in place", n)
    gdnspec.gdn_linear_seq_forward(*args, x["S0"], out, None, ws, record=rec)
    dS = torch.randn_like(S)
    g = ref.backward(**x64, lengths=lengths, dout=dout.flatten(0, 1).double().cpu().numpy(), dS_T=dS.double().cpu().numpy())
    gdnspec.gdn_linear_seq_backward(*args, dout, dS, rec, *d, dS, ws)
    check(dS, g["S0"], "dS0 in place", n)
    assert gdnspec.gdn_last_error() == gdnspec.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    H, Hk, dk, dv = 2, 1, 64, 32
    x, off = make([0, 0], H, Hk, dk, dv, dtype)
    full = (2, 0, H, Hk, dk, dv, TYPES[dtype])
    ws, rec = gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full)
    S_T, dS = torch.empty_like(x["S0"]), torch.randn_like(x["S0"])
    gdnspec.gdn_linear_seq_forward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["S0"], torch.empty_like(x["v"]), S_T, ws, offsets=off, record=rec)
    assert torch.equal(S_T, x["S0"])
    d = [torch.empty_like(x[m]) for m in NAMES]
    gdnspec.gdn_linear_seq_backward(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], torch.empty_like(x["v"]), dS, rec, *d, ws, offsets=off)
    assert torch.equal(d[-1], dS) and gdnspec.gdn_last_error() == gdnspec.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_is_zero_and_kept_out(dtype):
    """Tokens before the first offset and behind the last: NaN in the inputs, zeros in the outputs."""
    dims, lengths, lead, rest = (4, 2, 64, 64), [70, 0, 531], 3, 40
    H, Hk, dk, dv = dims
    x, off = make([lead] + lengths + [rest], *dims, dtype)
    x["S0"] = x["S0"][:3].contiguous()
    rng = np.random.default_rng(3)
    total = lead + sum(lengths) + rest
    dout = torch.from_numpy(rng.standard_normal((total, H, dv))).to(TYPES[dtype]).cuda()
    dS = torch.from_numpy(rng.standard_normal((3, H, dv, dk))).float().cuda()
    inner = slice(lead, total - rest)
    x64 = {m: (y[inner] if m != "S0" else y) for m, y in wide64(x).items()}
    for y in [x[m] for m in NAMES[:-1]] + [dout]:
        y[:lead] = float("nan")
        y[total - rest:] = float("nan")
    got = run(x, off[1:-1].contiguous(), lengths, dims, dtype, dout=dout, dS=dS)
    o, S = ref.forward(**x64, lengths=lengths)
    g = ref.backward(**x64, lengths=lengths, dout=dout[inner].double().cpu().numpy(), dS_T=dS.double().cpu().numpy())
    for name, want in [("out", o)] + [("d" + m, g[m]) for m in NAMES[:-1]]:
        check(got[name][inner], want, name, 192)
        assert (got[name][:lead] == 0).all() and (got[name][total - rest:] == 0).all(), name
    check(got["S_T"], S, "S_T", 192)
    check(got["dS0"], g["S0"], "dS0", 192)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_value_stays_in_its_sequence(dtype, value):
    dims, lengths = (2, 1, 64, 64), [100, 37, 600, 5]
    x, off = make(lengths, *dims, dtype)
    dout, dS = torch.randn(742, 2, 64, device="cuda").to(TYPES[dtype]), torch.randn(4, 2, 64, 64, device="cuda")
    want = run(x, off, lengths, dims, dtype, dout=dout, dS=dS)
    for m in ("q", "k", "v", "log_alpha", "beta"):
        y = {n: z.clone() for n, z in x.items()}
        y[m][110] = value if m != "log_alpha" else float("nan")
        got = dict()
        n, total = len(lengths), 742
        full = (n, total, *dims, TYPES[dtype])
        ws, rec = gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full)
        got = {"out": torch.empty_like(y["v"]), "S_T": torch.empty_like(y["S0"])}
        got.update({"d" + w: torch.empty_like(y[w]) for w in NAMES})
        gdnspec.gdn_linear_seq_forward(*(y[w] for w in NAMES), got["out"], got["S_T"], ws, offsets=off, record=rec)
        gdnspec.gdn_linear_seq_backward(*(y[w] for w in NAMES[:-1]), dout, dS, rec, *(got["d" + w] for w in NAMES), ws, offsets=off)
        for name in want:
            rows = [0, 2, 3] if name in ("S_T", "dS0") else [t for t in range(742) if not 100 <= t < 137]
            assert torch.equal(got[name][rows], want[name][rows]), (m, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_offsets_are_reported(dtype):
    dims, total = (2, 2, 64, 64), 300
    x, _ = make([total], *dims, dtype)
    x["S0"] = torch.randn(3, 2, 64, 64, device="cuda")
    full = (3, total, *dims, TYPES[dtype])
    ws = gdnspec.empty_linear_seq_workspace(*full, backward=False)
    want = run(x, torch.tensor([0, 100, 150, 300], dtype=torch.int32).cuda(), [100, 50, 150], dims, dtype, back=False)
    for bad, good in (([0, 100, 90, 300], 0), ([0, 100, 150, 301], 0), ([-1, 100, 150, 300], 1), ([0, 100, 2 ** 31 - 1, 300], 0)):
        out, S_T = torch.zeros_like(x["v"]), torch.zeros_like(x["S0"])
        gdnspec.gdn_linear_seq_forward(*(x[m] for m in NAMES), out, S_T, ws, offsets=torch.tensor(bad, dtype=torch.int32).cuda())
        assert gdnspec.gdn_last_error() == gdnspec.ERR_INDEX
        rows = slice(0, 90) if good == 0 else slice(100, 150)      # from 90 on, the first offsets name a row twice
        assert torch.equal(out[rows], want["out"][rows]) and torch.equal(S_T[good], want["S_T"][good]), bad
    assert gdnspec.gdn_last_error() == gdnspec.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_bits_captured_and_on_two_streams(dtype):
    dims, lengths = (4, 2, 128, 64), [333, 1, 700]
    x, off = make(lengths, *dims, dtype)
    dout, dS = torch.randn(1034, 4, 64, device="cuda").to(TYPES[dtype]), torch.randn(3, 4, 64, 128, device="cuda")
    want = run(x, off, lengths, dims, dtype, dout=dout, dS=dS)
    full = (3, 1034, *dims, TYPES[dtype])

    def buffers():
        d = {"out": torch.zeros_like(x["v"]), "S_T": torch.zeros_like(x["S0"])}
        d.update({"d" + m: torch.zeros_like(x[m]) for m in NAMES})
        return d, gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full)

    def both(d, ws, rec):
        gdnspec.gdn_linear_seq_forward(*(x[m] for m in NAMES), d["out"], d["S_T"], ws, offsets=off, record=rec)
        gdnspec.gdn_linear_seq_backward(*(x[m] for m in NAMES[:-1]), dout, dS, rec, *(d["d" + m] for m in NAMES), ws, offsets=off)

    runs = [buffers() for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, b in zip(streams, runs):
            with torch.cuda.stream(st):
                both(*b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(*runs[2])
    for y in runs[2][0].values():
        y.fill_(float("nan"))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for d, _, _ in runs:
        for m in want:
            assert torch.equal(d[m], want[m]), m


def test_gradient_against_differences():
    dims, lengths = (2, 1, 32, 48), [90, 20]
    x, off = make(lengths, *dims, "f32")
    dout, dS = torch.randn(110, 2, 48, device="cuda"), torch.randn(2, 2, 48, 32, device="cuda")
    got = run(x, off, lengths, dims, "f32", dout=dout, dS=dS)
    for m in NAMES:
        u = torch.randn_like(x[m])
        if m == "log_alpha":
            u = u * x[m].abs()
        e, loss = 1e-2, []
        for sign in (1, -1):
            y = run(dict(x, **{m: x[m] + sign * e * u}), off, lengths, dims, "f32", back=False)
            loss.append(((y["out"] * dout).double().sum() + (y["S_T"] * dS).double().sum()).item())
        want = (got["d" + m].double() * u).sum().item()
        # e^2 of a third derivative, and the values' rounding (10^4 of them, 1e-6 of their size) over 2 e
        assert abs((loss[0] - loss[1]) / (2 * e) - want) < 1e-3 * (abs(want) + (got["d" + m].double() * u).norm().item()), m


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 8, 8, 256, 256), (9, 4, 2, 128, 64), (5, 2, 1, 16, 48), (3, 2, 2, 192, 80)])
def test_step(dtype, B, H, Hk, dk, dv):
    x, _ = make([B], H, Hk, dk, dv, dtype)
    pool = torch.randn(B + 3, H, dv, dk, device="cuda")
    index = torch.randperm(B + 3)[:B].int()
    if B > 1:
        index[1] = -1
    before, out = pool.clone(), poisoned(B, H, dv, dtype=TYPES[dtype])
    gdnspec.gdn_linear_seq_step(*(x[m] for m in NAMES[:-1]), pool, out, state_index=index.cuda())
    assert gdnspec.gdn_last_error() == gdnspec.OK
    x64, want = wide64(x), before.double().cpu().numpy()
    for b, at in enumerate(index.tolist()):
        if at < 0:
            assert (out[b] == 0).all()
            continue
        one = {m: x64[m][b:b + 1] for m in NAMES[:-1]}
        o, S = ref.forward(**one, S0=want[at:at + 1], lengths=[1])
        want[at] = S[0]
        check(out[b:b + 1], o, "out", dk + dv + 64)
    check(pool, want, "S", dk + dv + 64)
    live = set(index.tolist())
    for at in range(B + 3):
        if at not in live:
            assert torch.equal(pool[at], before[at])


def test_step_reports_a_slot_out_of_range():
    x, _ = make([3], 2, 2, 32, 32, "bf16")
    pool, out = torch.randn(4, 2, 32, 32, device="cuda"), torch.empty(3, 2, 32, dtype=torch.bfloat16, device="cuda")
    before = pool.clone()
    gdnspec.gdn_linear_seq_step(*(x[m] for m in NAMES[:-1]), pool, out, state_index=torch.tensor([4, 1, -2], dtype=torch.int32).cuda())
    assert gdnspec.gdn_last_error() == gdnspec.ERR_INDEX
    assert (out[0] == 0).all() and (out[2] == 0).all() and torch.equal(pool[[0, 2, 3]], before[[0, 2, 3]])


def test_prompt_rotary_steps_and_a_verified_draft():
    """One layer as a decoder uses it: prompts rotated and read, tokens one by one, a draft tree from the state, its path accepted."""
    H, Hk, dk, dv, lengths, steps = 2, 2, 64, 64, [130, 45], 3
    x, _ = make([n + steps for n in lengths], H, Hk, dk, dv, "bf16")
    freq = gdnspec.gdn_rotary_frequencies(32, 10000.0, 4.0, 64.0)
    pos = torch.cat([torch.arange(n + steps) for n in lengths]).int().cuda()
    gdnspec.gdn_rotary(x["q"], x["k"], pos, freq, x["q"], x["k"])
    x64 = wide64(x)
    ends = np.cumsum([n + steps for n in lengths])
    whole, states = ref.forward(**x64, lengths=[n + steps for n in lengths])
    keep = torch.cat([torch.arange(e - n - steps, e - steps) for e, n in zip(ends, lengths)]).cuda()
    p = {m: x[m][keep].contiguous() for m in NAMES[:-1]}
    pool, out = torch.empty_like(x["S0"]), torch.empty_like(p["v"])
    off = torch.tensor([0, lengths[0], sum(lengths)], dtype=torch.int32).cuda()
    ws = gdnspec.empty_linear_seq_workspace(2, sum(lengths), H, Hk, dk, dv, "bf16", backward=False)
    gdnspec.gdn_linear_seq_forward(*p.values(), x["S0"], out, pool, ws, offsets=off)
    for t in range(steps, 0, -1):
        rows = torch.tensor([e - t for e in ends]).cuda()
        one = [x[m][rows].contiguous() for m in NAMES[:-1]]
        o = torch.empty_like(one[2])
        gdnspec.gdn_linear_seq_step(*one, pool, o)
        check(o, whole[rows.cpu().numpy()], "step", 192)
    check(pool, states, "states", 192)
    # a tree of five drafts a sequence: rotated at the state's position plus the depth, verified, a path committed
    N = 5
    d, _ = make([2 * N], H, Hk, dk, dv, "bf16", seed=9)
    d = {m: d[m].view(2, N, *d[m].shape[1:]) for m in NAMES[:-1]}
    parent = torch.tensor([[-1, 0, 1, 1, 0]] * 2, dtype=torch.int32).cuda()
    mask, depth = torch.empty(2, N, dtype=torch.int64, device="cuda"), torch.empty(2, N, dtype=torch.int32, device="cuda")
    gdnspec.gdn_tree_mask(parent, mask, depth)
    dpos = (depth + torch.tensor([[n + steps] for n in lengths], device="cuda")).int()
    gdnspec.gdn_rotary(d["q"], d["k"], dpos, freq, d["q"], d["k"])
    alpha = d["log_alpha"].exp()
    fac, o = gdnspec.empty_factors(2, N, H, dk, dv, torch.bfloat16), torch.empty(2, N, H, dv, device="cuda")
    gdnspec.gdn_linear_tree_verify(d["q"], d["k"], d["v"], alpha, d["beta"], parent, pool, o, fac, gdnspec.empty_workspace(2, N, H, dk, dv))
    path = torch.tensor([[0, 1, 3, -1]] * 2, dtype=torch.int32).cuda()
    S_new = torch.empty_like(pool)
    gdnspec.gdn_commit(pool, fac, path, S_new, N, torch.bfloat16)
    # the same path as a prompt from the same state
    chain = {m: d[m][:, [0, 1, 3]].contiguous() for m in NAMES[:-1]}
    o2, S2 = torch.empty_like(chain["v"]), torch.empty_like(pool)
    ws = gdnspec.empty_linear_seq_workspace(2, 6, H, Hk, dk, dv, "bf16", backward=False)
    gdnspec.gdn_linear_seq_forward(*chain.values(), pool, o2, S2, ws)
    check(o2.flatten(0, 1), o[:, [0, 1, 3]].flatten(0, 1).double().cpu().numpy(), "verified path", 192)
    check(S2, S_new.double().cpu().numpy(), "committed state", 192)
    assert gdnspec.gdn_last_error() == gdnspec.OK
