"""Decay-gated linear attention over sequences and rotary positions on the GPU: places, decays and positions at the edges of what is allowed."""
import numpy as np
import pytest
import torch

from speculative_decoding_linear_gb300 import gdnspec
from test_gpu_linear_seq_forms import NAMES, both, held, inputs, outputs, plain

pytestmark = pytest.mark.gpu


def behind(n, at):
    """n bytes that start `at` bytes behind a 32-byte boundary."""
    store = torch.full((n + 32,), 0xff, dtype=torch.uint8, device="cuda")
    y = store[at:at + n]
    assert y.data_ptr() % 32 == at
    return y


@pytest.mark.parametrize("lengths,dims", [([700, 3, 130], (4, 2, 64, 64)), ([513, 0, 90], (8, 2, 128, 128)), ([300, 77], (2, 1, 256, 64)),
                                          ([200, 65], (2, 2, 96, 80))])
@pytest.mark.parametrize("ws_at,rec_at", [(16, 0), (0, 16), (16, 16)])
def test_workspace_and_record_on_16_bytes(lengths, dims, ws_at, rec_at):
    """Shared heads' sums pass through the workspace: equal bits wherever it and the record start."""
    x, off, dout, dS = inputs(lengths, *dims, seed=21)
    full = (len(lengths), sum(lengths), *dims, torch.bfloat16)
    want, got = outputs(x), outputs(x)
    both(x, off, dout, dS, want, gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full))
    ws = behind(gdnspec.gdn_linear_seq_workspace_bytes(*full), ws_at)
    rec = behind(gdnspec.gdn_linear_seq_record_bytes(*full), rec_at)
    both(x, off, dout, dS, got, ws, rec)
    assert gdnspec.gdn_last_error() == gdnspec.OK
    for m in want:
        assert torch.equal(got[m], want[m]), m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths", [[512], [300, 64, 130, 3]])
@pytest.mark.parametrize("end", [True, False])
def test_gradient_of_fast_decays_element_by_element(dtype, lengths, end):
    """dlog_alpha where nothing but the decays' gradient from one end is left: each element is far smaller than its neighbour.

    end: dO = 0, so dlog_alpha_u = sum_{s < u} beta_s v_s.(e^{G - g_s} dS k_s) + e^G <dS, S0>; the last token's own term is none
    of its element's.  Else v = 0 and dS = 0: sum_{t >= u} q_t.(e^{g_t} S0^T dO_t).  All inputs are positive, so sums keep
    their relative accuracy: of two products over 64 and of a segment's tokens, (64 + 64 + 512) 2^-24 = 3.8e-5, and a
    decay e^x of |x| up to 16 x 7 is off by 2 |x| 2^-24 = 1.4e-5 of itself: 1e-4 of each element.  Held are elements above
    1e-30: their factors are below 10^4, so the decays of what they are made of are above 1e-34, ten thousand times
    the least normal number (2^-126 = 1.2e-38, below which fp32 has fewer bits and exponentials may be zero).
    """
    dims = (2, 1, 64, 64)
    x, off, dout, dS = inputs(lengths, *dims, seed=31)
    x = {m: y.abs().to(dtype if m in "qkv" else torch.float32) for m, y in x.items()}
    x["log_alpha"].fill_(-7.0 if end else -5.0)
    dout, dS = dout.abs().to(dtype), dS.abs()
    (dout if end else dS).zero_()
    if not end:
        x["v"].zero_()
    full = (len(lengths), sum(lengths), *dims, dtype)
    d = outputs(x)
    both(x, off, dout, dS, d, gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full))
    assert gdnspec.gdn_last_error() == gdnspec.OK
    b = 0
    for i, n in enumerate(lengths):
        # by the formula (differentiation by a running sum takes its end away again, 1e-16 of the largest element)
        q, k, v, do, la, beta = (y[b:b + n].double() for y in (x["q"], x["k"], x["v"], dout, x["log_alpha"], x["beta"]))
        g, S0, dS_T = la.cumsum(0), x["S0"][i].double(), dS[i].double()
        if end:
            each = beta * (g[-1] - g).exp() * torch.einsum("shv,hvk,sk->sh", v, dS_T, k[:, 0])
            start = g[-1].exp() * (dS_T * S0).sum((-1, -2))
            want = torch.cat([start[None], start + each.cumsum(0)[:-1]])
        else:
            each = g.exp() * torch.einsum("tk,hvk,thv->th", q[:, 0], S0, do)
            want = each.flip(0).cumsum(0).flip(0)
        rows = slice(max(0, n - 16), n) if end else slice(0, min(n, 16))
        got, want = d["dlog_alpha"][b:b + n][rows].double(), want[rows]
        got, want = got[want > 1e-30], want[want > 1e-30]
        assert len(want) >= min(n, 9) and ((got - want).abs() <= 1e-4 * want).all(), (n, ((got - want) / want).abs().max())
        b += n


@pytest.mark.parametrize("cut", [0, 1, 63, 64, 100, 127, 290])
def test_nothing_passes_a_decay_of_zero(cut):
    """fp32, log_alpha = -inf at a token: each term of its gradient has that decay as a factor, so the gradient is zero, not
    what differences of sums would leave."""
    lengths, dims = [300, 70], (2, 1, 64, 48)
    x, off, dout, dS = inputs(lengths, *dims, seed=41)
    x, dout = {m: y.float() for m, y in x.items()}, dout.float()
    x["log_alpha"][cut] = -float("inf")
    full = (2, 370, *dims, torch.float32)
    d = outputs(x)
    both(x, off, dout, dS, d, gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full))
    assert gdnspec.gdn_last_error() == gdnspec.OK
    assert (d["dlog_alpha"][cut] == 0).all()
    assert torch.isfinite(d["dlog_alpha"]).all() and (d["dlog_alpha"][:cut] != 0).all() and (d["dlog_alpha"][cut + 1:] != 0).all()


U = 2.0 ** -24


@pytest.mark.parametrize("dtype,n", [(torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 512)])
def test_long_decays_keep_their_bits(dtype, n):
    """No writes (beta = 0): S_T = e^G S0 and, without dO, dS0 = e^G dS_T, with G about -80.

    An exponential is off by 2 ulp (4 x 2^-24) at most, the low part's and the state's products by 2^-24 each: 6 x 2^-24 of
    each element.  An exponent rounded to a float alone would be off by 80 x 2^-24.  Below 2^-126 (e^-87.3) a float's step is
    2^-149 whatever its size: 2 steps of the exponential and half a one of the low part's product, times the state, and
    half a one of the result.
    """
    dims = (2, 1, 16, 16)
    x, off, dout, dS = inputs([n], *dims, seed=51)
    x = {m: y.to(dtype) if m in "qkv" else y for m, y in x.items()}
    x["beta"].zero_()
    x["log_alpha"] = -(torch.rand(n, 2, generator=torch.Generator().manual_seed(1)) * 160 / n).cuda()
    dout = torch.zeros_like(x["v"])
    full = (1, n, *dims, dtype)
    d = outputs(x)
    both(x, off, dout, dS, d, gdnspec.empty_linear_seq_workspace(*full), gdnspec.empty_linear_seq_record(*full))
    assert gdnspec.gdn_last_error() == gdnspec.OK
    decay = x["log_alpha"].double().sum(0).exp()[None, :, None, None]
    for got, before in ((d["S_T"], x["S0"]), (d["dS0"], dS)):
        want = decay * before.double()
        tol = 6 * U * want.abs() + 2.0 ** -149 * (2.5 * before.double().abs() + 0.5)
        assert ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() / tol).max()


def test_far_tokens_keep_their_bits():
    """fp32, one write: o_t = e^{g_t - g_0} beta_0 v_0 (k_0.q_t), all positive, with decays down to e^-75.

    A dot over 16 (16 x 2^-24), an exponential (4), its low part, beta, the decay's and v's products (4): 24 x 2^-24 of each.
    """
    n, dims = 64, (2, 1, 16, 16)
    x, off, _, _ = inputs([n], *dims, seed=52)
    x = {m: y.abs().float() for m, y in x.items()}
    x["S0"].zero_()
    x["beta"][1:] = 0.0
    x["log_alpha"] = -(1.0 + 0.4 * torch.rand(n, 2, generator=torch.Generator().manual_seed(2))).cuda()
    out = torch.empty_like(x["v"])
    ws = gdnspec.empty_linear_seq_workspace(1, n, *dims, torch.float32, backward=False)
    gdnspec.gdn_linear_seq_forward(*(x[m] for m in NAMES), out, None, ws, offsets=off)
    y = {m: z.double() for m, z in x.items()}
    g = y["log_alpha"].cumsum(0)
    want = (g - g[0]).exp()[..., None] * (y["beta"][0][:, None] * y["v"][0])[None] * (y["q"][:, 0] @ y["k"][0, 0])[:, None, None]
    assert ((out.double() - want).abs() <= 24 * U * want).all(), ((out.double() - want) / want).abs().max() / U


def turns_of(positions, freqs):
    """position x frequency in turns, modulo one, in whole numbers: 1 / 2 pi to 300 bits (pi by Machin's formula)."""
    bits = 320

    def arctan_of_one_over(n):
        term = total = (1 << bits) // n
        k = 1
        while term:
            term //= n * n
            total += (-term if k % 2 else term) // (2 * k + 1)
            k += 1
        return total

    inv = (1 << 2 * bits) // (2 * 4 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239)))      # 2^bits / 2 pi
    whole = 1 << (bits + 149)
    steps = [int(f * 2.0 ** 75) << 74 if abs(f) >= 2.0 ** -50 else int(f * 2.0 ** 149) for f in freqs]      # exact multiples of 2^-149
    # the nearest multiple of a turn taken off
    return np.array([[((p * m * inv + whole // 2) % whole - whole // 2) / whole for m in steps] for p in positions])


def test_angles_of_any_position_and_frequency():
    """(1, 0) turned: cosine and sine themselves, for all int32 positions and frequencies up to 2^26.

    The angle is off by 5e-9 turns.  Near an axis (one of the two below 0.1) a rounding of both by 2 x 2^-24 of themselves
    turns the vector by 4 x 0.1 x 2^-24 / 2 pi = 4e-9 turns at most.  And everywhere each is off by 2 x 2^-24 of itself and the
    angle's 3.2e-8 rad.
    """
    g = torch.Generator().manual_seed(61)
    freqs = [1.0, 0.7, -0.37, 2.0 ** -20, 1e-4, 1e-30, 7.3, 99.9, 3000.7, -40000.1, 123456.7, 2.0 ** 20 * 1.1, -2.0 ** 23 * 1.7, 2.0 ** 25 * 1.37, 2.0 ** 26 * (1 - U), 0.0]
    f = torch.tensor(freqs, dtype=torch.float32)
    pos = torch.randint(-2 ** 31, 2 ** 31, (3000,), generator=g)
    pos[:8] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, -2 ** 31 + 1, 0, 1, -1, 1 << 30])
    pos[1500:] %= 1 << 20
    t = turns_of(pos.tolist(), f.tolist())
    x = torch.zeros(len(pos), 1, 32)
    x[..., :16] = 1.0
    for inverse in (False, True):
        out = torch.empty(len(pos), 1, 32, device="cuda")
        gdnspec.gdn_rotary(x.cuda(), None, pos.int().cuda(), f.cuda(), out, None, inverse=inverse)
        assert gdnspec.gdn_last_error() == gdnspec.OK
        y = out.double().cpu().numpy()[:, 0]
        c, s = y[:, :16], y[:, 16:] * (-1 if inverse else 1)
        d = np.arctan2(s, c) / (2 * np.pi) - t
        d -= np.round(d)
        near = np.minimum(np.abs(c), np.abs(s)) < 0.1
        assert np.abs(d[near]).max() <= 9e-9, np.abs(d[near]).max()
        for got, want in ((c, np.cos(2 * np.pi * t)), (s, np.sin(2 * np.pi * t))):
            assert (np.abs(got - want) <= 2 * U * np.abs(want) + 3.2e-8).all(), np.abs(got - want).max() / U


def test_hundreds_of_thousands_of_sequences():
    """What one warp does for all sequences keeps no other waiting: with a limit of 5 ms no wait of the call runs out."""
    n, dims = 300_000, (1, 1, 16, 16)
    g = torch.Generator(device="cuda").manual_seed(71)
    lengths = torch.randint(1, 4, (n,), generator=g, device="cuda")
    lengths[::1000] = torch.randint(1, 600, (n // 1000,), generator=g, device="cuda")
    off = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)]).int()
    total = int(off[-1])
    x = {m: torch.randn(total, 1, 16, generator=g, device="cuda").bfloat16() for m in "qkv"}
    x["log_alpha"], x["beta"] = -torch.rand(total, 1, generator=g, device="cuda"), torch.rand(total, 1, generator=g, device="cuda")
    x["S0"] = torch.randn(n, 1, 16, 16, generator=g, device="cuda")
    out, S_T = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    ws = gdnspec.empty_linear_seq_workspace(n, total, *dims, torch.bfloat16, backward=False)
    gdnspec.gdn_set_wait_limit_ns(5_000_000)
    try:
        gdnspec.gdn_linear_seq_forward(*(x[m] for m in NAMES), out, S_T, ws, offsets=off)
        assert gdnspec.gdn_last_error() == gdnspec.OK
    finally:
        gdnspec.gdn_set_wait_limit_ns(1_000_000_000)
    # a token at a time, each from the state before it
    S, want = x["S0"].double(), torch.empty_like(out, dtype=torch.double)
    for t in range(int(lengths.max())):
        live = (lengths > t).nonzero()[:, 0]
        at = off[live].long() + t
        q, k, v, la, beta = (x[m][at].double() for m in ("q", "k", "v", "log_alpha", "beta"))
        S[live] = la.exp()[..., None, None] * S[live] + (beta[..., None] * v)[..., None] * k[:, :, None, :]
        want[at] = (S[live] @ q[..., None])[..., 0]
    held(out, want, "out")
    held(S_T, S, "S_T")


@pytest.mark.parametrize("dims", [(4, 1, 16, 48), (2, 2, 96, 96), (1, 1, 192, 80), (2, 1, 48, 208), (4, 2, 240, 16)])
@pytest.mark.parametrize("slow", [False, True])
def test_narrow_and_odd_heads_in_their_own_rounding(dims, slow):
    """Sizes that are no whole boxes of 64 columns, and lengths that end inside a block, a piece of 16 and a segment."""
    lengths = [129, 300, 17, 515, 1, 0, 1100]
    x, off, dout, dS = inputs(lengths, *dims, seed=81, slow=slow)
    full = (len(lengths), sum(lengths), *dims, torch.bfloat16)
    d = outputs(x)
    both(x, off, dout, dS, d, gdnspec.empty_linear_seq_workspace(*full).fill_(0xff), gdnspec.empty_linear_seq_record(*full).fill_(0xff))
    assert gdnspec.gdn_last_error() == gdnspec.OK
    want = plain(x, lengths, dout, dS)
    for m in want:
        held(d[m], want[m], m)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offsets", [[0, 0, 0], [700, 700, 700], [350, 350, 350]])
def test_tokens_of_no_sequence(dtype, offsets):
    """A batch that is all padding: states and their gradients pass through, rows are zero, whatever the tokens hold."""
    dims = (4, 2, 64, 64)
    x, _, dout, dS = inputs([700, 0], *dims, seed=91)
    x = {m: torch.full_like(y, float("nan"), dtype=dtype if m in "qkv" else None) if m != "S0" else y for m, y in x.items()}
    full = (2, 700, *dims, dtype)
    d = outputs(x)
    both(x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), torch.full_like(x["v"], float("nan")), dS, d,
         gdnspec.empty_linear_seq_workspace(*full).fill_(0xff), gdnspec.empty_linear_seq_record(*full).fill_(0xff))
    assert gdnspec.gdn_last_error() == gdnspec.OK
    for m, y in d.items():
        assert torch.equal(y, x["S0"] if m == "S_T" else dS if m == "dS0" else torch.zeros_like(y)), m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,H,Hk", [(16, 16, 1, 0), (16, 2, 1, 1), (16, 8, 3, 2), (48, 6, 2, 1), (64, 64, 1, 1), (128, 64, 8, 2), (256, 256, 1, 2)])
def test_rotary_by_several_tokens_a_block(dtype, interleaved, d, rot, H, Hk):
    """Where there are many tokens a block takes up to sixteen: the same bits as a call of few, whose blocks take one."""
    total = 9973
    g = torch.Generator(device="cuda").manual_seed(d + rot)
    q = torch.randn(total, H, d, generator=g, device="cuda").to(dtype)
    k = torch.randn(total, Hk, d, generator=g, device="cuda").to(dtype) if Hk else None
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (total,), generator=g, device="cuda").int()
    f = gdnspec.gdn_rotary_frequencies(rot)
    whole, parts = [[torch.full_like(y, float("nan")) if y is not None else None for y in (q, k)] for _ in range(2)]
    at = lambda y, b: None if y is None else y[b:b + 499]  # noqa: E731
    gdnspec.gdn_rotary(q, k, pos, f, *whole, scale=1.5, interleaved=interleaved)
    for b in range(0, total, 499):
        gdnspec.gdn_rotary(at(q, b), at(k, b), pos[b:b + 499], f, at(parts[0], b), at(parts[1], b), scale=1.5, interleaved=interleaved)
    assert gdnspec.gdn_last_error() == gdnspec.OK
    for y, z, x in zip(whole, parts, (q, k)):
        assert y is None or (torch.equal(y, z) and torch.isfinite(y).all() and torch.equal(y[..., rot:], x[..., rot:]))
