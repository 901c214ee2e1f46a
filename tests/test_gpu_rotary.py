"""Rotary positions on the GPU against the fp64 oracle.

Tolerances, before any run: the angle is a multiple of 2^-32 turns (off by 1.5e-9 rad) and as half turns in fp32 off by
2^-25 of at most one half turn, 9.4e-8 rad = 1.6 x 2^-24; sine and cosine are rounded (2 ulp at most, 2^-22), times the
scale 2^-24, and two products and a sum round by 2^-24 each: below 10 x 2^-24 of the pair's size.  The output adds its
own rounding, 2^-8 of itself in bf16 and 2^-24 in fp32.
"""
import numpy as np
import pytest
import torch

from oracle import linear_seq as ref
from speculative_decoding_linear_gb300 import gdnspec

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def pair_size(x, rot, interleaved, scale):
    y = np.abs(x.copy())
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    size = scale * np.hypot(y[..., a], y[..., b])
    y[...] = 0.0
    y[..., a], y[..., b] = size, size
    return y


def check(got, x, positions, freq, scale, interleaved, inverse):
    x64, f64, rot = x.double().cpu().numpy(), freq.double().cpu().numpy(), 2 * freq.numel()
    want = ref.rotary(x64, positions.cpu().numpy(), f64, scale, interleaved, inverse)
    half = 2.0 ** -8 if x.dtype is torch.bfloat16 else 2.0 ** -24
    tol = 10 * 2.0 ** -24 * pair_size(x64, rot, interleaved, abs(scale)) + half * np.abs(want)
    d = np.abs(got.double().cpu().numpy() - want)
    assert (d <= tol).all(), (d - tol).max()
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,H,Hk", [(16, 16, 1, 1), (16, 2, 3, 1), (64, 64, 8, 2), (64, 24, 2, 2), (128, 96, 4, 1), (128, 6, 8, 8), (192, 100, 5, 1),
                                        (256, 256, 8, 8), (48, 4, 40, 3)])
def test_rotary(dtype, interleaved, d, rot, H, Hk):
    g = torch.Generator(device="cuda").manual_seed(d + rot)
    for total, inverse, scale in ((1, False, 1.0), (37, True, 1.25), (515, False, -0.5)):
        q = torch.randn(total, H, d, generator=g, device="cuda").to(TYPES[dtype])
        k = torch.randn(total, Hk, d, generator=g, device="cuda").to(TYPES[dtype])
        pos = torch.randint(-1000, 2 ** 20, (total,), generator=g, device="cuda", dtype=torch.int32)
        pos[0] = 2 ** 31 - 1 if total > 1 else 0
        pos[-1] = -2 ** 31 if total > 1 else 5
        freq = gdnspec.gdn_rotary_frequencies(rot, 10000.0, 1.0 if inverse else 4.0, 4096.0)
        qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
        gdnspec.gdn_rotary(q, k, pos, freq, qo, ko, scale=scale, interleaved=interleaved, inverse=inverse)
        check(qo, q, pos, freq, scale, interleaved, inverse)
        check(ko, k, pos, freq, scale, interleaved, inverse)
        only = torch.full_like(q, float("nan"))
        gdnspec.gdn_rotary(q, None, pos, freq, only, None, scale=scale, interleaved=interleaved, inverse=inverse)
        assert torch.equal(only, qo)
        gdnspec.gdn_rotary(q, k, pos, freq, q, k, scale=scale, interleaved=interleaved, inverse=inverse)      # in place
        assert torch.equal(q, qo) and torch.equal(k, ko)
    assert gdnspec.gdn_last_error() == gdnspec.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_columns_of_a_projection(dtype):
    total, H, Hk, d = 130, 4, 2, 64
    wide = torch.randn(total, (H + 2 * Hk) * d, device="cuda").to(TYPES[dtype])
    view = lambda w: (w[:, : H * d].view(total, H, d), w[:, H * d:(H + Hk) * d].view(total, Hk, d))  # noqa: E731
    q, k = view(wide)
    pos, freq = torch.arange(total, dtype=torch.int32).cuda(), gdnspec.gdn_rotary_frequencies(d)
    q0, k0, rest = q.clone(), k.clone(), wide[:, (H + Hk) * d:].clone()
    gdnspec.gdn_rotary(q, k, pos, freq, q, k)
    check(q.contiguous(), q0, pos, freq, 1.0, False, False)
    check(k.contiguous(), k0, pos, freq, 1.0, False, False)
    assert torch.equal(wide[:, (H + Hk) * d:], rest)
    other = torch.zeros_like(wide)
    gdnspec.gdn_rotary(q0, k0, pos, freq, *view(other))
    assert torch.equal(other[:, : (H + Hk) * d], wide[:, : (H + Hk) * d]) and (other[:, (H + Hk) * d:] == 0).all()
    batch = q0.view(2, 65, H, d), k0.view(2, 65, Hk, d)
    out = torch.empty_like(batch[0]), torch.empty_like(batch[1])
    gdnspec.gdn_rotary(*batch, pos.view(2, 65), freq, *out)
    assert torch.equal(out[0].flatten(0, 1), q.contiguous())


def test_frequencies_of_any_size():
    """Above one turn a token, tiny, subnormal, negative; NaN and what is too large give NaN."""
    f = torch.tensor([1.0, 7.3, 1e-30, 1e-40, -0.37, 123456.7, float("nan"), 1e9], device="cuda")
    q = torch.randn(9, 1, 16, device="cuda")
    pos = torch.tensor([0, 1, 2, 100, -5, 4095, 65536, 99999, 10 ** 6], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    gdnspec.gdn_rotary(q, None, pos, f, out, None)
    assert torch.isnan(out[..., [6, 7, 14, 15]]).all()
    fine = [0, 1, 2, 3, 4, 5, 8, 9, 10, 11, 12, 13]
    check(out[..., fine].contiguous(), q[..., fine].contiguous(), pos, f[:6], 1.0, False, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_is_the_inverse_turn(interleaved):
    """<y, R x> = <R^T y, x>, and against differences: the turn is linear, so a difference is exact but for rounding."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y, u = (torch.randn(50, 2, 64, generator=g, device="cuda") for _ in range(3))
    pos, freq = torch.arange(3, 53, dtype=torch.int32).cuda(), gdnspec.gdn_rotary_frequencies(48)
    turned = lambda t, inv=False: (lambda o: (gdnspec.gdn_rotary(t, None, pos, freq, o, None, scale=1.3, interleaved=interleaved, inverse=inv), o)[1])(  # noqa: E731
        torch.empty_like(t))
    grad = turned(y, True)
    e = 0.5
    diff = ((turned(x + e * u) - turned(x - e * u)).double() * y).sum() / (2 * e)
    # 6400 products, each off by a few 2^-24 of itself
    assert abs(diff - (grad.double() * u).sum()) < 6400 ** 0.5 * 20 * 2.0 ** -24 * 4


def test_no_tokens_and_capture():
    e = torch.empty(0, 2, 32, device="cuda")
    freq = gdnspec.gdn_rotary_frequencies(32)
    gdnspec.gdn_rotary(e, None, torch.empty(0, dtype=torch.int32, device="cuda"), freq, torch.empty_like(e), None)
    q, out = torch.randn(7, 2, 32, device="cuda"), torch.empty(7, 2, 32, device="cuda")
    pos = torch.arange(7, dtype=torch.int32).cuda()
    gdnspec.gdn_rotary(q, None, pos, freq, out, None)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdnspec.gdn_rotary(q, None, pos, freq, out, None)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and gdnspec.gdn_last_error() == gdnspec.OK
