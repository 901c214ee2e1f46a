"""The block's norms on the GPU against fp64.

Tolerances, before any run (u = 2^-24): a row's statistics are sums of n products, off by n u at most; each value then
takes a few more roundings.  A gradient subtracts two such terms.  Column sums over R rows are off by R u of the sum of
sizes, which for terms of random sign is sqrt(R) times the root mean square of the sums.  bf16 outputs add 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import seq
from speculative_decoding_linear_gb300 import gdnspec

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def check(got, ref, what, n):
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape and np.isfinite(g).all(), what
    rms = max(np.sqrt(np.mean(ref ** 2)), 1e-30)
    tol = 4 * n * 2.0 ** -24 * rms + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0) * np.abs(ref)
    bad = np.abs(g - ref) > tol
    assert not bad.any(), "%s: %d off, worst %.3g of rms" % (what, bad.sum(), np.abs(g - ref).max() / rms)


def rand(*s, t=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(s, device="cuda") * std + mean).to(t)


def w64(*xs):
    return [None if x is None else x.double().cpu().numpy() for x in xs]


@pytest.mark.parametrize("ot", ["bf16", "f32"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,H,d", [(1, 1, 16), (3, 5, 48), (700, 1, 64), (13, 8, 96), (40, 3, 128), (2500, 2, 256)])
def test_gated_norm(rows, H, d, t, ot):
    torch.manual_seed(rows + d)
    T = TYPES[t]
    o, z, w, dy = rand(rows, H, d, t=TYPES[ot], std=0.3), rand(rows, H, d, t=T, std=3.0), rand(d, t=T), rand(rows, H, d, t=T)
    o[0] = 0.0                     # a row of zeros: r is eps^-1/2
    z[-1, :, 0], z[-1, :, 1] = 120.0, -120.0
    y = torch.full_like(z, float("nan"))
    gdnspec.gdn_gated_norm(o, z, w, y, eps=EPS)
    check(y, seq.gated_norm(*w64(o, z, w), EPS), "y", d + 8)
    do, dz, dw = torch.full_like(o, float("nan")), torch.full_like(z, float("nan")), torch.full((d,), float("nan"), device="cuda")
    ws = gdnspec.empty_norm_workspace(rows * H, d)
    gdnspec.gdn_gated_norm_backward(o, z, w, dy, do, dz, dw, ws, eps=EPS)
    a, b, c = seq.gated_norm_backward(*w64(o, z, w, dy), EPS)
    # the zero row's gradient, eps^-1/2 times dy, is far larger than the others: each part by itself
    check(do[1:], a[1:], "do", 2 * d + 8) if rows > 1 else None
    check(do[:1], a[:1], "do of zeros", 2 * d + 8)
    check(dz, b, "dz", d + 8)
    check(dw, c, "dw", d + 8 + int(np.sqrt(rows * H)) * 4)
    again = torch.empty_like(dw)
    gdnspec.gdn_gated_norm_backward(o, z, w, dy, torch.empty_like(do), torch.empty_like(dz), again, ws, eps=EPS)
    assert torch.equal(dw, again)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("rows,D", [(1, 8), (9, 64), (300, 264), (3000, 504), (65, 1000), (700, 2048), (5, 2560), (3, 4104), (2, 8192)])
def test_block_norm(rows, D, post, t):
    torch.manual_seed(rows + D)
    T = TYPES[t]
    x, w = rand(rows, D, t=T), rand(D, t=T)
    z, wp, g = (rand(rows, D, t=T, std=0.5), rand(D, t=T), rand(D, t=T)) if post else (None, None, None)
    rho = 0.75 if post else 1.0
    h, x2 = torch.full_like(x, float("nan")), torch.full_like(x, float("nan")) if post else None
    gdnspec.gdn_block_norm(x, z, wp, g, w, x2, h, eps=EPS, res_scale=rho)
    rx, rh = seq.block_norm(*w64(x, z, wp, g, w), EPS, rho)
    check(h, rh, "h", 2 * D + 8)
    if post:
        check(x2, rx, "x_out", D + 8)
    at = x2 if post else x
    dh, dx2 = rand(rows, D, t=T), rand(rows, D, t=T)
    dx, dw = torch.full_like(x, float("nan")), torch.full((D,), float("nan"), device="cuda")
    dz, dwp, dg = (torch.full_like(x, float("nan")), torch.empty_like(dw), torch.empty_like(dw)) if post else (None, None, None)
    ws = gdnspec.empty_norm_workspace(rows, D)
    for with_dx2 in (True, False):
        gdnspec.gdn_block_norm_backward(at, z, wp, g, w, dh, dx2 if with_dx2 else None, dx, dz, dwp, dg, dw, ws, eps=EPS,
                                        res_scale=rho)
        y = dx2 if with_dx2 else torch.zeros_like(dx2)
        ref = seq.block_norm_backward(*w64(at, z, wp, g, w, dh, y), EPS, rho)
        n = 2 * D + 8
        for got, r, what in zip((dx, dz, dwp, dg, dw), ref, ("dx", "dz", "dpost_weight", "dgate", "dweight")):
            if r is not None:
                check(got, r, what, n + int(np.sqrt(rows)) * 4)


def test_in_place():
    torch.manual_seed(0)
    x, z, w = rand(70, 2048, t=torch.bfloat16), rand(70, 2048, t=torch.bfloat16), rand(2048, t=torch.bfloat16)
    h, x2 = torch.empty_like(x), torch.empty_like(x)
    gdnspec.gdn_block_norm(x, z, w, w, w, x2, h, eps=EPS)
    a, b = x.clone(), z.clone()
    gdnspec.gdn_block_norm(a, b, w, w, w, a, b, eps=EPS)
    assert torch.equal(a, x2) and torch.equal(b, h)
    o, g = rand(64, 8, 256, t=torch.bfloat16), rand(64, 8, 256, t=torch.bfloat16)
    y = torch.empty_like(o)
    gdnspec.gdn_gated_norm(o, g, w[:256].clone(), y)
    gdnspec.gdn_gated_norm(o, g, w[:256].clone(), o)
    assert torch.equal(o, y)
