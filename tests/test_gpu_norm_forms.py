"""Norm gradients where a CTA takes several rows, and fp32 results beside bf16 gates, on the GPU against fp64."""
import numpy as np
import pytest
import torch

from oracle import seq
from speculative_decoding_linear_gb300 import gdnspec
from test_gpu_norm import EPS, TYPES, check, rand, w64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("rows,D", [(400, 4096), (400, 5120), (400, 8192), (5000, 64), (5000, 256), (1400, 1000)])
def test_block_norm_gradients_over_many_rows(rows, D, post, t):
    torch.manual_seed(rows + D)
    T = TYPES[t]
    x, w, dh, dx2 = rand(rows, D, t=T), rand(D, t=T), rand(rows, D, t=T), rand(rows, D, t=T)
    z, wp, g = (rand(rows, D, t=T, std=0.5), rand(D, t=T), rand(D, t=T)) if post else (None, None, None)
    rho = 0.75 if post else 1.0
    dx, dw = torch.full_like(x, float("nan")), torch.full((D,), float("nan"), device="cuda")
    dz, dwp, dg = (torch.full_like(x, float("nan")), torch.full_like(dw, float("nan")), torch.full_like(dw, float("nan"))) if post else (None,) * 3
    ws = gdnspec.empty_norm_workspace(rows, D)
    ws.fill_(0xFF)
    gdnspec.gdn_block_norm_backward(x, z, wp, g, w, dh, dx2, dx, dz, dwp, dg, dw, ws, eps=EPS, res_scale=rho)
    ref = seq.block_norm_backward(*w64(x, z, wp, g, w, dh, dx2), EPS, rho)
    for got, r, what in zip((dx, dz, dwp, dg, dw), ref, ("dx", "dz", "dpost_weight", "dgate", "dweight")):
        if r is not None:
            check(got, r, what, 2 * D + 8 + int(np.sqrt(rows)) * 4)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(70000, 16), (40000, 32), (9000, 128)])
def test_gated_norm_gradients_over_many_rows(rows, d, t):
    torch.manual_seed(rows + d)
    T = TYPES[t]
    o, z, w, dy = rand(rows, d, t=T, std=0.3), rand(rows, d, t=T), rand(d, t=T), rand(rows, d, t=T)
    do, dz, dw = torch.full_like(o, float("nan")), torch.full_like(z, float("nan")), torch.full((d,), float("nan"), device="cuda")
    ws = gdnspec.empty_norm_workspace(rows, d)
    ws.fill_(0xFF)
    gdnspec.gdn_gated_norm_backward(o, z, w, dy, do, dz, dw, ws, eps=EPS)
    a, b, c = seq.gated_norm_backward(*w64(o, z, w, dy), EPS)
    check(do, a, "do", 2 * d + 8)
    check(dz, b, "dz", d + 8)
    check(dw, c, "dw", d + 8 + int(np.sqrt(rows)) * 4)


@pytest.mark.parametrize("gate", [-60.0, -20.0, -3.0, 2.0])
def test_f32_gradient_beside_bf16_gates(gate):
    """d_o is fp32 where o is: some 16 roundings of 2^-24 in the mean square of a row, whatever the gates' type."""
    torch.manual_seed(5)
    rows, d = 300, 128
    o, w, dy = rand(rows, d), rand(d, t=torch.bfloat16), rand(rows, d, t=torch.bfloat16)
    z = rand(rows, d, t=torch.bfloat16, mean=gate)
    do, dz, dw = torch.empty_like(o), torch.empty_like(z), torch.empty(d, device="cuda")
    gdnspec.gdn_gated_norm_backward(o, z, w, dy, do, dz, dw, gdnspec.empty_norm_workspace(rows, d), eps=EPS)
    ref, _, _ = seq.gated_norm_backward(*w64(o, z, w, dy), EPS)
    err = np.sqrt(((do.double().cpu().numpy() - ref) ** 2).sum(-1) / (ref ** 2).sum(-1))
    assert err.max() <= 16 * 2.0 ** -24
