"""Forms of the sequence operators that a call's sizes and addresses choose, on the GPU against the fp64 oracle."""
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
