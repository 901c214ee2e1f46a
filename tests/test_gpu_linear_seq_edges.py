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
