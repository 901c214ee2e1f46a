"""Argument checks of the sequence operators beyond shapes: alignment, sizes and products of sizes (CPU, no kernel runs)."""
import pytest
import torch

from speculative_decoding_linear_gb300 import build as gbuild
from speculative_decoding_linear_gb300 import gdnspec
from test_seq_oracle import backward_args, far, forward_args

NO_GPU = (gdnspec.ERR_CUDA, gdnspec.ERR_DEVICE)
without_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a valid call would launch on made-up addresses")


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdnspec.lib()


@pytest.mark.parametrize("at", [4, 8, 16, 48])
def test_record_of_bf16_calls_starts_on_32_bytes(L, at):
    """The kernels take a record in 32-byte accesses."""
    assert L.gdn_seq_forward(*forward_args(rec=far(9) + at)) == gdnspec.ERR_ARG
    assert L.gdn_seq_backward(*backward_args(rec=far(8) + at)) == gdnspec.ERR_ARG


@without_gpu
def test_what_16_bytes_are_enough_for(L):
    for dtype in (0, 1):
        assert L.gdn_seq_forward(*forward_args(dtype=dtype, ws=far(10) + 16)) in NO_GPU
        assert L.gdn_seq_backward(*backward_args(dtype=dtype, ws=far(15) + 16)) in NO_GPU
    assert L.gdn_seq_forward(*forward_args(rec=far(9) + 32)) in NO_GPU
    assert L.gdn_seq_forward(*forward_args(dtype=1, rec=far(9) + 16)) in NO_GPU
    assert L.gdn_seq_backward(*backward_args(dtype=1, rec=far(8) + 16)) in NO_GPU


@pytest.mark.parametrize("Hk,dk", [(1 << 23, 256), (1 << 24, 256), (1 << 24, 128)])
def test_rows_wider_than_an_int_counts(L, Hk, dk):
    """No stride is as long as such a row: Hk d_k does not wrap to something smaller."""
    shape = dict(nseq=1, total=1, H=Hk, Hk=Hk, dk=dk, dv=16, ldq=8, ldk=8, ldv=16 * Hk, off=None, dtype=1)
    assert L.gdn_seq_forward(*forward_args(**shape)) == gdnspec.ERR_ARG
    assert L.gdn_seq_backward(*backward_args(**shape)) == gdnspec.ERR_ARG


def test_a_forward_pass_asks_for_the_workspace_that_it_uses(L):
    dims = (1, 8192, 8, 8, 256, 256)
    fwd = gdnspec.gdn_seq_forward_workspace_bytes(*dims, "bf16")
    # the operands of a (chunk, head): 128 x 64 values in two bf16 terms and the gates
    assert 129 * 8 * 2 * 16384 <= fwd <= 129 * 8 * (2 * 16384 + 2048) + 256
    assert 10 * fwd < gdnspec.gdn_seq_workspace_bytes(*dims, "bf16")
    assert gdnspec.gdn_seq_forward_workspace_bytes(*dims, "f32") == 0
    assert L.gdn_seq_forward_workspace_bytes(1, 64, 8, 3, 64, 64, 0, None) == gdnspec.ERR_ARG


@without_gpu
def test_a_forward_workspace_may_end_where_another_array_begins(L):
    n = gdnspec.gdn_seq_forward_workspace_bytes(2, 64, 8, 4, 64, 128, "bf16")
    assert L.gdn_seq_forward(*forward_args(ws=far(0) - n)) in NO_GPU
    assert L.gdn_seq_forward(*forward_args(ws=far(0) - n + 16)) == gdnspec.ERR_ARG
    assert L.gdn_seq_forward(*forward_args(dtype=1, ws=None)) in NO_GPU
    assert L.gdn_seq_forward(*forward_args(dtype=1, ws=far(0) + 16)) in NO_GPU
    assert L.gdn_seq_backward(*backward_args(dtype=1, ws=None)) == gdnspec.ERR_ARG
