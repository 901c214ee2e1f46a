"""The rotary oracle at far positions against whole-number arithmetic (CPU)."""
import numpy as np
import pytest

from oracle import linear_seq as ref
from test_gpu_linear_seq_edges import turns_of


@pytest.mark.parametrize("inverse", [False, True])
def test_far_positions(inverse):
    """Angles up to 2^32 rad: 2^32 x 2^-64 of a product in extended precision, and as much of what is taken off: 1e-9 and more."""
    freqs = np.array([1.0, 0.7, -0.37, 2.0 ** -20, 1e-4, 1.9], np.float32).astype(np.float64)
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -987654321, 4095, 0, 1])
    x = np.zeros((len(pos), 1, 12))
    x[..., :6] = 1.0
    y = ref.rotary(x, pos, freqs, inverse=inverse)[:, 0]
    t = 2 * np.pi * turns_of(pos.tolist(), freqs.tolist()) * (-1 if inverse else 1)
    assert np.abs(y[:, :6] - np.cos(t)).max() < 2e-9 and np.abs(y[:, 6:] - np.sin(t)).max() < 2e-9
