"""The blocks example runs: training lowers its loss, decode continues prefill, a draft chain agrees with the sequence."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_blocks_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gdn_blocks.py")
    spec = importlib.util.spec_from_file_location("gdn_blocks", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, step_err, state_err, tree_err = m.main()
    assert losses[-1] < losses[0]
    # bf16 activations: each of a block's roundings is 2^-9 of its value in the mean, some ten of them a block
    assert step_err < 2 * 10 * 2.0 ** -9 and state_err < 2 * 10 * 2.0 ** -9
    assert tree_err < 2.0 ** -8
