"""Rules that the linear-attention tensor-core kernels' source keeps and no run can show (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_linear_gb300", "csrc")
KERNELS = ("lin_local_tc_kernel", "lin_rows_tc_kernel", "lin_pairs_tc_kernel")


def body(kernel):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "gdn_linear_tc.cu")).read())
    at = re.search(r"__global__[^;{]*\b%s\(" % kernel, text).end()
    end = text.find("__global__", at)
    return text[at:end if end > 0 else text.find("encode_fn()", at)]


@pytest.mark.parametrize("kernel", KERNELS)
def test_every_barrier_is_initialised_once(kernel):
    """An mbarrier.init on a barrier that is live already is undefined: one loop or list over all of them."""
    text = body(kernel)
    assert len(re.findall(r"\b(?:mbar_init|init_barriers)\(", text)) == 1


@pytest.mark.parametrize("kernel", KERNELS)
def test_copies_and_products_end_before_the_cta_does(kernel):
    """After a wait that gave up the CTA waits once more, with a limit: nothing may write to its shared memory or TMEM later."""
    text = body(kernel)
    again = re.findall(r"wait_here\(([^;]*), a\.err, nullptr\)", text)
    assert any("full0" in a for a in again)                       # the ring's copies
    assert any(re.match(r"(drain|done)\b", a) for a in again)     # the products
    if "rfull" in text:
        assert any("rfull" in a for a in again)                   # the rows' operand
    # no wait without a limit
    assert not re.search(r"\bmbar_wait\(|while\s*\(\s*!\s*mbar_test", text)


def test_kernels_wait_for_the_ones_before_them():
    """Launches overlap: a kernel reads and writes memory that others use only behind its wait for them."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "gdn_linear_tc.cu")).read() + open(os.path.join(CSRC, "gdn_linear_seq.cu")).read())
    kernels = [m.end() for m in re.finditer(r"__global__[^;{]*\b(lin_\w+)\(", text)]
    assert len(kernels) >= 10
    for at in kernels:
        head = text[at:text.index("griddep_launch();", at)]
        assert "griddep_wait();" in head
        assert not re.search(r"zero_rows|slot_entry\(|ld4<|tma_\dd\(|bulk_copy", head)
