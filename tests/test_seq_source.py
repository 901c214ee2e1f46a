"""Rules that the tensor-core kernels' source keeps and no run can show (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_linear_gb300", "csrc")
KERNELS = ("seq_prep_kernel", "seq_fwd_kernel", "seq_bwd_kernel", "seq_grad_kernel")


def body(kernel):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "gdn_seq_tc.cu")).read())
    at = re.search(r"__global__[^;{]*\b%s\(" % kernel, text).end()
    end = text.find("__global__", at)
    return text[at:end if end > 0 else text.find("encode_fn()", at)]


@pytest.mark.parametrize("kernel", KERNELS)
def test_every_barrier_is_initialised_once(kernel):
    """An mbarrier.init on a barrier that is live already is undefined."""
    text = body(kernel)
    single = [re.sub(r"\s", "", a) for a in re.findall(r"\bmbar_init\(([^,;]*),", text)]
    ranges = len(re.findall(r"\binit_barriers\(", text)) + sum("*i" in a for a in single)
    assert len(set(single)) == len(single)
    assert single or ranges
    assert ranges == 0 or (ranges == 1 and not [a for a in single if "*i" not in a])


@pytest.mark.parametrize("kernel", KERNELS)
def test_copies_and_products_end_before_the_cta_does(kernel):
    """After a wait that gave up the CTA waits once more, with a limit: nothing may write to its shared memory or TMEM later."""
    text = body(kernel)
    copies = {re.sub(r"\W.*", "", a.strip()) for a in re.findall(r"\b(?:tma_[23]d|bulk_copy_g2s)\([^;]*,\s*([^,;()]*(?:\([^()]*\))?)\);", text)}
    copies = {"full0" if c == "f" else c for c in copies}
    waited = {re.sub(r"\W.*", "", a.strip()) for a in re.findall(r"\bmbar_wait\(([^,;]*),", text)}
    assert copies and copies <= waited
    # every barrier that a commit arrives on is waited for by all, or the products are by the last commit of their thread
    assert "drain" in waited or waited >= {"bar2", "bar3"}
    # the scans' products may be in flight when their thread ends its loop, whoever gives up later
    drained = re.search(r"(if \(leader && \*dead\)|if \(\*dead\))\s*\{[^{}]*mma_commit\(drain\)", text)
    assert not (kernel in ("seq_fwd_kernel", "seq_bwd_kernel") and drained)
