"""Rules of the linear-attention kernels' source that hold for each kernel's own text, from its brace to its brace (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_linear_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def calls(text, name):
    """Argument lists of the calls of `name`, split at their own commas."""
    for m in re.finditer(r"\b%s(?:<[^>;]*>)?\(" % name, text):
        depth, args, start = 1, [], m.end()
        for i in range(m.end(), len(text)):
            depth += {"(": 1, "[": 1, "{": 1, ")": -1, "]": -1, "}": -1}.get(text[i], 0)
            if depth == 0 or (depth == 1 and text[i] == ","):
                args.append(text[start:i].strip())
                start = i + 1
            if depth == 0:
                break
        yield args


def test_wide_stores_ask_for_their_place():
    """A 32-byte store faults on a place of 16 bytes, which outputs, record and workspace may have: never without a flag."""
    found = [a for a in calls(source("gdn_linear_tc.cu"), "stg_pieces")]
    assert found and all(len(a) == 4 for a in found)
    assert not [a for a in found if a[3] == "true"]


KERNELS = ("lin_local_tc_kernel", "lin_rows_tc_kernel", "lin_pairs_tc_kernel")


def body(kernel):
    """A kernel's text from its opening brace to the closing one."""
    text = source("gdn_linear_tc.cu")
    at = re.search(r"__global__[^;{]*\b%s\([^{;]*\{" % kernel, text)
    assert at, kernel
    depth = 1
    for i in range(at.end(), len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at.end():i]
    raise AssertionError("%s does not end" % kernel)


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_kernels_own_text(kernel):
    """Each kernel initialises its barriers once, allocates and frees its tensor memory, and ends copies and products after a wait that gave up."""
    text = body(kernel)
    assert "__global__" not in text and "cudaError_t" not in text
    assert len(re.findall(r"\b(?:mbar_init|init_barriers)\(", text)) == 1
    assert len(re.findall(r"\btmem_alloc\(", text)) == len(re.findall(r"\btmem_dealloc\(", text)) == 1
    again = re.findall(r"wait_here\(([^;]*), a\.err, nullptr\)", text)
    assert any("full0" in a for a in again) and any(re.match(r"(drain|done)\b", a) for a in again)
    assert "rfull" not in text or any("rfull" in a for a in again)
    assert not re.search(r"\bmbar_wait\(|while\s*\(\s*!\s*mbar_test", text)
