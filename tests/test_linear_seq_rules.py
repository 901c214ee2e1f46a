"""Rules of the linear-attention kernels' source that hold for each kernel's own text, from its brace to its brace (CPU)."""
import os
import re

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
