"""What no test can provoke on a GPU without harm, or at all, read from the sources (CPU
only): what the library initialises is complete before a kernel uses it, and no C++
exception leaves a C entry point of the feed-forward block and MXFP4."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_mixture_experts_24_b200",
                    "csrc")


def body(path, name):
    """Text of the function `name`, from its signature to its closing brace in column 0."""
    with open(os.path.join(CSRC, path)) as f:
        text = f.read()
    at = re.search(r"^\w[\w ]* %s\(" % name, text, re.M)
    assert at, "%s has no %s" % (path, name)
    return text[at.start():text.index("\n}", at.start())]


@pytest.mark.parametrize("path,name", [
    ("moe_api.cu", "grow"),             # the forward layer's workspace
    ("ffn_api.cu", "need"),             # status word of the feed-forward block and MXFP4
    ("moe_api.cu", "moe_sync_status"),  # both status words, once they have been reported
])
def test_nothing_is_zeroed_on_the_legacy_stream(path, name):
    """cudaMemset returns before it has run and is ordered on the legacy stream only; a
    non-blocking stream's kernels may come first."""
    assert not re.search(r"\bcudaMemset\(", body(path, name))


def test_no_exception_leaves_a_workspace_that_grows():
    """The list of replaced buffers is the one thing there that may throw (no memory)."""
    text = body("ffn_api.cu", "room")
    at = text.index("kept.push_back")
    assert text.rfind("try {", 0, at) > text.rfind("}", 0, at) and "catch (...)" in text[at:]
