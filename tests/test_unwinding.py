"""What a kernel does once a bounded wait has run out, read off the sources (no GPU): a block has to
take the same way with all of its warps, and a warp with all of its lanes, or those that stay wait
for the others at the next barrier or vote without end."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_softmax_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh"))))
def test_a_block_reads_the_timeout_as_one(name):
    """The status word decides whether a block goes on only by way of a vote of the whole block."""
    text = source(name)
    for m in re.finditer(r"== *ATTN_ERR_TIMEOUT", text):
        line = text[text.rfind("\n", 0, m.start()) + 1:text.find("\n", m.end())]
        assert "__syncthreads_or(" in line, line.strip()
